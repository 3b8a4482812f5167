// The 8-bit key-value cache: rows added to sequences (kv8_append) and read back
// (kv8_load).  Layout and format: kv8.cuh.
//
// Append: a warp takes one block of one head, K then V.  It has all of the block's
// new rows in registers, finds their largest magnitude (integer maxima of the bits,
// one redux), and writes codes at the scale of the block: what the new rows need,
// or the one that is there if it is larger.  Where a block with earlier rows grows,
// these are rounded again.  A lane takes 16 bytes of a row at a time, so every access
// is whole sectors.
//
// Load: a thread writes two vectors of 16 bytes of a K row and of a V row.
//
// Both move bytes, and are bound by HBM: a token and head of d features is 4 d bytes of
// bf16 and 2 d + 1 of cache.  8192 tokens x 80 heads of 128, 504 MB, replayed from a graph:
// append 73 us, load 74, in random order 77 (6.5 to 6.9 TB/s; the last writes are still in
// L2 then), launched one by one 77; as many bytes of d = 64: 74, 75 and 97, of d = 96 (a lane in
// four idle, rows of two lines) 87, 75 and 93, of d = 32 90, 76 and 128.  One row of 32
// sequences: latency, 3.5 us and 2.3.
#include <type_traits>

#include "kv8.cuh"

namespace iha {
namespace {

IHA_DEVICE_ERROR_WORD(kv8_cache)

constexpr int kWarps = 4;  // (8192 tokens x 80 heads: 73 us, 8 warps 80)

struct AppendParams {
  const void *k, *v;
  const int32_t *table, *lens, *counts;
  uint8_t* cache;
  iha_strides sk, sv;
  FastDiv heads, blocks;  // heads; blocks that one call can touch of a sequence
  int64_t items;
  Kv8Pages pages;
  int N, n_pages, page, table_w;
};

// 16 bytes of a row: the largest magnitude as fp32 bits (infinite or above: not finite).
template <typename T>
__device__ __forceinline__ uint32_t magnitude(const uint4& u);
template <>
__device__ __forceinline__ uint32_t magnitude<__nv_bfloat16>(const uint4& u) {
  uint32_t m = __vmaxu2(u.x & 0x7FFF7FFFu, u.y & 0x7FFF7FFFu);
  m = __vmaxu2(m, __vmaxu2(u.z & 0x7FFF7FFFu, u.w & 0x7FFF7FFFu));
  return max(m << 16, m & 0xFFFF0000u);
}
template <>
__device__ __forceinline__ uint32_t magnitude<float>(const uint4& u) {
  return max(max(u.x & 0x7FFFFFFFu, u.y & 0x7FFFFFFFu), max(u.z & 0x7FFFFFFFu, u.w & 0x7FFFFFFFu));
}
// ... times f, as codes, to cache memory.
__device__ __forceinline__ void encode(uint8_t* to, const uint4& u, float f, __nv_bfloat16) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
  uint32_t c[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    c[i] = e4m3_pair(bf16lo_to_f32(w[2 * i]) * f, bf16hi_to_f32(w[2 * i]) * f) |
           (uint32_t)e4m3_pair(bf16lo_to_f32(w[2 * i + 1]) * f, bf16hi_to_f32(w[2 * i + 1]) * f)
               << 16;
  *reinterpret_cast<uint2*>(to) = make_uint2(c[0], c[1]);
}
__device__ __forceinline__ void encode(uint8_t* to, const uint4& u, float f, float) {
  *reinterpret_cast<uint32_t*>(to) =
      e4m3_pair(__uint_as_float(u.x) * f, __uint_as_float(u.y) * f) |
      (uint32_t)e4m3_pair(__uint_as_float(u.z) * f, __uint_as_float(u.w) * f) << 16;
}

// ITER: iterations that hold a block's new rows, from the first on.
template <typename T, int D, int ITER>
__global__ void __launch_bounds__(32 * kWarps) kv8_append_kernel(const AppendParams p) {
  constexpr int V = 16 / sizeof(T);            // features of a lane
  constexpr int LPR = D / V, RPI = 32 / LPR;   // lanes of a row, rows at once
  constexpr bool BOTH = ITER <= 8;             // K and V are loaded before either is used
  const int lane = threadIdx.x & 31;
  const int64_t id64 = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (id64 >= p.items) return;
  const int id = (int)id64, rest = p.heads.div(id), head = id - rest * p.heads.d;
  const int b = p.blocks.div(rest), nth = rest - b * p.blocks.d;

  const int raw = __ldg(p.lens + b), len = min(max(raw, 0), p.table_w * p.page);
  const int want = p.counts ? __ldg(p.counts + b) : p.N, cnt = min(max(want, 0), p.N);
  if ((raw != len || want != cnt) && nth == 0 && head == 0 && lane == 0)
    atomicOr(&g_dev_error, DEV_ERR_CACHE_INDEX);
  const int first = max(0, len - cnt);  // the first new position
  const int blk = first / kKv8Tok + nth, pos0 = blk * kKv8Tok;
  if (first >= len || pos0 >= len) return;
  const int bpp = p.pages.bpp, pi = blk / bpp, page_id = __ldg(p.table + (int64_t)b * p.table_w + pi);
  const int had = max(0, first - pos0), end = min(len - pos0, kKv8Tok);  // new rows [had, end)
  const int r = lane / LPR, c = lane - r * LPR;  // row of an iteration, vector of the row

  auto load = [&](int which, uint4 (&x)[ITER]) {
    const iha_strides& st = which ? p.sv : p.sk;
    const T* src = static_cast<const T*>(which ? p.v : p.k) + b * st.b_outer + head * st.head +
                   (int64_t)(pos0 + had - (len - p.N)) * st.seq + c * V;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      x[i] = make_uint4(0, 0, 0, 0);
      if (r < RPI && had + i * RPI + r < end)
        x[i] = __ldg(reinterpret_cast<const uint4*>(src + (i * RPI + r) * st.seq));
    }
  };
  uint4 xk[ITER], xv[ITER];
  load(0, xk);
  if (BOTH) load(1, xv);

  if (page_id < 0 || page_id >= p.n_pages) {
    if (lane == 0) atomicOr(&g_dev_error, DEV_ERR_CACHE_INDEX);
    return;
  }
  uint8_t* const base = p.cache + p.pages.block(page_id, head, blk - pi * bpp, D);
  uint8_t* const tail_at = p.cache + p.pages.tail(page_id, head, blk - pi * bpp);
  Kv8Tail tail = {{0.f, 0.f}, 0u, 0u};
  if (had > 0) tail = kv8_tail(tail_at);

  const uint32_t row_lanes =
      LPR == 32 ? ~0u : ((1u << (LPR % 32)) - 1u) << (r * LPR % 32);
  auto store = [&](uint8_t* rows, uint4 (&x)[ITER], float old, int before_bit, float& scale) {
    uint32_t top = 0, nan = 0;
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      uint32_t m = magnitude<T>(x[i]);
      const uint32_t bad = __ballot_sync(0xffffffffu, m >= 0x7F800000u);
      if (bad != 0 && r < RPI && (bad & row_lanes) != 0) {  // a row of NaN: codes of 0
        m = 0;
        x[i] = make_uint4(0, 0, 0, 0);
        nan |= 1u << (had + i * RPI + r);
      }
      top = max(top, m);
    }
    top = __reduce_max_sync(0xffffffffu, top);
    nan = __reduce_or_sync(0xffffffffu, nan);
    // 448 = 1.75 * 2^8
    int e = max((int)(top >> 23) - 127 - 8 + ((top & 0x7FFFFFu) > 0x600000u ? 1 : 0), kKv8LowestE);
    const int before = kv8_exponent(old);
    if (had > 0) e = max(e, before);
    const float f = kv8_two(-e), again = kv8_two(before - e);
    auto at = [&](int row) {  // the lane's codes of a row
      return rows + row * D + (((c * V / 16) ^ kv8_swap(D, row)) * 16 + c * V % 16);
    };
#pragma unroll
    for (int i = 0; i < ITER; ++i) {
      const int row = had + i * RPI + r;
      if (r < RPI && row < end) encode(at(row), x[i], f, T());
    }
    // rows behind the last one of a fresh block become zeros; earlier ones of a block
    // that grows are rounded again
    const int other0 = had > 0 ? 0 : end, other1 = had > 0 ? (e > before ? had : 0) : kKv8Tok;
#pragma unroll 1
    for (int row = other0 + r; row < other1; row += RPI)
      if (r < RPI) {
        uint32_t* w = reinterpret_cast<uint32_t*>(at(row));
#pragma unroll
        for (int j = 0; j < V / 4; ++j) w[j] = had > 0 ? e4m3_rescale(w[j], again) : 0u;
      }
    scale = kv8_two(e);
    const uint32_t fresh = ((1u << end) - 1u) & ~((1u << had) - 1u);
    tail.nan = (tail.nan & ~(fresh << before_bit)) | (nan << before_bit);
  };
  float sk, sv;
  store(base, xk, tail.scale[0], 0, sk);
  if (!BOTH) load(1, xv);
  store(base + kKv8Tok * D, xv, tail.scale[1], 16, sv);
  if (lane == 0)
    *reinterpret_cast<uint4*>(tail_at) =
        make_uint4(__float_as_uint(sk), __float_as_uint(sv), tail.nan, 0u);
}

template <typename T, int D>
void launch_append(const AppendParams& p, unsigned grid, cudaStream_t s) {
  constexpr int RPI = 32 / (D / (16 / (int)sizeof(T))), FULL = (kKv8Tok + RPI - 1) / RPI;
  // few new rows of a block: forms that hold no more, and load K and V before the table and
  // the block's scales have come (32 sequences x 80 heads of 128, one row each: with the
  // next call that reads them back 7.2 us, by the long form 11.1)
  if (p.N <= RPI)
    kv8_append_kernel<T, D, 1><<<grid, 32 * kWarps, 0, s>>>(p);
  else if (FULL > 4 && p.N <= 4 * RPI)
    kv8_append_kernel<T, D, 4><<<grid, 32 * kWarps, 0, s>>>(p);
  else
    kv8_append_kernel<T, D, FULL><<<grid, 32 * kWarps, 0, s>>>(p);
}

struct LoadParams {
  const uint8_t* cache;
  const int32_t* slots;
  void *k, *v;
  iha_strides sk, sv;
  FastDiv heads, N, Bi, page;  // heads; as kv4_load
  int64_t items;
  Kv8Pages pages;
  int n_slots;
};

// Codes of 16 bytes of values: 8 bf16 (the products are exact), 4 fp32.
template <typename T>
using Codes = typename std::conditional<sizeof(T) == 2, uint2, uint32_t>::type;
__device__ __forceinline__ uint4 decode(uint2 c, float s, bool nan) {
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = e4m3_to_f16((uint16_t)((i < 2 ? c.x : c.y) >> (16 * (i & 1))));
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
    v[i] = nan ? 0x7FC07FC0u : pack_bf16x2(x.x * s, x.y * s);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ uint4 decode(uint32_t c, float s, bool nan) {
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t h = e4m3_to_f16((uint16_t)(c >> (16 * i)));
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
    v[2 * i] = nan ? 0x7FC00000u : __float_as_uint(x.x * s);
    v[2 * i + 1] = nan ? 0x7FC00000u : __float_as_uint(x.y * s);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}

// A thread: two vectors of a row, half a row apart (a warp's stores are whole sectors).
template <typename T, int D>
__global__ void __launch_bounds__(256) kv8_load_kernel(const LoadParams p) {
  constexpr int V = 16 / sizeof(T), TPR = D / V / 2;  // threads of a row
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (id >= p.items) return;
  const int row = (int)(id / TPR), c = (int)(id - (int64_t)row * TPR);
  const int tok = p.heads.div(row), head = row - tok * p.heads.d;
  const int slot = __ldg(p.slots + tok);
  const bool in = slot >= 0 && slot < p.n_slots;
  if (!in && slot != -1) atomicOr(&g_dev_error, DEV_ERR_CACHE_INDEX);
  uint4 k[2], v[2];
  k[0] = k[1] = v[0] = v[1] = make_uint4(0, 0, 0, 0);
  if (in) {
    const int pg = p.page.div(slot), off = slot - pg * p.page.d, r = off % kKv8Tok;
    const uint8_t* blk = p.cache + p.pages.block(pg, head, off / kKv8Tok, D);
    const Kv8Tail t = kv8_tail(p.cache + p.pages.tail(pg, head, off / kKv8Tok));
    Codes<T> ck[2], cv[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int f = (c + q * TPR) * V;  // the vector's first feature
      const uint8_t* at = blk + r * D + (((f / 16) ^ kv8_swap(D, r)) * 16 + f % 16);
      ck[q] = *reinterpret_cast<const Codes<T>*>(at);
      cv[q] = *reinterpret_cast<const Codes<T>*>(at + kKv8Tok * D);
    }
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      k[q] = decode(ck[q], t.scale[0], (t.nan >> r) & 1u);
      v[q] = decode(cv[q], t.scale[1], (t.nan >> (16 + r)) & 1u);
    }
  }
  const int b = p.N.div(tok), n = tok - b * p.N.d, bo = p.Bi.div(b), bi = b - bo * p.Bi.d;
  T* yk = static_cast<T*>(p.k) + bo * p.sk.b_outer + bi * p.sk.b_inner + n * p.sk.seq +
          head * p.sk.head + c * V;
  T* yv = static_cast<T*>(p.v) + bo * p.sv.b_outer + bi * p.sv.b_inner + n * p.sv.seq +
          head * p.sv.head + c * V;
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    *reinterpret_cast<uint4*>(yk + q * TPR * V) = k[q];
    *reinterpret_cast<uint4*>(yv + q * TPR * V) = v[q];
  }
}

// Checks of k, v views that append and load share; strides of extents of 1 become 0.
iha_status check_rows(const char* name, const void* k, const void* v, int Bo, int Bi, int N, int H,
                      int d, iha_strides& sk, iha_strides& sv, iha_dtype dt, int64_t* bk,
                      int64_t* bv) {
  if (dt != IHA_BF16 && dt != IHA_F32) return fail(IHA_ERR_INVALID_ARG, "%s: bad dtype", name);
  const int es = dt == IHA_BF16 ? 2 : 4;
  if (!aligned16(k) || !aligned16(v))
    return fail(IHA_ERR_ALIGNMENT, "%s: k and v must be 16-byte aligned", name);
  for (iha_strides* t : {&sk, &sv}) {
    if (Bo == 1) t->b_outer = 0;
    if (Bi == 1) t->b_inner = 0;
    if (N == 1) t->seq = 0;
    if (H == 1) t->head = 0;
  }
  if (!strides_ok(sk, es) || !strides_ok(sv, es))
    return fail(IHA_ERR_ALIGNMENT, "%s: strides must be multiples of 16 bytes", name);
  bool nk, nv;
  *bk = view_bytes(sk, Bo, Bi, N, H, d, es, &nk);
  *bv = view_bytes(sv, Bo, Bi, N, H, d, es, &nv);
  if (nk || nv) return fail(IHA_ERR_INVALID_ARG, "%s: negative stride", name);
  return IHA_OK;
}

}  // namespace

iha_status kv8_check_cache(const char* name, const void* cache, int n_pages, int page, int Hkv,
                           int d) {
  if (n_pages <= 0 || page <= 0 || Hkv <= 0 || d <= 0)
    return fail(IHA_ERR_INVALID_ARG, "%s: sizes must be positive", name);
  if (d % 32 || d > 128)
    return fail(IHA_ERR_UNSUPPORTED, "%s: needs d in {32, 64, 96, 128}, got %d", name, d);
  if (page % kKv8Tok)
    return fail(IHA_ERR_UNSUPPORTED, "%s: page size %d is not a multiple of %d", name, page,
                kKv8Tok);
  if ((int64_t)n_pages * page > INT32_MAX)
    return fail(IHA_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 slots", name);
  if (!aligned16(cache))
    return fail(IHA_ERR_ALIGNMENT, "%s: the cache must be 16-byte aligned", name);
  return IHA_OK;
}

}  // namespace iha

extern "C" {

size_t kv8_page_bytes(int page, int Hkv, int d) {
  if (page <= 0 || page % iha::kKv8Tok || Hkv <= 0 || d <= 0 || d % 32 || d > 128) return 0;
  iha::Kv8Pages pages;
  pages.set(page, Hkv, d);
  return (size_t)pages.bytes;
}

iha_status kv8_append(const void* k, const void* v, const int32_t* block_table,
                      const int32_t* seq_lens, const int32_t* counts, void* cache, int B, int N,
                      int n_pages, int page, int table_width, int Hkv, int d, iha_strides sk,
                      iha_strides sv, iha_dtype dt, void* stream) {
  using namespace iha;
  const char* name = "kv8_append";
  if (!k || !v || !block_table || !seq_lens || !cache)
    return fail(IHA_ERR_INVALID_ARG, "%s: null pointer", name);
  if (B <= 0 || N <= 0 || table_width <= 0)
    return fail(IHA_ERR_INVALID_ARG, "%s: sizes must be positive", name);
  iha_status st = kv8_check_cache(name, cache, n_pages, page, Hkv, d);
  if (st != IHA_OK) return st;
  sk.b_inner = sv.b_inner = 0;
  int64_t bk, bv;
  st = check_rows(name, k, v, B, 1, N, Hkv, d, sk, sv, dt, &bk, &bv);
  if (st != IHA_OK) return st;
  if ((reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(seq_lens) |
       reinterpret_cast<uintptr_t>(counts)) & 3)
    return fail(IHA_ERR_ALIGNMENT, "%s: block_table, seq_lens and counts must be 4-byte aligned",
                name);
  if ((int64_t)table_width * page > (1 << 30))
    return fail(IHA_ERR_UNSUPPORTED, "%s: block table longer than 2^30 tokens", name);
  const int64_t bc = (int64_t)n_pages * kv8_page_bytes(page, Hkv, d);
  if (overlaps(cache, bc, k, bk) || overlaps(cache, bc, v, bv) ||
      overlaps(cache, bc, block_table, (int64_t)B * table_width * 4) ||
      overlaps(cache, bc, seq_lens, (int64_t)B * 4) ||
      (counts && overlaps(cache, bc, counts, (int64_t)B * 4)))
    return fail(IHA_ERR_INVALID_ARG, "%s: the cache overlaps another buffer", name);
  AppendParams p;
  p.k = k;
  p.v = v;
  p.table = block_table;
  p.lens = seq_lens;
  p.counts = counts;
  p.cache = static_cast<uint8_t*>(cache);
  p.sk = sk;
  p.sv = sv;
  p.N = N;
  p.n_pages = n_pages;
  p.page = page;
  p.pages.set(page, Hkv, d);
  p.table_w = table_width;
  // N neighbours touch at most this many blocks, a table no more than it has
  const int64_t touched = ((int64_t)N + 2 * kKv8Tok - 2) / kKv8Tok;
  const int64_t most = (int64_t)table_width * p.pages.bpp;
  p.blocks.set((int)(touched < most ? touched : most));
  p.heads.set(Hkv);
  p.items = (int64_t)B * p.blocks.d * Hkv;
  if (p.items > INT32_MAX)
    return fail(IHA_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 blocks in one call", name);
  const unsigned grid = (unsigned)((p.items + kWarps - 1) / kWarps);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  IHA_KV8_D_SWITCH(d, {
    if (dt == IHA_BF16)
      launch_append<__nv_bfloat16, kD>(p, grid, s);
    else
      launch_append<float, kD>(p, grid, s);
  })
  return check_launch(name);
}

iha_status kv8_load(const void* cache, const int32_t* slots, void* k, void* v, int B_outer,
                    int B_inner, int N, int n_pages, int page, int Hkv, int d, iha_strides sk,
                    iha_strides sv, iha_dtype dt, void* stream) {
  using namespace iha;
  const char* name = "kv8_load";
  if (!k || !v || !slots || !cache) return fail(IHA_ERR_INVALID_ARG, "%s: null pointer", name);
  if (B_outer <= 0 || B_inner <= 0 || N <= 0)
    return fail(IHA_ERR_INVALID_ARG, "%s: sizes must be positive", name);
  iha_status st = kv8_check_cache(name, cache, n_pages, page, Hkv, d);
  if (st != IHA_OK) return st;
  int64_t bk, bv;
  st = check_rows(name, k, v, B_outer, B_inner, N, Hkv, d, sk, sv, dt, &bk, &bv);
  if (st != IHA_OK) return st;
  if (reinterpret_cast<uintptr_t>(slots) & 3)
    return fail(IHA_ERR_ALIGNMENT, "%s: slots must be 4-byte aligned", name);
  const int64_t toks = (int64_t)B_outer * B_inner * N, rows = toks * Hkv;
  if (toks > INT32_MAX - 1 || rows > INT32_MAX)
    return fail(IHA_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 rows in one call", name);
  const int64_t bc = (int64_t)n_pages * kv8_page_bytes(page, Hkv, d);
  if (overlaps(cache, bc, k, bk) || overlaps(cache, bc, v, bv) ||
      overlaps(k, bk, slots, toks * 4) || overlaps(v, bv, slots, toks * 4))
    return fail(IHA_ERR_INVALID_ARG, "%s: an output overlaps another tensor", name);
  const int es = dt == IHA_BF16 ? 2 : 4;
  for (const iha_strides* t : {&sk, &sv}) {
    const Kv4View w = {4, {B_outer, B_inner, N, Hkv}, {t->b_outer, t->b_inner, t->seq, t->head}};
    if ((B_outer > 1 && t->b_outer == 0) || (B_inner > 1 && t->b_inner == 0) ||
        (N > 1 && t->seq == 0) || (Hkv > 1 && t->head == 0) || kv4_views_meet(w, w, 0, d, true))
      return fail(IHA_ERR_INVALID_ARG, "%s: rows of an output overlap one another", name);
  }
  const Kv4View wk = {4, {B_outer, B_inner, N, Hkv}, {sk.b_outer, sk.b_inner, sk.seq, sk.head}};
  const Kv4View wv = {4, {B_outer, B_inner, N, Hkv}, {sv.b_outer, sv.b_inner, sv.seq, sv.head}};
  const int64_t apart = static_cast<const char*>(v) - static_cast<const char*>(k);
  if (overlaps(k, bk, v, bv) && kv4_views_meet(wk, wv, apart / es, d, false))
    return fail(IHA_ERR_INVALID_ARG, "%s: the outputs overlap one another", name);
  LoadParams p;
  p.cache = static_cast<const uint8_t*>(cache);
  p.slots = slots;
  p.k = k;
  p.v = v;
  p.sk = sk;
  p.sv = sv;
  p.heads.set(Hkv);
  p.N.set(N);
  p.Bi.set(B_inner);
  p.page.set(page);
  p.items = rows * (d * es / 32);
  p.n_slots = n_pages * page;
  p.pages.set(page, Hkv, d);
  const int64_t ctas = (p.items + 255) / 256;
  if (ctas > INT32_MAX)
    return fail(IHA_ERR_UNSUPPORTED, "%s: too many rows in one call", name);
  const unsigned grid = (unsigned)ctas;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  IHA_KV8_D_SWITCH(d, {
    if (dt == IHA_BF16)
      kv8_load_kernel<__nv_bfloat16, kD><<<grid, 256, 0, s>>>(p);
    else
      kv8_load_kernel<float, kD><<<grid, 256, 0, s>>>(p);
  })
  return check_launch(name);
}

}  // extern "C"
