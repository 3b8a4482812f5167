// The 4-bit key-value cache: rows quantised as they are written (kv4_store)
// and read back (kv4_load).  Layout and format: kv4.cuh.
//
// Both are byte movers.  Writing a token and head of d features reads 2 d
// values (4 d bytes of bf16) and writes d + d / 8 bytes; reading back moves
// the same bytes the other way.  A thread owns 8 neighbouring features, the
// four threads of a group of 32 find its maximum with two shuffles.
//
// Rounding x / s without a division per value: y = x * (1 / s) is off by at
// most 2^-21 (|y| < 7.1, one rounding of the reciprocal), and x / s of a bf16
// x and a bf16 s is either exactly half-way between two codes or at least
// 1 / 512 away from it (2 x and (2 k + 1) s are 8-bit integers times powers of
// two, so they differ by at least the smaller unit or not at all).  So y is
// first rounded to a multiple of 2^-14 by adding 776 in the same FMA (776 =
// 768 + 8 also shifts the code to its nibble), which puts half-way cases
// exactly half-way, and then to an integer, ties to even, by adding
// 1.5 * 2^23.
#include "kv4.cuh"

namespace iha {
namespace {

IHA_DEVICE_ERROR_WORD(kv4_cache)

struct Kv4Geom {
  int N, H, page, blocks_per_page;  // tokens of a batch row, heads
  int n_slots;                      // n_pages * page
  int64_t rows;                     // B_outer * B_inner * N * H
  int Bi;
};

template <typename T>
__device__ __forceinline__ void load8(const T* p, uint32_t (&v)[4]);  // 8 values as bf16 pairs
template <>
__device__ __forceinline__ void load8<__nv_bfloat16>(const __nv_bfloat16* p, uint32_t (&v)[4]) {
  const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
  v[0] = u.x;
  v[1] = u.y;
  v[2] = u.z;
  v[3] = u.w;
}
template <>
__device__ __forceinline__ void load8<float>(const float* p, uint32_t (&v)[4]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p));
  const float4 b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = pack_bf16x2(a.x, a.y);  // round to nearest even; NaN and infinity stay
  v[1] = pack_bf16x2(a.z, a.w);
  v[2] = pack_bf16x2(b.x, b.y);
  v[3] = pack_bf16x2(b.z, b.w);
}

// 8 features -> their code word and the group's scale (the four lanes of the
// group call together).  A group with a NaN or an infinity has scale NaN and
// zero codes, so that it reads back as NaN.
__device__ __forceinline__ uint32_t quantise8(const uint32_t (&v)[4], uint32_t& scale_bits) {
  uint32_t m2 = 0;  // largest magnitudes of the even and the odd features, as bits
#pragma unroll
  for (int i = 0; i < 4; ++i) m2 = __vmaxu2(m2, v[i] & 0x7FFF7FFFu);
  uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
  const float top = __uint_as_float(m << 16);
  uint32_t word = 0x88888888u;
  scale_bits = 0;
  if (m >= 0x7F80u) {
    scale_bits = 0x7FC0u;
  } else if (top >= kKv4Tiny) {
    const float s = __bfloat162float(__float2bfloat16_rn(__fdiv_rn(top, 7.f)));
    scale_bits = __float_as_uint(s) >> 16;
    const float inv = __frcp_rn(s);
    word = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = (e & 1) ? bf16hi_to_f32(v[e >> 1]) : bf16lo_to_f32(v[e >> 1]);
      const float r = fmaf(x, inv, 776.f) + 12582912.f;
      word |= (__float_as_uint(r) & 15u) << (4 * e);
    }
  }
  return word;
}

// One thread per 8 features of a row; a row is (batch, token, head).
template <typename T, int NG>
__global__ void __launch_bounds__(256)
    kv4_store_kernel(const T* __restrict__ k, const T* __restrict__ v,
                     const int32_t* __restrict__ slots, uint8_t* __restrict__ cache, Kv4Geom g,
                     iha_strides sk, iha_strides sv) {
  constexpr int TPR = 4 * NG;  // threads per row
  const int64_t gi = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = gi / TPR;
  const int o = (int)(gi - row * TPR);  // octet of the row
  const bool live = row < g.rows;
  const int64_t r = live ? row : 0;
  const int64_t tok = r / g.H;
  const int head = (int)(r - tok * g.H);
  const int64_t b = tok / g.N;
  const int n = (int)(tok - b * g.N);
  const int64_t bo = b / g.Bi, bi = b - bo * g.Bi;
  const int slot = __ldg(slots + tok);
  const bool in = slot >= 0 && slot < g.n_slots;
  if (live && !in && slot != -1) atomicOr(&g_dev_error, DEV_ERR_CACHE_INDEX);
  const int pg = in ? slot / g.page : 0, off = in ? slot - pg * g.page : 0;
  uint8_t* blk = cache + kv4_block_of(pg, off / kKv4Tok, head, g.H, g.blocks_per_page, NG);
  const int tk = off % kKv4Tok;
  const int j = o >> 2, t = o & 3;
  uint32_t x[4], sc;
  load8<T>(k + bo * sk.b_outer + bi * sk.b_inner + n * sk.seq + head * sk.head + o * 8, x);
  const uint32_t kw = quantise8(x, sc);
  if (live && in) {
    *reinterpret_cast<uint32_t*>(blk + kv4_k_word(NG, tk, t, j)) = kw;
    if (t == 0)
      *reinterpret_cast<uint16_t*>(blk + kv4_k_scales(NG) + kv4_scale(NG, tk, j)) = (uint16_t)sc;
  }
  load8<T>(v + bo * sv.b_outer + bi * sv.b_inner + n * sv.seq + head * sv.head + o * 8, x);
  const uint32_t vw = quantise8(x, sc);
  if (live && in) {
    *reinterpret_cast<uint16_t*>(blk + kv4_v_half(NG, tk, 2 * t, j)) = (uint16_t)vw;
    *reinterpret_cast<uint16_t*>(blk + kv4_v_half(NG, tk, 2 * t + 1, j)) = (uint16_t)(vw >> 16);
    if (t == 0)
      *reinterpret_cast<uint16_t*>(blk + kv4_v_scales(NG) + kv4_scale(NG, tk, j)) = (uint16_t)sc;
  }
}

// Code word and scale -> 8 values, written as T (s * c is exact in fp32; the
// bf16 form rounds once, to nearest even).
template <typename T>
__device__ __forceinline__ void write8(T* p, uint32_t word, float s);
template <>
__device__ __forceinline__ void write8<__nv_bfloat16>(__nv_bfloat16* p, uint32_t word, float s) {
  uint32_t u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    u[i] = pack_bf16x2(s * (float)((int)((word >> (8 * i)) & 15u) - 8),
                       s * (float)((int)((word >> (8 * i + 4)) & 15u) - 8));
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
template <>
__device__ __forceinline__ void write8<float>(float* p, uint32_t word, float s) {
  float f[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) f[e] = s * (float)((int)((word >> (4 * e)) & 15u) - 8);
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

template <typename T, int NG>
__global__ void __launch_bounds__(256)
    kv4_load_kernel(const uint8_t* __restrict__ cache, const int32_t* __restrict__ slots,
                    T* __restrict__ k, T* __restrict__ v, Kv4Geom g, iha_strides sk,
                    iha_strides sv) {
  constexpr int TPR = 4 * NG;
  const int64_t gi = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = gi / TPR;
  if (row >= g.rows) return;
  const int o = (int)(gi - row * TPR);
  const int64_t tok = row / g.H;
  const int head = (int)(row - tok * g.H);
  const int64_t b = tok / g.N;
  const int n = (int)(tok - b * g.N);
  const int64_t bo = b / g.Bi, bi = b - bo * g.Bi;
  const int slot = __ldg(slots + tok);
  const bool in = slot >= 0 && slot < g.n_slots;
  if (!in && slot != -1) atomicOr(&g_dev_error, DEV_ERR_CACHE_INDEX);
  const int j = o >> 2, t = o & 3;
  uint32_t kw = 0x88888888u, vw = 0x88888888u;
  float ks = 0.f, vs = 0.f;
  if (in) {
    const int pg = slot / g.page, off = slot - pg * g.page, tk = off % kKv4Tok;
    const uint8_t* blk =
        cache + kv4_block_of(pg, off / kKv4Tok, head, g.H, g.blocks_per_page, NG);
    kw = *reinterpret_cast<const uint32_t*>(blk + kv4_k_word(NG, tk, t, j));
    vw = *reinterpret_cast<const uint16_t*>(blk + kv4_v_half(NG, tk, 2 * t, j)) |
         ((uint32_t)*reinterpret_cast<const uint16_t*>(blk + kv4_v_half(NG, tk, 2 * t + 1, j))
          << 16);
    ks = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(
                             blk + kv4_k_scales(NG) + kv4_scale(NG, tk, j))
                         << 16);
    vs = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(
                             blk + kv4_v_scales(NG) + kv4_scale(NG, tk, j))
                         << 16);
  }
  write8<T>(k + bo * sk.b_outer + bi * sk.b_inner + n * sk.seq + head * sk.head + o * 8, kw, ks);
  write8<T>(v + bo * sv.b_outer + bi * sv.b_inner + n * sv.seq + head * sv.head + o * 8, vw, vs);
}

bool strides_ok(const iha_strides& s, int es) {
  const int64_t m = 16 / es;
  return s.b_outer % m == 0 && s.b_inner % m == 0 && s.seq % m == 0 && s.head % m == 0;
}

// Bytes from the first to one past the last element of a strided view.
int64_t view_bytes(const iha_strides& s, int Bo, int Bi, int N, int H, int d, int es, bool* neg) {
  *neg = s.b_outer < 0 || s.b_inner < 0 || s.seq < 0 || s.head < 0;
  return ((int64_t)(Bo - 1) * s.b_outer + (int64_t)(Bi - 1) * s.b_inner +
          (int64_t)(N - 1) * s.seq + (int64_t)(H - 1) * s.head + d) *
         es;
}

bool overlaps(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

#define IHA_NG_SWITCH(NG, ...)                                  \
  switch (NG) {                                                 \
    case 1: { constexpr int kNG = 1; __VA_ARGS__; } break;      \
    case 2: { constexpr int kNG = 2; __VA_ARGS__; } break;      \
    case 3: { constexpr int kNG = 3; __VA_ARGS__; } break;      \
    default: { constexpr int kNG = 4; __VA_ARGS__; } break;     \
  }

iha_status move(const char* name, bool store, const void* k, const void* v, const int32_t* slots,
                const void* cache, int B_outer, int B_inner, int N, int n_pages, int page, int Hkv,
                int d, iha_strides sk, iha_strides sv, iha_dtype dt, void* stream) {
  if (!k || !v || !slots || !cache) return fail(IHA_ERR_INVALID_ARG, "%s: null pointer", name);
  if (B_outer <= 0 || B_inner <= 0 || N <= 0)
    return fail(IHA_ERR_INVALID_ARG, "%s: sizes must be positive", name);
  if (dt != IHA_BF16 && dt != IHA_F32) return fail(IHA_ERR_INVALID_ARG, "%s: bad dtype", name);
  iha_status st = kv4_check_cache(name, cache, n_pages, page, Hkv, d);
  if (st != IHA_OK) return st;
  const int es = dt == IHA_BF16 ? 2 : 4;
  if (!aligned16(k) || !aligned16(v))
    return fail(IHA_ERR_ALIGNMENT, "%s: k and v must be 16-byte aligned", name);
  if (reinterpret_cast<uintptr_t>(slots) & 3)
    return fail(IHA_ERR_ALIGNMENT, "%s: slots must be 4-byte aligned", name);
  for (iha_strides* t : {&sk, &sv}) {  // the stride of an extent of 1 is never used
    if (B_outer == 1) t->b_outer = 0;
    if (B_inner == 1) t->b_inner = 0;
    if (N == 1) t->seq = 0;
    if (Hkv == 1) t->head = 0;
  }
  if (!strides_ok(sk, es) || !strides_ok(sv, es))
    return fail(IHA_ERR_ALIGNMENT, "%s: strides must be multiples of 16 bytes", name);
  const int64_t toks = (int64_t)B_outer * B_inner * N, rows = toks * Hkv;
  if (toks > INT32_MAX || rows > INT32_MAX)
    return fail(IHA_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 rows in one call", name);
  bool nk, nv;
  const int64_t bk = view_bytes(sk, B_outer, B_inner, N, Hkv, d, es, &nk);
  const int64_t bv = view_bytes(sv, B_outer, B_inner, N, Hkv, d, es, &nv);
  if (nk || nv) return fail(IHA_ERR_INVALID_ARG, "%s: negative stride", name);
  const int64_t bc = (int64_t)n_pages * kv4_page_bytes(page, Hkv, d);
  if (overlaps(cache, bc, k, bk) || overlaps(cache, bc, v, bv) ||
      overlaps(cache, bc, slots, toks * 4))
    return fail(IHA_ERR_INVALID_ARG, "%s: the cache overlaps another buffer", name);
  if (!store) {
    if (k == v || overlaps(k, bk, slots, toks * 4) || overlaps(v, bv, slots, toks * 4))
      return fail(IHA_ERR_INVALID_ARG, "%s: an output overlaps another tensor", name);
    for (const iha_strides* t : {&sk, &sv})
      if ((B_outer > 1 && t->b_outer == 0) || (B_inner > 1 && t->b_inner == 0) ||
          (N > 1 && t->seq == 0) || (Hkv > 1 && t->head == 0))
        return fail(IHA_ERR_INVALID_ARG, "%s: an output repeats rows (stride 0)", name);
  }
  Kv4Geom g;
  g.N = N;
  g.H = Hkv;
  g.page = page;
  g.blocks_per_page = page / kKv4Tok;
  g.n_slots = n_pages * page;
  g.rows = rows;
  g.Bi = B_inner;
  const int ng = d / kKv4Group;
  const int64_t blocks = (rows * 4 * ng + 255) / 256;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* c = static_cast<uint8_t*>(const_cast<void*>(cache));
  IHA_NG_SWITCH(ng, {
    if (store) {
      if (dt == IHA_BF16)
        kv4_store_kernel<__nv_bfloat16, kNG><<<(unsigned)blocks, 256, 0, s>>>(
            static_cast<const __nv_bfloat16*>(k), static_cast<const __nv_bfloat16*>(v), slots, c,
            g, sk, sv);
      else
        kv4_store_kernel<float, kNG><<<(unsigned)blocks, 256, 0, s>>>(
            static_cast<const float*>(k), static_cast<const float*>(v), slots, c, g, sk, sv);
    } else {
      if (dt == IHA_BF16)
        kv4_load_kernel<__nv_bfloat16, kNG><<<(unsigned)blocks, 256, 0, s>>>(
            c, slots, static_cast<__nv_bfloat16*>(const_cast<void*>(k)),
            static_cast<__nv_bfloat16*>(const_cast<void*>(v)), g, sk, sv);
      else
        kv4_load_kernel<float, kNG><<<(unsigned)blocks, 256, 0, s>>>(
            c, slots, static_cast<float*>(const_cast<void*>(k)),
            static_cast<float*>(const_cast<void*>(v)), g, sk, sv);
    }
  })
  return check_launch(name);
}

}  // namespace

iha_status kv4_check_cache(const char* name, const void* cache, int n_pages, int page, int Hkv,
                           int d) {
  if (n_pages <= 0 || page <= 0 || Hkv <= 0 || d <= 0)
    return fail(IHA_ERR_INVALID_ARG, "%s: sizes must be positive", name);
  if (d % kKv4Group || d > 128)
    return fail(IHA_ERR_UNSUPPORTED, "%s: needs d in {32, 64, 96, 128}, got %d", name, d);
  if (page % kKv4Tok)
    return fail(IHA_ERR_UNSUPPORTED, "%s: page size %d is not a multiple of %d", name, page,
                kKv4Tok);
  if ((int64_t)n_pages * page > INT32_MAX)
    return fail(IHA_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 slots", name);
  if (!aligned16(cache))
    return fail(IHA_ERR_ALIGNMENT, "%s: the cache must be 16-byte aligned", name);
  return IHA_OK;
}

}  // namespace iha

extern "C" {

size_t kv4_page_bytes(int page, int Hkv, int d) {
  if (page <= 0 || page % iha::kKv4Tok || Hkv <= 0 || d <= 0 || d % iha::kKv4Group || d > 128)
    return 0;
  return (size_t)(page / iha::kKv4Tok) * Hkv * iha::kv4_block_bytes(d / iha::kKv4Group);
}

iha_status kv4_store(const void* k, const void* v, const int32_t* slots, void* cache, int B_outer,
                     int B_inner, int N, int n_pages, int page, int Hkv, int d, iha_strides sk,
                     iha_strides sv, iha_dtype dt, void* stream) {
  return iha::move("kv4_store", true, k, v, slots, cache, B_outer, B_inner, N, n_pages, page, Hkv,
                   d, sk, sv, dt, stream);
}

iha_status kv4_load(const void* cache, const int32_t* slots, void* k, void* v, int B_outer,
                    int B_inner, int N, int n_pages, int page, int Hkv, int d, iha_strides sk,
                    iha_strides sv, iha_dtype dt, void* stream) {
  return iha::move("kv4_load", false, k, v, slots, cache, B_outer, B_inner, N, n_pages, page, Hkv,
                   d, sk, sv, dt, stream);
}

}  // extern "C"
