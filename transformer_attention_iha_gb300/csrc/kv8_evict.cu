// Eviction from the 8-bit cache by the attention weight that keys have gathered
// (kv8_evict; layout of the cache: kv8.cuh).
//
// Two launches.  Select, a CTA per sequence and head: the weights as integers in their
// order (a float's bits, the negative ones turned round), held in shared memory, the
// smallest kept one found from counts of 11 bits at a time (a radix select), then the
// kept ones in the order of their positions: each warp counts its stretch of keys, the
// counts are summed over the warps, each warp writes its own.  Copy, a warp per block of 16 kept rows of a head: rows are
// gathered whole, 16 bytes a lane, rounded again where their block's scale is not
// the largest of the sixteen.
#include "kv8.cuh"

namespace iha {
namespace {

IHA_DEVICE_ERROR_WORD(kv8_evict)

constexpr int kWarps = 32;
constexpr int kThreads = 32 * kWarps;

struct EvictParams {
  uint8_t* cache;
  const int32_t *table, *lens, *dest;
  const float* weights;
  int32_t *new_lens, *kept;
  float* weights_out;  // nullable
  int B, H, n_pages, page, bpp, table_w, dest_w, keep, recent;
  int64_t cap, dest_cap;
  FastDiv blocks, heads;  // copy: blocks of keep rows; heads
  int64_t items;
};

// Larger weights as larger numbers; NaN as the lowest, -0 as 0.
__device__ __forceinline__ uint32_t order_of(float w) {
  if (w != w) w = -INFINITY;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kDigit = 11, kBins = 1 << kDigit;  // three digits: 11, 11 and 10 bits
constexpr int kCached = 48 * 1024;  // keys whose numbers stay in shared memory

__global__ void __launch_bounds__(kThreads, 1) kv8_select_kernel(const EvictParams p) {
  extern __shared__ uint32_t held[];
  __shared__ int hist[kBins];
  __shared__ int count[2][kWarps];
  __shared__ int found[3];  // the digit, how many of it are kept, how many have it
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int plane = blockIdx.x, b = plane / p.H, h = plane - b * p.H;
  const int raw = __ldg(p.lens + b), n = min(max(raw, 0), (int)p.cap);
  if (raw != n && h == 0 && tid == 0) atomicOr(&g_dev_error, DEV_ERR_CACHE_INDEX);
  const int m = min(n, p.keep);
  if (h == 0 && tid == 0) p.new_lens[b] = m;
  const float* w = p.weights + plane * p.cap;
  int32_t* kept = p.kept + (int64_t)plane * p.keep;
  float* out = p.weights_out ? p.weights_out + plane * p.dest_cap : nullptr;
  for (int i = m + tid; i < p.keep; i += kThreads) kept[i] = -1;
  if (out)
    for (int64_t i = m + tid; i < p.dest_cap; i += kThreads) out[i] = 0.f;
  const int older = n > p.keep ? n - p.recent : 0;  // keys [0, older) compete
  int need = n > p.keep ? p.keep - p.recent : 0;
  uint32_t low = 0;  // the smallest kept weight, in order_of's numbers
  auto number = [&](int j) { return j < kCached ? held[j] : order_of(__ldg(w + j)); };
  if (need > 0) {
    for (int j = tid; j < min(older, kCached); j += kThreads) held[j] = order_of(__ldg(w + j));
#pragma unroll 1
    for (int shift = 32 - kDigit; ; shift = max(0, shift - kDigit)) {
      const int upto = shift == 32 - kDigit ? 32 : shift == 0 ? 32 - 2 * kDigit : shift + kDigit;
      const uint32_t mask = (1u << (upto - shift)) - 1u;
      for (int i = tid; i < kBins; i += kThreads) hist[i] = 0;
      __syncthreads();
      for (int j0 = warp * 32; j0 < older; j0 += kThreads) {
        const int j = j0 + lane;
        const uint32_t u = j < older ? number(j) : 0u;
        const bool in = j < older && (upto == 32 || (u >> upto) == (low >> upto));
        const uint32_t who = __ballot_sync(0xffffffffu, in);
        if (who == 0) continue;
        const int digit = (int)((u >> shift) & mask);
        // equal weights (zeros, most often) would add to one counter 32 times
        const int first = __shfl_sync(0xffffffffu, digit, __ffs(who) - 1);
        if (__all_sync(0xffffffffu, !in || digit == first)) {
          if (lane == 0) atomicAdd(&hist[first], __popc(who));
        } else if (in) {
          atomicAdd(&hist[digit], 1);
        }
      }
      __syncthreads();
      // from the largest digit down: the one at which `need` is reached
      constexpr int PER = kBins / kThreads;
      int c[PER], sum = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) sum += c[i] = hist[kBins - 1 - (PER * tid + i)];
      int incl = sum;
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, k);
        if (lane >= k) incl += v;
      }
      if (lane == 31) count[0][warp] = incl;
      __syncthreads();
      for (int k = 0; k < warp; ++k) incl += count[0][k];
      int before = incl - sum;
      if (before < need && incl >= need)
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          if (before < need && before + c[i] >= need) {
            found[0] = kBins - 1 - (PER * tid + i);
            found[1] = need - before;
            found[2] = c[i];
          }
          before += c[i];
        }
      __syncthreads();
      low |= (uint32_t)found[0] << shift;
      need = found[1];  // of those equal so far
      if (shift == 0 || found[2] == need) break;  // all that have the digits so far are kept
    }
    __syncthreads();
  }
  // each warp's stretch of keys: how many are above `low`, how many equal it
  const bool all = n <= p.keep;
  const int per = ((n + kWarps - 1) / kWarps + 31) & ~31;
  const int j0 = min(n, warp * per), j1 = min(n, j0 + per);
  int above = 0, equal = 0;
  for (int j = j0 + lane; j < j1; j += 32) {
    if (all || j >= older) {
      ++above;
    } else if (p.keep > p.recent) {
      const uint32_t u = number(j);
      above += u > low;
      equal += u == low;
    }
  }
  above = __reduce_add_sync(0xffffffffu, above);
  equal = __reduce_add_sync(0xffffffffu, equal);
  if (lane == 0) {
    count[0][warp] = above;
    count[1][warp] = equal;
  }
  __syncthreads();
  int at = 0, eq = 0;  // kept ones, equal ones before this warp's
  for (int k = 0; k < warp; ++k) {
    at += count[0][k];
    eq += count[1][k];
  }
  at += min(eq, need);
  const uint32_t below = (1u << lane) - 1u;
  for (int j = j0; j < j1; j += 32) {
    const int i = j + lane;
    const bool in = i < j1;
    bool is_above = in && (all || i >= older), is_equal = false;
    if (in && !is_above && p.keep > p.recent) {
      const uint32_t u = number(i);
      is_above = u > low;
      is_equal = u == low;
    }
    const uint32_t me = __ballot_sync(0xffffffffu, is_equal);
    const bool take = is_above || (is_equal && eq + __popc(me & below) < need);
    const uint32_t mt = __ballot_sync(0xffffffffu, take);
    if (take) {
      const int to = at + __popc(mt & below);
      kept[to] = i;
      if (out) out[to] = __ldg(w + i);
    }
    at += __popc(mt);
    eq += __popc(me);
  }
}

template <int D>
__global__ void __launch_bounds__(256) kv8_copy_kernel(const EvictParams p) {
  constexpr int LPR = D / 16, RPI = 32 / LPR, ITER = (kKv8Tok + RPI - 1) / RPI;
  const int lane = threadIdx.x & 31;
  const int64_t id64 = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (id64 >= p.items) return;
  const int id = (int)id64, plane = p.blocks.div(id), blk = id - plane * p.blocks.d;
  const int b = p.heads.div(plane), head = plane - b * p.heads.d;
  const int n = min(max(__ldg(p.lens + b), 0), (int)p.cap), m = min(n, p.keep);
  const int rows = min(m - blk * kKv8Tok, kKv8Tok);
  if (rows <= 0) return;
  const int dpi = blk / p.bpp, dest_page = __ldg(p.dest + (int64_t)b * p.dest_w + dpi);
  if (dest_page < 0 || dest_page >= p.n_pages) {
    if (lane == 0) atomicOr(&g_dev_error, DEV_ERR_CACHE_INDEX);
    return;
  }
  uint8_t* const to =
      p.cache + kv8_block_of(dest_page, blk - dpi * p.bpp, head, p.heads.d, p.bpp, D);
  // lane i < 16: where row i comes from
  int64_t from = -1;
  int row = 0;
  Kv8Tail tail = {{0.f, 0.f}, 0u, 0u};
  if (lane < rows) {
    const int j = __ldg(p.kept + (int64_t)plane * p.keep + blk * kKv8Tok + lane);
    const int pi = j / p.page, off = j - pi * p.page;
    const int pg = __ldg(p.table + (int64_t)b * p.table_w + pi);
    row = off % kKv8Tok;
    if (pg >= 0 && pg < p.n_pages) {
      from = kv8_block_of(pg, off / kKv8Tok, head, p.heads.d, p.bpp, D);
      tail = kv8_tail(p.cache + from, D);
    } else {
      atomicOr(&g_dev_error, DEV_ERR_CACHE_INDEX);
    }
  }
  const int ek = from >= 0 ? kv8_exponent(tail.scale[0]) : kKv8LowestE;
  const int ev = from >= 0 ? kv8_exponent(tail.scale[1]) : kKv8LowestE;
  const int tk = __reduce_max_sync(0xffffffffu, ek), tv = __reduce_max_sync(0xffffffffu, ev);
  const uint32_t nan_k = __ballot_sync(0xffffffffu, (tail.nan >> row) & 1u);
  const uint32_t nan_v = __ballot_sync(0xffffffffu, (tail.nan >> (16 + row)) & 1u);
  const int r = lane / LPR, c = lane - r * LPR;
  uint4 k[ITER], v[ITER];
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int tok = i * RPI + r;
    const int64_t f = __shfl_sync(0xffffffffu, from, tok & 15);
    const int fr = __shfl_sync(0xffffffffu, row, tok & 15);
    k[i] = v[i] = make_uint4(0, 0, 0, 0);
    if (r < RPI && tok < rows && f >= 0) {
      const uint8_t* at = p.cache + f + fr * D + ((c ^ kv8_swap(D, fr)) << 4);
      k[i] = *reinterpret_cast<const uint4*>(at);
      v[i] = *reinterpret_cast<const uint4*>(at + kKv8Tok * D);
    }
  }
#pragma unroll
  for (int i = 0; i < ITER; ++i) {
    const int tok = i * RPI + r;
    const int sk = __shfl_sync(0xffffffffu, ek, tok & 15) - tk;
    const int sv = __shfl_sync(0xffffffffu, ev, tok & 15) - tv;
    if (r < RPI && tok < kKv8Tok) {
      if (sk < 0) {
        const float f = kv8_two(sk);
        k[i] = make_uint4(e4m3_rescale(k[i].x, f), e4m3_rescale(k[i].y, f),
                          e4m3_rescale(k[i].z, f), e4m3_rescale(k[i].w, f));
      }
      if (sv < 0) {
        const float f = kv8_two(sv);
        v[i] = make_uint4(e4m3_rescale(v[i].x, f), e4m3_rescale(v[i].y, f),
                          e4m3_rescale(v[i].z, f), e4m3_rescale(v[i].w, f));
      }
      uint8_t* at = to + tok * D + ((c ^ kv8_swap(D, tok)) << 4);
      *reinterpret_cast<uint4*>(at) = k[i];
      *reinterpret_cast<uint4*>(at + kKv8Tok * D) = v[i];
    }
  }
  if (lane == 0)
    *reinterpret_cast<uint4*>(to + 32 * D) =
        make_uint4(__float_as_uint(kv8_two(tk)), __float_as_uint(kv8_two(tv)),
                   (nan_k & 0xFFFFu) | (nan_v << 16), 0u);
}

}  // namespace
}  // namespace iha

extern "C" {

iha_status kv8_evict(void* cache, const int32_t* block_table, const int32_t* seq_lens,
                     const float* weights, const int32_t* dest_table, int32_t* new_lens,
                     int32_t* kept, float* weights_out, int B, int n_pages, int page,
                     int table_width, int dest_width, int Hkv, int d, int keep, int recent,
                     void* stream) {
  using namespace iha;
  const char* name = "kv8_evict";
  if (!cache || !block_table || !seq_lens || !weights || !dest_table || !new_lens || !kept)
    return fail(IHA_ERR_INVALID_ARG, "%s: null pointer", name);
  if (B <= 0 || table_width <= 0 || dest_width <= 0 || keep <= 0)
    return fail(IHA_ERR_INVALID_ARG, "%s: sizes must be positive", name);
  if (recent < 0 || recent > keep)
    return fail(IHA_ERR_INVALID_ARG, "%s: recent %d is not within [0, keep = %d]", name, recent,
                keep);
  iha_status st = kv8_check_cache(name, cache, n_pages, page, Hkv, d);
  if (st != IHA_OK) return st;
  const int64_t cap = (int64_t)table_width * page, dest_cap = (int64_t)dest_width * page;
  if (cap > (1 << 30) || dest_cap > (1 << 30))
    return fail(IHA_ERR_UNSUPPORTED, "%s: block table longer than 2^30 tokens", name);
  if (dest_cap < (keep < cap ? keep : cap))
    return fail(IHA_ERR_INVALID_ARG, "%s: dest_table holds %lld tokens, keep is %d", name,
                (long long)dest_cap, keep);
  if ((reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(seq_lens) |
       reinterpret_cast<uintptr_t>(weights) | reinterpret_cast<uintptr_t>(dest_table) |
       reinterpret_cast<uintptr_t>(new_lens) | reinterpret_cast<uintptr_t>(kept) |
       reinterpret_cast<uintptr_t>(weights_out)) & 3)
    return fail(IHA_ERR_ALIGNMENT, "%s: tables, lengths, ids and weights must be 4-byte aligned",
                name);
  const int64_t planes = (int64_t)B * Hkv, blocks = ((int64_t)keep + kKv8Tok - 1) / kKv8Tok;
  if (planes * blocks > INT32_MAX)
    return fail(IHA_ERR_UNSUPPORTED, "%s: more than 2^31 - 1 blocks in one call", name);
  struct Span {
    const void* p;
    int64_t n;
  };
  const Span out[] = {{cache, (int64_t)n_pages * (int64_t)kv8_page_bytes(page, Hkv, d)},
                      {new_lens, (int64_t)B * 4},
                      {kept, planes * keep * 4},
                      {weights_out, weights_out ? planes * dest_cap * 4 : 0}};
  const Span in[] = {{block_table, (int64_t)B * table_width * 4},
                     {seq_lens, (int64_t)B * 4},
                     {weights, planes * cap * 4},
                     {dest_table, (int64_t)B * dest_width * 4}};
  for (int i = 0; i < 4; ++i) {
    if (!out[i].p) continue;
    for (int j = 0; j < 4; ++j)
      if (overlaps(out[i].p, out[i].n, in[j].p, in[j].n) ||
          (j < i && overlaps(out[i].p, out[i].n, out[j].p, out[j].n)))
        return fail(IHA_ERR_INVALID_ARG, "%s: an output overlaps another tensor", name);
  }
  EvictParams p;
  p.cache = static_cast<uint8_t*>(cache);
  p.table = block_table;
  p.lens = seq_lens;
  p.dest = dest_table;
  p.weights = weights;
  p.new_lens = new_lens;
  p.kept = kept;
  p.weights_out = weights_out;
  p.B = B;
  p.H = Hkv;
  p.n_pages = n_pages;
  p.page = page;
  p.bpp = page / kKv8Tok;
  p.table_w = table_width;
  p.dest_w = dest_width;
  p.keep = keep;
  p.recent = recent;
  p.cap = cap;
  p.dest_cap = dest_cap;
  p.blocks.set((int)blocks);
  p.heads.set(Hkv);
  p.items = planes * blocks;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  static SmemLimit limit;
  const cudaError_t e = limit.ensure(kv8_select_kernel, kCached * 4);
  if (e != cudaSuccess)
    return fail(IHA_ERR_CUDA, "%s (smem attribute): %s", name, cudaGetErrorString(e));
  const int held = (int)(cap < kCached ? cap : kCached) * 4;
  kv8_select_kernel<<<(unsigned)planes, kThreads, held, s>>>(p);
  st = check_launch(name);
  if (st != IHA_OK) return st;
  const unsigned grid = (unsigned)((p.items + 7) / 8);
  IHA_KV8_D_SWITCH(d, (kv8_copy_kernel<kD><<<grid, 256, 0, s>>>(p)))
  return check_launch(name);
}

}  // extern "C"
