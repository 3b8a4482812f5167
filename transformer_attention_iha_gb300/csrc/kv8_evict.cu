// Eviction from the 8-bit cache by the attention weight that keys have gathered
// (kv8_evict; layout of the cache: kv8.cuh).
//
// Two launches.  Select, one or several CTAs per sequence and head: the weights as integers in their
// order (a float's bits, the negative ones turned round), held in shared memory, the
// smallest kept one found from counts of 11 bits at a time (a radix select; those that
// share its first digit are listed, and only they are looked at again), then the kept ones
// written in the order of their positions, 4096 keys at a time by a scan over the CTA.  Few
// heads of many keys have a cluster of CTAs each, that read one another's counts.
// Copy, a warp per block of 16 kept rows of a head: a lane finds where a row is, then the
// rows are gathered whole, 16 bytes a lane, and rounded again where their block's scale
// is not the largest of its sixteen.
//
// What bounds it: 32768 keys x 80 heads of 128 to 8192, 353 MB, replayed from a graph: 79 us
// (floor 53; launched one by one 83), select 25, copy 52 behind it.  Select: issue (0.64 a cycle, one CTA a head: 72 of 152 SMs idle),
// and three phases in lockstep (counts 6 us, list and its digits 6, order 8).  Copy: HBM, by
// rows of one line each.  Few rows: latency, 4 x 8 heads of 1100 keys 11 us.
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
  int B, H, n_pages, page, table_w, dest_w, keep, recent;
  Kv8Pages pages;
  int64_t cap, dest_cap;
  FastDiv blocks, heads;  // copy: blocks that a head can fill; heads
  int64_t items;
};

// Larger weights as larger numbers; NaN as the lowest, -0 as 0.
constexpr uint32_t kLowest = 0x007FFFFFu;  // of -inf, and of NaN
__device__ __forceinline__ float weight_of(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u);
}
__device__ __forceinline__ uint32_t order_of(float w) {
  if (w != w) w = -INFINITY;
  const uint32_t u = __float_as_uint(w + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kBins = 2048;        // three digits: 11, 11 and 10 bits
constexpr int kReplicas = 4;       // of the counts, by lane: neighbours count apart
constexpr int kReplica = kBins + 8;  // from one to the next, in other banks
constexpr int kList = 4096;        // keys that share the first digit of the smallest kept
constexpr int kCached = 40 * 1024;  // keys of a CTA whose numbers stay in shared memory
constexpr int kChunk = 4 * kThreads;
// counts, [2][kBins] counts of the whole CTA, the list; and 4 bytes a cached key
constexpr int kSelectSmem = (kReplicas * kReplica + 2 * kBins + kList) * 4;

__device__ __forceinline__ int cluster_rank() {
  int r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ int cluster_size() {
  int r;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;"
               ::: "memory");
}
// A word of shared memory, of the cluster's CTA `rank`.
__device__ __forceinline__ int load_of(int rank, const int* p) {
  uint32_t a = smem_u32(p);
  int v;
  asm volatile("mapa.shared::cluster.u32 %0, %0, %1;" : "+r"(a) : "r"(rank));
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}

// A cluster per sequence and head, each CTA a stretch of its keys.  VEC: weights on 16 bytes.
template <bool VEC>
__global__ void __launch_bounds__(kThreads, 1) kv8_select_kernel(const EvictParams p) {
  extern __shared__ uint4 smem[];
  int* const hist = reinterpret_cast<int*>(smem);
  int* const bins = hist + kReplicas * kReplica;
  uint32_t* const list = reinterpret_cast<uint32_t*>(bins + 2 * kBins);
  uint32_t* const held = list + kList;
  __shared__ int totals[2][kWarps];
  __shared__ int found[3];   // the digit, how many of it are kept, how many have it
  __shared__ int sums[3];    // this CTA's: above the digits so far, equal to all, listed
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int size = cluster_size(), rank = cluster_rank();
  const int plane = blockIdx.x / size, b = plane / p.H, h = plane - b * p.H;
  const int raw = __ldg(p.lens + b), n = min(max(raw, 0), (int)p.cap);
  const bool writer = rank == 0 && tid == 0 && h == 0;
  if (raw != n && writer) atomicOr(&g_dev_error, DEV_ERR_CACHE_INDEX);
  const int m = min(n, p.keep);
  if (writer) p.new_lens[b] = m;
  const float* w = p.weights + plane * p.cap;
  int32_t* kept = p.kept + (int64_t)plane * p.keep;
  float* out = p.weights_out ? p.weights_out + plane * p.dest_cap : nullptr;
  const int all_tid = rank * kThreads + tid, all_threads = size * kThreads;
  for (int i = m + all_tid; i < p.keep; i += all_threads) kept[i] = -1;
  if (out)
    for (int64_t i = m + all_tid; i < p.dest_cap; i += all_threads) out[i] = 0.f;
  // keys [0, older) compete for `need` places; this CTA has keys [first, end)
  const bool all = n <= p.keep;
  const int older = all ? 0 : n - p.recent;
  int need = all ? 0 : p.keep - p.recent;
  const int per = ((n + size - 1) / size + 127) & ~127;
  const int first = min(n, rank * per), end = min(n, first + per), mine = min(end, older);
  // kept: numbers above `low`, and the first `need` of those that equal it
  uint32_t low = ~0u;
  // four numbers from key j on, j a multiple of 4; what lies past `mine` means nothing
  auto numbers = [&](int j, uint32_t (&u)[4], bool fresh) {
    const bool cached = j + 4 - first <= kCached;
    if (!fresh && cached) {
      const uint4 v = *reinterpret_cast<const uint4*>(held + (j - first));
      u[0] = v.x, u[1] = v.y, u[2] = v.z, u[3] = v.w;
      return;
    }
    float x[4];
    if (VEC) {  // rows are whole pages, so the vector lies within them
      const float4 v = __ldg(reinterpret_cast<const float4*>(w + j));
      x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = __ldg(w + j + i);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) u[i] = order_of(x[i]);
    if (fresh && cached)
      *reinterpret_cast<uint4*>(held + (j - first)) = make_uint4(u[0], u[1], u[2], u[3]);
  };
  if (tid < 3) sums[tid] = 0;
  if (need > 0) {
    low = 0;
    bool has_list = false;
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const int up = pass == 1 ? 21 : 10;  // of the digits before
      const uint32_t mask = pass < 2 ? 2047u : 1023u;
      const int replicas = has_list ? 1 : kReplicas;
      for (int i = tid; i < replicas * kReplica; i += kThreads) hist[i] = 0;
      __syncthreads();
      int* const count = hist + (lane & (replicas - 1)) * kReplica;
      if (has_list) {
        const int listed = sums[2];
        for (int j = tid; j < listed; j += kThreads)
          if (list[j] >> up == low >> up) atomicAdd(&count[(list[j] >> shift) & mask], 1);
      } else {
#pragma unroll 4
        for (int j = first + 4 * tid; j < mine; j += kChunk) {
          uint32_t u[4];
          numbers(j, u, pass == 0);
          if (pass == 0 && j + 4 <= mine && (u[0] >> 21) == (u[1] >> 21) &&
              (u[0] >> 21) == (u[2] >> 21) && (u[0] >> 21) == (u[3] >> 21)) {
            atomicAdd(&count[u[0] >> 21], 4);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (j + i < mine && (pass == 0 || u[i] >> up == low >> up))
                atomicAdd(&count[(u[i] >> shift) & mask], 1);
          }
        }
      }
      __syncthreads();
      // this CTA's counts, then the cluster's, from the largest digit down
      constexpr int PER = kBins / kThreads;
      int c[PER], own[PER], sum = 0;
      int* const my_bins = bins + (pass & 1) * kBins;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int bin = kBins - 1 - (PER * tid + i);
        own[i] = 0;
        for (int k = 0; k < replicas; ++k) own[i] += hist[k * kReplica + bin];
        my_bins[bin] = own[i];
        c[i] = own[i];
      }
      if (size > 1) {
        cluster_sync();
        for (int k = 1; k < size; ++k)
#pragma unroll
          for (int i = 0; i < PER; ++i)
            c[i] += load_of((rank + k) & (size - 1), my_bins + kBins - 1 - (PER * tid + i));
      }
#pragma unroll
      for (int i = 0; i < PER; ++i) sum += c[i];
      int incl = sum;
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, k);
        if (lane >= k) incl += v;
      }
      if (lane == 31) totals[0][warp] = incl;
      __syncthreads();
      int before = incl - sum + __reduce_add_sync(0xffffffffu, lane < warp ? totals[0][lane] : 0);
      // the one at which `need` is reached
      if (before < need && before + sum >= need)
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
      const int digit = found[0], same = found[2];
      low |= (uint32_t)digit << shift;
      need = found[1];
      const bool whole = same == need;  // all that have the digits so far are kept
      int gt = 0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const int bin = kBins - 1 - (PER * tid + i);
        if (bin > digit || (whole && bin == digit)) gt += own[i];
        if (!whole && pass == 2 && bin == digit) sums[1] = own[i];
      }
      gt = __reduce_add_sync(0xffffffffu, gt);
      if (lane == 0 && gt != 0) atomicAdd(&sums[0], gt);
      if (whole) {  // (low is above 0: no number is below that of -inf)
        low -= 1;
        need = 0;
        break;
      }
      if (pass == 0 && same <= kList) {
        has_list = true;
        for (int j = first + 4 * tid; j < mine; j += kChunk) {
          uint32_t u[4];
          numbers(j, u, false);
          uint32_t hit = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) hit |= j + i < mine && u[i] >> 21 == low >> 21 ? 1u << i : 0u;
          if (hit == 0) continue;
          int to = atomicAdd(&sums[2], __popc(hit));
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if ((hit >> i) & 1u) list[to++] = u[i];
        }
        __syncthreads();
      }
    }
  }
  launch_dependents();  // the copy's CTAs may come; they wait for this grid's end
  // the kept ones in order: key j goes to (those above `low` before it) + (those equal to
  // it before it, of which the first `need` are kept)
  int above = max(0, first - older), equal = 0;  // before this CTA's keys
  if (size > 1) {
    cluster_sync();
    for (int k = 0; k < rank; ++k) {
      above += load_of(k, &sums[0]);
      equal += load_of(k, &sums[1]);
    }
  }
  for (int j0 = first, buf = 0; j0 < end; j0 += kChunk, buf ^= 1) {
    const int j = j0 + 4 * tid;
    uint32_t u[4] = {0, 0, 0, 0};
    if (j < mine) numbers(j, u, false);
    int kinds = 0;  // above in the low half, equal in the high
    uint32_t is_above = 0, is_equal = 0;
    const bool whole = j0 + kChunk <= mine;  // the same in the CTA
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool in = whole || j + i < mine;
      const bool a = in ? u[i] > low : j + i < end, q = in && u[i] == low;
      is_above |= a ? 1u << i : 0u;
      is_equal |= q ? 1u << i : 0u;
      kinds += (a ? 1 : 0) + (q ? 1 << 16 : 0);
    }
    int incl = kinds;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, incl, k);
      if (lane >= k) incl += v;
    }
    if (lane == 31) totals[buf][warp] = incl;
    __syncthreads();
    const int t = lane < kWarps ? totals[buf][lane] : 0;
    const int before = incl - kinds + __reduce_add_sync(0xffffffffu, lane < warp ? t : 0);
    const int chunk = __reduce_add_sync(0xffffffffu, t);
    int eq = equal + (before >> 16), to = above + (before & 0xFFFF) + min(eq, need);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const bool q = (is_equal >> i) & 1u;
      if (((is_above >> i) & 1u) || (q && eq < need)) {
        kept[to] = j + i;
        if (out) {
          const bool again = (!whole && j + i >= mine) || u[i] == kLowest;
          out[to] = again ? __ldg(w + j + i) : weight_of(u[i]);
        }
        ++to;
      }
      eq += q;
    }
    above += chunk & 0xFFFF;
    equal += chunk >> 16;
  }
  if (size > 1) cluster_sync();  // the others have read this CTA's sums
}

constexpr int kCopyWarps = 4;

template <int D>
__global__ void __launch_bounds__(32 * kCopyWarps) kv8_copy_kernel(const EvictParams p) {
  constexpr int LPR = D / 16, RPI = 32 / LPR, ITER = (kKv8Tok + RPI - 1) / RPI;
  const int lane = threadIdx.x & 31;
  const int64_t id64 = (int64_t)blockIdx.x * kCopyWarps + (threadIdx.x >> 5);
  if (id64 >= p.items) return;
  const int id = (int)id64, plane = p.blocks.div(id), blk = id - plane * p.blocks.d;
  const int b = p.heads.div(plane), head = plane - b * p.heads.d;
  const int n = min(max(__ldg(p.lens + b), 0), (int)p.cap), m = min(n, p.keep);
  const int rows = min(m - blk * kKv8Tok, kKv8Tok);
  wait_for_grid();
  if (rows <= 0) return;
  // (not through the read-only path: written while this grid was already there)
  const int j = lane < rows ? __ldcg(p.kept + (int64_t)plane * p.keep + blk * kKv8Tok + lane) : 0;
  const int bpp = p.pages.bpp, dpi = blk / bpp;
  const int dest_page = __ldg(p.dest + (int64_t)b * p.dest_w + dpi);
  if (dest_page < 0 || dest_page >= p.n_pages) {
    if (lane == 0) atomicOr(&g_dev_error, DEV_ERR_CACHE_INDEX);
    return;
  }
  uint8_t* const to = p.cache + p.pages.block(dest_page, head, blk - dpi * bpp, D);
  // lane i < 16: where row i comes from
  int64_t from = -1;
  int row = 0;
  Kv8Tail tail = {{0.f, 0.f}, 0u, 0u};
  if (lane < rows) {
    const int pi = j / p.page, off = j - pi * p.page;
    const int pg = __ldg(p.table + (int64_t)b * p.table_w + pi);
    row = off % kKv8Tok;
    if (pg >= 0 && pg < p.n_pages) {
      from = p.pages.block(pg, head, off / kKv8Tok, D);
      tail = kv8_tail(p.cache + p.pages.tail(pg, head, off / kKv8Tok));
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
    *reinterpret_cast<uint4*>(p.cache + p.pages.tail(dest_page, head, blk - dpi * bpp)) =
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
  if (keep > (1 << 30))  // (places of the list are counted in 32 bits)
    return fail(IHA_ERR_UNSUPPORTED, "%s: keep %d is more than 2^30", name, keep);
  const int64_t most = keep < cap ? keep : cap;  // keys that a head can have afterwards
  if (dest_cap < most)
    return fail(IHA_ERR_INVALID_ARG, "%s: dest_table holds %lld tokens, keep is %d", name,
                (long long)dest_cap, keep);
  if ((reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(seq_lens) |
       reinterpret_cast<uintptr_t>(weights) | reinterpret_cast<uintptr_t>(dest_table) |
       reinterpret_cast<uintptr_t>(new_lens) | reinterpret_cast<uintptr_t>(kept) |
       reinterpret_cast<uintptr_t>(weights_out)) & 3)
    return fail(IHA_ERR_ALIGNMENT, "%s: tables, lengths, ids and weights must be 4-byte aligned",
                name);
  const int64_t planes = (int64_t)B * Hkv, blocks = (most + kKv8Tok - 1) / kKv8Tok;
  if (planes > (1 << 26) || planes * blocks > INT32_MAX)
    return fail(IHA_ERR_UNSUPPORTED, "%s: more than 2^26 heads or 2^31 - 1 blocks in one call",
                name);
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
  p.pages.set(page, Hkv, d);
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
  static SmemLimit limit[2];
  const bool vec = aligned16(weights);
  auto* const select = vec ? kv8_select_kernel<true> : kv8_select_kernel<false>;
  const cudaError_t e = limit[vec].ensure(select, kSelectSmem + kCached * 4);
  if (e != cudaSuccess)
    return fail(IHA_ERR_CUDA, "%s (smem attribute): %s", name, cudaGetErrorString(e));
  // CTAs of a head: as many as the GPU runs at once (one on an SM), while each has 4096
  // keys or more
  unsigned size = 1;
  while (size < 8 && planes * size * 2 <= (int64_t)sm_count() && cap >= 4096 * 2 * size) size *= 2;
  int64_t held = ((cap + size - 1) / size + 127) & ~(int64_t)127;
  if (held > kCached) held = kCached;
  if (planes * size > INT32_MAX)
    return fail(IHA_ERR_UNSUPPORTED, "%s: too many heads in one call", name);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = size;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)planes * size);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSelectSmem + held * 4;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t le = cudaLaunchKernelEx(&cfg, select, p);
  if (le != cudaSuccess) return fail(IHA_ERR_CUDA, "%s: %s", name, cudaGetErrorString(le));
  st = check_launch(name);
  if (st != IHA_OK) return st;
  const unsigned grid = (unsigned)((p.items + kCopyWarps - 1) / kCopyWarps);
  IHA_KV8_D_SWITCH(d, return launch_behind(name, kv8_copy_kernel<kD>, grid, 32 * kCopyWarps, s, p))
  return IHA_OK;
}

}  // extern "C"
