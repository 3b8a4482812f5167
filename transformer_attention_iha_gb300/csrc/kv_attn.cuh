// What the attentions over a paged cache share (4 and 8 bits): the line of work and its
// stretches, the rows that a column sees, parts of results and how they are joined, the
// matrix instructions on fp16, the host's checks.
//
// Work is one line of positions: sequence by sequence, head by head, column block by
// column block (a unit); a unit takes one position per block of 16 tokens it sees and
// kUnitCost for what a unit costs by itself.  Every warp of the grid takes an equal
// contiguous stretch of the line, so a long sequence, a ragged batch and many short ones
// all fill the GPU.  A unit that spans warps is joined from their parts (m, l, O in fp32)
// in an order that follows from the lengths and the grid.
#pragma once

#include <math.h>

#include "kv4.cuh"

namespace iha {
namespace {

IHA_DEVICE_ERROR_WORD(kv_attn)  // one for each file that includes this

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kKvTok = 16;  // tokens of a block
static_assert(kKvTok == kKv4Tok, "blocks of the caches");
// Positions a unit takes besides its blocks: its Q, output and ramp (each cache's kernel
// says what it measured).
constexpr int kUnitCost = IHA_KV_UNIT_COST;
// A warp's stretch is at least this long: shorter ones cost more in joining
// than they save (777 keys x 80 heads: 3 12.0 us, 4 11.6, 6 12.8).
constexpr int kMinShare = 4;
constexpr int kMaxCtas = 480;  // counters for 152 SMs x 3 CTAs and some
// The word behind the counters: not 0 once a wait has given up (written for 8 bits).  With it
// they end on a line.
constexpr int kGaveUp = kMaxCtas;
constexpr int kCounterBytes = 2048;
static_assert((kGaveUp + 1) * 4 <= kCounterBytes, "the workspace's first words");
// Parts a CTA may leave in the workspace: of the unit it begins in and the one it
// ends in; and of the unit each of its warps begins in, for the CTA itself.
constexpr int kCtaParts = 2 + kWarps;

struct KvAttnParams {
  const __nv_bfloat16* q;
  const uint8_t* cache;
  const int32_t* table;
  const int32_t* lens;
  __nv_bfloat16* o;
  float* lse;
  unsigned* counters;  // [kMaxCtas] and the word kGaveUp, zero between calls
  float* parts;        // [CTAs][kCtaParts][part_stride]
  int part_cols, part_stride;
  int B, Nq, Hq, Hkv, G, ncols, ncb;  // ncols = Nq * G columns of a key-value head, in ncb blocks
  unsigned long long inv_g;           // ceil(2^32 / G): col / G = col * inv_g >> 32
  int n_pages, page, blocks_per_page, table_w;
  int mask, window;
  float scale_log2;
  iha_strides sq, so;
  uint64_t wait_ns;
  int withhold;  // failure-path test: the first stage of CTA 0's warps never completes
  __device__ __forceinline__ void write_row(int64_t row, float ref, float l, float inv) const;
};

// d = a b + c on fp16 or bf16 operands, fp32 accumulators.
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1,
                                        const float (&c)[4]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]),
        "f"(c[3]));
}
__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ int token_of(const KvAttnParams& p, int col) {
  return (int)((unsigned long long)(unsigned)col * p.inv_g >> 32);
}

// A row's lse (natural logarithm) from its reference and sum.
__device__ __forceinline__ float lse_of(float ref, float l) {
  return l == 0.f ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
}
__device__ __forceinline__ void KvAttnParams::write_row(int64_t row, float ref, float l,
                                                        float) const {
  if (lse) lse[row] = lse_of(ref, l);
}
// Features of one output row, O / l; with the first ones what is written of the row besides.
template <typename P>
__device__ __forceinline__ void write_out(const P& p, int b, int hk, int col, int f, float4 o,
                                          float ref, float l) {
  const int qi = token_of(p, col), qh = hk * p.G + (col - qi * p.G);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint2 u;
  u.x = pack_bf16x2(o.x * inv, o.y * inv);
  u.y = pack_bf16x2(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>(p.o + b * p.so.b_outer + qi * p.so.seq + qh * p.so.head + f) = u;
  if (f == 0) p.write_row(((int64_t)b * p.Hq + qh) * p.Nq + qi, ref, l, inv);
}
template <typename P>
__device__ __forceinline__ void write_out(const P& p, int b, int hk, int col, int f, float2 o,
                                          float ref, float l) {
  const int qi = token_of(p, col), qh = hk * p.G + (col - qi * p.G);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  *reinterpret_cast<uint32_t*>(p.o + b * p.so.b_outer + qi * p.so.seq + qh * p.so.head + f) =
      pack_bf16x2(o.x * inv, o.y * inv);
  if (f == 0) p.write_row(((int64_t)b * p.Hq + qh) * p.Nq + qi, ref, l, inv);
}

// Visible keys [lo, hi) of column col of a sequence of len keys.
__device__ __forceinline__ void col_range(const KvAttnParams& p, int len, int col, int& lo,
                                          int& hi) {
  const int i = len - p.Nq + token_of(p, col);  // position of the new token
  hi = p.mask == IHA_MASK_NONE ? len : min(len, i + 1);
  lo = p.mask == IHA_MASK_CAUSAL_WINDOW && i >= p.window ? i - p.window + 1 : 0;
}

// First block and number of blocks that column block cb (COLS columns) sees.
template <int COLS>
__device__ __forceinline__ void unit_blocks(const KvAttnParams& p, int len, int cb, int& b0,
                                            int& n) {
  int lo, hi, x;
  col_range(p, len, cb * COLS, lo, x);
  col_range(p, len, min(p.ncols, cb * COLS + COLS) - 1, x, hi);
  b0 = lo / kKvTok;
  n = max(0, (hi + kKvTok - 1) / kKvTok - b0);
}

__device__ __forceinline__ int seq_len(const KvAttnParams& p, int b) {
  return min(max(__ldg(p.lens + b), 0), p.table_w * p.page);
}

// Positions of one head of a sequence over its column blocks.
template <int COLS>
__device__ __forceinline__ int head_positions(const KvAttnParams& p, int len) {
  int sum = p.ncb * kUnitCost;
  for (int cb = 0; cb < p.ncb; ++cb) {
    int b0, n;
    unit_blocks<COLS>(p, len, cb, b0, n);
    sum += n;
  }
  return sum;
}

// A unit of the line, and a warp's share of it.
struct Unit {
  int b, hk, cb, len, b0, n;
  int at;  // the unit's first position, from the start of the warp's stretch
};
// Blocks [r0, r1) of the unit that positions [0, stretch) hold.
__device__ __forceinline__ void my_blocks(const Unit& u, int stretch, int& r0, int& r1) {
  r0 = max(0, -u.at - kUnitCost);
  r1 = min(u.n, stretch - u.at - kUnitCost);
}
// The unit after u; false behind the last sequence.
template <int COLS>
__device__ __forceinline__ bool next_unit(const KvAttnParams& p, Unit& u) {
  u.at += u.n + kUnitCost;
  if (++u.cb == p.ncb) {
    u.cb = 0;
    if (++u.hk == p.Hkv) {
      u.hk = 0;
      if (++u.b == p.B) return false;
      u.len = seq_len(p, u.b);
    }
  }
  unit_blocks<COLS>(p, u.len, u.cb, u.b0, u.n);
  return true;
}

// Running join of softmax parts.
struct Joined {
  float m, l;
  float4 o;
  __device__ __forceinline__ void clear() {
    m = -INFINITY;
    l = 0.f;
    o = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  __device__ __forceinline__ void add(float pm, float pl, float4 po) {
    const float n = fmaxf(m, pm), ref = n == -INFINITY ? 0.f : n;
    const float a = exp2f(m - ref), c = exp2f(pm - ref);
    m = n;
    l = fmaf(l, a, pl * c);
    o.x = fmaf(o.x, a, po.x * c);
    o.y = fmaf(o.y, a, po.y * c);
    o.z = fmaf(o.z, a, po.z * c);
    o.w = fmaf(o.w, a, po.w * c);
  }
  // U parts at once: one rescale for all of them.
  template <int U>
  __device__ __forceinline__ void add(const float (&pm)[U], const float (&pl)[U],
                                      const float4 (&po)[U]) {
    float n = m;
#pragma unroll
    for (int k = 0; k < U; ++k) n = fmaxf(n, pm[k]);
    const float ref = n == -INFINITY ? 0.f : n, a = exp2f(m - ref);
    m = n;
    l *= a;
    o = make_float4(o.x * a, o.y * a, o.z * a, o.w * a);
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const float c = exp2f(pm[k] - ref);
      l = fmaf(pl[k], c, l);
      o.x = fmaf(po[k].x, c, o.x);
      o.y = fmaf(po[k].y, c, o.y);
      o.z = fmaf(po[k].z, c, o.z);
      o.w = fmaf(po[k].w, c, o.w);
    }
  }
  template <typename P>
  __device__ __forceinline__ void write(const P& p, const int* span, int col, int f) const {
    write_out(p, span[0], span[1], col, f, o, m == -INFINITY ? 0.f : m, l);
  }
};

// Joins the parts that CTAs of[0] .. of[1] left of a unit (all threads of the CTA).
template <int D, int COLS, typename P>
__device__ __forceinline__ void join_ctas(const P& p, const int* span, const int* of,
                                          float* scratch) {
  const int c_first = span[2] * COLS, first = of[0], last = of[1];
  const int ncolv = min(COLS, p.ncols - c_first), items = ncolv * (D / 4);
  // few items: several threads share one, each taking every groups-th part
  const int groups = items >= kThreads ? 1 : kThreads / items;
  const int tid = threadIdx.x;
  for (int i0 = 0; i0 < items; i0 += kThreads) {
    const int grp = groups > 1 ? tid / items : 0, i = groups > 1 ? tid - grp * items : i0 + tid;
    const bool mine = i < items && grp < groups;
    const int cc = mine ? i / (D / 4) : 0, f = mine ? (i - cc * (D / 4)) * 4 : 0;
    Joined a;
    a.clear();
    if (mine) {
      constexpr int U = 8;  // parts read at once: the join waits for memory, not for bandwidth
      for (int c0 = first + grp; c0 <= last; c0 += U * groups) {
        float pm[U], pl[U];
        float4 po[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int c = c0 + k * groups;
          pm[k] = -INFINITY;
          pl[k] = 0.f;
          po[k] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (c <= last) {
            const float* pp =
                p.parts + ((int64_t)c * kCtaParts + (c == first ? 1 : 0)) * p.part_stride;
            pm[k] = __ldcg(pp + p.part_cols * D + cc);
            pl[k] = __ldcg(pp + p.part_cols * D + p.part_cols + cc);
            po[k] = __ldcg(reinterpret_cast<const float4*>(pp + cc * D + f));
          }
        }
        a.add(pm, pl, po);
      }
    }
    if (groups > 1) {
      float* s = scratch + tid * 6;
      s[0] = a.m;
      s[1] = a.l;
      s[2] = a.o.x;
      s[3] = a.o.y;
      s[4] = a.o.z;
      s[5] = a.o.w;
      __syncthreads();
      if (grp == 0)
        for (int k = 1; k < groups; ++k) {
          const float* t = scratch + (tid + k * items) * 6;
          a.add(t[0], t[1], make_float4(t[2], t[3], t[4], t[5]));
        }
      __syncthreads();
    }
    if (mine && grp == 0) a.write(p, span, c_first + cc, f);
  }
}

// One more arrival at a unit's counter; releases what the CTA wrote before its
// last barrier, and acquires what the CTAs that arrived earlier wrote.
__device__ __forceinline__ unsigned arrive(unsigned* counter) {
  unsigned old;
  asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(old) : "l"(counter) : "memory");
  return old;
}


// CTAs an SM holds at once (registers and shared memory allow that many).
__host__ __device__ constexpr int ctas_per_sm(int nt) { return nt == 1 ? 3 : 2; }

// Column blocks of 8 or 16: a pass of 16 columns unpacks each code once for both
// halves.  (4 bits, 8 sequences of 16384 keys, 8 key heads of 128: 16 columns 70 us
// against 81 in two passes of 8; 32 columns 116, against 141 in passes of 8 and 138 in
// one of 32, whose accumulators leave too few warps and spill.)
inline int pick_nt(int64_t ncols) { return ncols <= 8 ? 1 : 2; }
inline int part_cols(int64_t ncols) {
  const int64_t cols = 8 * pick_nt(ncols);
  return (int)((ncols < cols ? ncols : cols) + 1) & ~1;  // even: rows of floats stay 16-byte
}
inline int part_stride(int64_t ncols, int d) {  // floats: O, then m, then l
  return (part_cols(ncols) * (d + 2) + 3) & ~3;
}

// Checks an attention call's arguments on the host and fills in what the kernels take
// of them: all but the wait limit.  check_cache, page_bytes and need are the cache's;
// nt: column blocks of 8 nt; grid: CTAs.
iha_status kv_attn_setup(const char* name, KvAttnParams& p, int& nt, int& grid,
                         iha_status (*check_cache)(const char*, const void*, int, int, int, int),
                         size_t page_bytes, size_t need, const void* q, const void* cache,
                         const int32_t* block_table, const int32_t* seq_lens, void* o,
                         float* lse_out, void* workspace, size_t workspace_bytes, int B, int Nq,
                         int Hq, int Hkv, int d, int n_pages, int page, int table_width,
                         iha_strides sq, iha_strides so, float scale, iha_mask mask_mode,
                         int window, iha_dtype dt) {
  if (!q || !cache || !block_table || !seq_lens || !o || !workspace)
    return fail(IHA_ERR_INVALID_ARG, "%s: null pointer", name);
  if (B <= 0 || Nq <= 0 || Hq <= 0 || table_width <= 0)
    return fail(IHA_ERR_INVALID_ARG, "%s: sizes must be positive", name);
  if (dt != IHA_BF16 && dt != IHA_F32) return fail(IHA_ERR_INVALID_ARG, "%s: bad dtype", name);
  if (mask_mode != IHA_MASK_NONE && mask_mode != IHA_MASK_CAUSAL &&
      mask_mode != IHA_MASK_CAUSAL_WINDOW)
    return fail(IHA_ERR_INVALID_ARG, "%s: bad mask_mode %d", name, (int)mask_mode);
  if (mask_mode == IHA_MASK_CAUSAL_WINDOW && window < 1)
    return fail(IHA_ERR_INVALID_ARG, "%s: window must be >= 1", name);
  iha_status st = check_cache(name, cache, n_pages, page, Hkv, d);
  if (st != IHA_OK) return st;
  if (dt != IHA_BF16) return fail(IHA_ERR_UNSUPPORTED, "%s: q and o must be bf16", name);
  if (Hq % Hkv)
    return fail(IHA_ERR_INVALID_ARG, "%s: Hq %d is not a multiple of Hkv %d", name, Hq, Hkv);
  if (B > (1 << 30))  // the scan of the lengths counts sequences in steps of a CTA
    return fail(IHA_ERR_UNSUPPORTED, "%s: more than 2^30 sequences", name);
  if ((int64_t)table_width * page > (1 << 30))
    return fail(IHA_ERR_UNSUPPORTED, "%s: block table longer than 2^30 tokens", name);
  const int G = Hq / Hkv;
  const int64_t ncols = (int64_t)Nq * G;
  nt = pick_nt(ncols);
  const int64_t ncb = (ncols + 8 * nt - 1) / (8 * nt);
  if (ncols > (1 << 20) || G > 2048 || ncb * ((int64_t)table_width * page / kKvTok + kUnitCost) > INT32_MAX)
    return fail(IHA_ERR_UNSUPPORTED, "%s: more than 2^20 new rows or 2048 query heads of a key head", name);
  if (!aligned16(q) || !aligned16(o))
    return fail(IHA_ERR_ALIGNMENT, "%s: q and o must be 16-byte aligned", name);
  if ((reinterpret_cast<uintptr_t>(block_table) | reinterpret_cast<uintptr_t>(seq_lens) |
       reinterpret_cast<uintptr_t>(lse_out)) &
      3)
    return fail(IHA_ERR_ALIGNMENT, "%s: block_table, seq_lens and lse must be 4-byte aligned", name);
  if (B == 1) sq.b_outer = so.b_outer = 0;
  if (Nq == 1) sq.seq = so.seq = 0;
  if (Hq == 1) sq.head = so.head = 0;
  if (sq.b_outer < 0 || sq.seq < 0 || sq.head < 0 || so.b_outer < 0 || so.seq < 0 || so.head < 0)
    return fail(IHA_ERR_INVALID_ARG, "%s: negative stride", name);
  if ((B > 1 && so.b_outer == 0) || (Nq > 1 && so.seq == 0) || (Hq > 1 && so.head == 0))
    return fail(IHA_ERR_INVALID_ARG, "%s: the output repeats rows (stride 0)", name);
  const Kv4View wo = {3, {B, Nq, Hq}, {so.b_outer, so.seq, so.head}};
  if (kv4_views_meet(wo, wo, 0, d, true))
    return fail(IHA_ERR_INVALID_ARG, "%s: rows of the output overlap one another", name);
  if ((sq.b_outer | sq.seq | sq.head | so.b_outer | so.seq | so.head) & 7)
    return fail(IHA_ERR_ALIGNMENT, "%s: strides must be multiples of 8 elements", name);
  if (reinterpret_cast<uintptr_t>(workspace) & 255)
    return fail(IHA_ERR_ALIGNMENT, "%s: workspace must be 256-byte aligned", name);
  if (workspace_bytes < need)
    return fail(IHA_ERR_INVALID_ARG, "%s: workspace of %zu bytes, needs %zu", name,
                workspace_bytes, need);
  auto span = [&](const iha_strides& s) {
    return ((int64_t)(B - 1) * s.b_outer + (int64_t)(Nq - 1) * s.seq + (int64_t)(Hq - 1) * s.head +
            d) * 2;
  };
  const int64_t nq = span(sq), no = span(so), nc = (int64_t)n_pages * (int64_t)page_bytes;
  const int64_t nl = lse_out ? (int64_t)B * Hq * Nq * 4 : 0;
  const int64_t ntab = (int64_t)B * table_width * 4;
  auto clash = [&](const void* a, int64_t na) {
    return overlaps(a, na, q, nq) || overlaps(a, na, cache, nc) ||
           overlaps(a, na, block_table, ntab) || overlaps(a, na, seq_lens, (int64_t)B * 4);
  };
  if (clash(o, no) || (lse_out && (clash(lse_out, nl) || overlaps(lse_out, nl, o, no))))
    return fail(IHA_ERR_INVALID_ARG, "%s: an output overlaps another tensor", name);
  if (clash(workspace, (int64_t)need) || overlaps(workspace, (int64_t)need, o, no) ||
      (lse_out && overlaps(workspace, (int64_t)need, lse_out, nl)))
    return fail(IHA_ERR_INVALID_ARG, "%s: the workspace overlaps another tensor", name);
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.cache = static_cast<const uint8_t*>(cache);
  p.table = block_table;
  p.lens = seq_lens;
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse_out;
  p.B = B;
  p.Nq = Nq;
  p.Hq = Hq;
  p.Hkv = Hkv;
  p.G = G;
  p.ncols = (int)ncols;
  p.ncb = (int)ncb;
  p.inv_g = ((1ull << 32) + G - 1) / G;
  p.counters = static_cast<unsigned*>(workspace);
  p.parts = reinterpret_cast<float*>(p.counters + kCounterBytes / 4);
  p.part_cols = part_cols(ncols);
  p.part_stride = part_stride(ncols, d);
  p.n_pages = n_pages;
  p.page = page;
  p.blocks_per_page = page / kKvTok;
  p.table_w = table_width;
  p.mask = mask_mode;
  p.window = window;
  if (!(scale > 0.f)) scale = 1.f / sqrtf((float)d);
  if (scale > 1e30f) return fail(IHA_ERR_INVALID_ARG, "%s: scale above 1e30", name);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.sq = sq;
  p.so = so;
  // every CTA resident at once; no more of them than there can be work
  const int64_t most =
      (int64_t)B * Hkv * ncb * ((int64_t)table_width * page / kKvTok + kUnitCost);
  int64_t ctas = (int64_t)sm_count() * ctas_per_sm(nt);
  const int64_t cap = (int64_t)kMaxCtas * ctas_per_sm(nt) / ctas_per_sm(1);
  const int64_t useful = (most + kMinShare * kWarps - 1) / (kMinShare * kWarps);
  if (ctas > useful) ctas = useful;
  if (ctas > cap) ctas = cap;
  // the kernel counts positions of a CTA (kWarps shares and a unit) in 32 bits
  if (most / (ctas * kWarps) > (1 << 28))
    return fail(IHA_ERR_UNSUPPORTED, "%s: too many new tokens or keys for one launch", name);
  grid = (int)ctas;
  return IHA_OK;
}

}  // namespace
}  // namespace iha
