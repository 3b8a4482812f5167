// Softmax attention of new queries over a paged cache held in 4 bits
// (mha_fwd_kv4; layout of the cache: kv4.cuh).
//
//   x_j = scale <q, k_j>,  o = sum_j softmax_j(x) v_j,  k_j = s c per group
//
// One warp works on a block of 16 tokens of one key-value head at a time, for
// 8 NT columns; a column is one (new token, query head of the group) pair.
//   S^T [16 tokens x 8 columns] = K Q^T: per group of 32 features two
//     mma.m16n8k16 with the codes as the A operand.  A nibble n becomes the
//     bf16 value 128 + n by one OR (exact: 7 mantissa bits), and the
//     accumulator starts at -136 sum_f q_f, so it ends at sum_f q_f c_f; the
//     group's scale multiplies it in fp32.
//   O^T [d x 8 columns] += V^T P^T: the codes c = (128 + n) - 136 are exact in
//     bf16; the scale of a token and group goes into P: bf16(p s), the one
//     rounding of this product (2^-9 relative per term, as P has in the bf16
//     attention).  P^T turns from accumulator to B operand by movmatrix.
//   Softmax in the log2 domain, fp32; a column's reference maximum moves only
//   when a score exceeds it by more than 8, then O and the sum are rescaled.
// Codes are never expanded in memory: 36 NG bytes per token and head are read
// once, straight into the registers of the lanes that use them, one block
// ahead of the block being computed.
//
// Work is one line of blocks: sequence by sequence, head by head, column block
// by column block (a unit), 16 tokens after 16 tokens.  Every CTA takes an
// equal contiguous stretch of the line, whatever the lengths of the sequences,
// so a single long sequence and a ragged batch both fill the GPU.  Lengths are
// read on the device (each CTA sums them up), so a captured call replays with
// other lengths.  A unit that lies in one CTA's stretch is finished there; one
// that spans several leaves partial results (m, l, O in fp32) in the workspace,
// and the CTA that arrives last joins them in order.
#include <math.h>

#include "kv4.cuh"

namespace iha {
namespace {

IHA_DEVICE_ERROR_WORD(attention_kv4)

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCtas = 640;  // workspace slots; 152 SMs x 4 CTAs and some
// A CTA's stretch is at least this many blocks (two for each warp): shorter
// ones cost more in joining than they save.
constexpr int kMinBlocks = 2 * kWarps;

struct Kv4AttnParams {
  const __nv_bfloat16* q;
  const uint8_t* cache;
  const int32_t* table;
  const int32_t* lens;
  __nv_bfloat16* o;
  float* lse;
  unsigned* counters;  // [kMaxCtas], zero between calls
  float* partials;     // [kMaxCtas][2][part_stride]
  int part_cols, part_stride;
  int B, Nq, Hq, Hkv, G, ncols, ncb;  // ncols = Nq * G columns of a key-value head, in ncb blocks
  int n_pages, page, blocks_per_page, table_w;
  int mask, window;
  float scale_log2;
  iha_strides sq, so;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// Nibbles i and i + 4 of w as the bf16 pair (128 + n, 128 + n').
__device__ __forceinline__ uint32_t nibbles(uint32_t w, int i) {
  return ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
}
// (128 + n) - 136 = n - 8 on a pair, exact.
__device__ __forceinline__ uint32_t minus136(uint32_t v) {
  __nv_bfloat162 x = *reinterpret_cast<__nv_bfloat162*>(&v);
  const uint32_t b = 0x43084308u;
  x = __hsub2(x, *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&x);
}

// NG words of one lane (contiguous, 4 NG-byte aligned).
template <int NG>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[NG]) {
  if constexpr (NG == 4) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = u.x;
    w[1] = u.y;
    w[2] = u.z;
    w[3] = u.w;
  } else if constexpr (NG == 2) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(p));
    w[0] = u.x;
    w[1] = u.y;
  } else {
#pragma unroll
    for (int j = 0; j < NG; ++j) w[j] = __ldg(reinterpret_cast<const uint32_t*>(p) + j);
  }
}

// One lane's share of a 16-token block: codes of both halves, scales of
// tokens g and g + 8.
template <int NG>
struct BlockRegs {
  uint32_t k[2][NG], v[2][NG], ks[NG], vs[NG];
  __device__ __forceinline__ void load(const uint8_t* blk, int lane) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      load_words<NG>(blk + (c * 32 + lane) * 4 * NG, k[c]);
      load_words<NG>(blk + kv4_v_codes(NG) + (c * 32 + lane) * 4 * NG, v[c]);
    }
    load_words<NG>(blk + kv4_k_scales(NG) + (lane >> 2) * 4 * NG, ks);
    load_words<NG>(blk + kv4_v_scales(NG) + (lane >> 2) * 4 * NG, vs);
  }
};
// Scale of token half c, group j, from a lane's NG scale words.
template <int NG>
__device__ __forceinline__ float scale_of(const uint32_t (&w)[NG], int c, int j) {
  const int h = c * NG + j;
  return (h & 1) ? bf16hi_to_f32(w[h >> 1]) : bf16lo_to_f32(w[h >> 1]);
}

// Four features of one output row: O / l, and with the first four the row's lse.
__device__ __forceinline__ void write_out(const Kv4AttnParams& p, int b, int hk, int col, int f,
                                          float4 o, float ref, float l) {
  const int qi = col / p.G, qh = hk * p.G + (col - qi * p.G);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint2 u;
  u.x = pack_bf16x2(o.x * inv, o.y * inv);
  u.y = pack_bf16x2(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>(p.o + b * p.so.b_outer + qi * p.so.seq + qh * p.so.head + f) = u;
  if (p.lse && f == 0)
    p.lse[((int64_t)b * p.Hq + qh) * p.Nq + qi] =
        l == 0.f ? -INFINITY : (ref + log2f(l)) * 0.6931471805599453f;
}

// Visible keys [lo, hi) of column col of a sequence of len keys.
__device__ __forceinline__ void col_range(const Kv4AttnParams& p, int len, int col, int& lo,
                                          int& hi) {
  const int i = len - p.Nq + col / p.G;  // position of the new token
  hi = p.mask == IHA_MASK_NONE ? len : min(len, i + 1);
  lo = p.mask == IHA_MASK_CAUSAL_WINDOW && i >= p.window ? i - p.window + 1 : 0;
}

// Blocks [b0, b1) that column block cb (COLS columns) of a sequence sees.
template <int COLS>
__device__ __forceinline__ void unit_blocks(const Kv4AttnParams& p, int len, int cb, int& b0,
                                            int& b1) {
  int lo, hi, x;
  col_range(p, len, cb * COLS, lo, x);
  col_range(p, len, min(p.ncols, cb * COLS + COLS) - 1, x, hi);
  b0 = lo / kKv4Tok;
  b1 = max(b0, (hi + kKv4Tok - 1) / kKv4Tok);
}

__device__ __forceinline__ int seq_len(const Kv4AttnParams& p, int b) {
  return min(max(__ldg(p.lens + b), 0), p.table_w * p.page);
}

// Blocks of one head of sequence b over its column blocks; a unit that sees
// nothing counts as one block, so that some CTA writes its empty rows.
template <int COLS>
__device__ __forceinline__ int head_blocks(const Kv4AttnParams& p, int len) {
  int n = 0;
  for (int cb = 0; cb < p.ncb; ++cb) {
    int b0, b1;
    unit_blocks<COLS>(p, len, cb, b0, b1);
    n += max(1, b1 - b0);
  }
  return n;
}

// Sum over the CTA; every thread gets it (s: kWarps entries).
__device__ __forceinline__ long long cta_sum(long long v, long long* s) {
#pragma unroll
  for (int k = 16; k > 0; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) v += s[w];
  return v;
}

template <int NG, int NT>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 4 : (NT == 2 ? 3 : 2))
    attn_kv4_kernel(const Kv4AttnParams p) {
  constexpr int D = 32 * NG, COLS = 8 * NT;
  __shared__ float sm_m[kWarps][COLS], sm_l[kWarps][COLS];
  __shared__ __align__(16) float sm_o[kWarps][8][D + 4];
  __shared__ uint4 sm_q[NT > 1 ? NT * NG * 32 : 1];
  __shared__ __align__(16) float sm_qc[NT * NG][8];  // -136 * sum of a group's q, per column
  __shared__ long long sm_scan[kWarps];
  __shared__ long long sm_base;
  __shared__ int sm_seq, sm_last;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;

  // ---- this CTA's stretch of the line
  long long mine = 0;
  for (int b = tid; b < p.B; b += kThreads) {
    const int raw = __ldg(p.lens + b), len = seq_len(p, b);
    if (blockIdx.x == 0 && raw != len) atomicOr(&g_dev_error, DEV_ERR_CACHE_INDEX);
    mine += (long long)head_blocks<COLS>(p, len) * p.Hkv;
  }
  const long long total = cta_sum(mine, sm_scan);
  const long long share = max((long long)kMinBlocks, (total + gridDim.x - 1) / gridDim.x);
  long long w = share * blockIdx.x;
  const long long w_end = min(total, w + share);
  if (w >= total) return;
  // the sequence that holds w
  {
    long long base = 0;
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
      const int b = b0 + tid;
      const long long v =
          b < p.B ? (long long)head_blocks<COLS>(p, seq_len(p, b)) * p.Hkv : 0;
      long long incl = v;
#pragma unroll
      for (int k = 1; k < 32; k <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, incl, k);
        if (lane >= k) incl += u;
      }
      __syncthreads();
      if (lane == 31) sm_scan[warp] = incl;
      __syncthreads();
      long long all = 0;
#pragma unroll
      for (int k = 0; k < kWarps; ++k) {
        if (k < warp) incl += sm_scan[k];
        all += sm_scan[k];
      }
      if (w >= base + incl - v && w < base + incl) {
        sm_seq = b;
        sm_base = base + incl - v;
      }
      base += all;
      if (base > w) break;  // the same for every thread
    }
    __syncthreads();
  }
  int b = sm_seq;
  long long seq_base = sm_base;

  // ---- units of the stretch
  while (w < w_end && b < p.B) {
    const int len = seq_len(p, b);
    const int per_head = head_blocks<COLS>(p, len);
    const long long rel = w - seq_base;
    const int hk = (int)(rel / per_head);
    int s0 = (int)(rel - (long long)hk * per_head);
    int cb = 0, ub0, ub1, n;
    for (;; ++cb) {
      unit_blocks<COLS>(p, len, cb, ub0, ub1);
      n = max(1, ub1 - ub0);
      if (s0 < n || cb == p.ncb - 1) break;
      s0 -= n;
    }
    const int s1 = (int)min((long long)n, s0 + (w_end - w));
    const long long unit_w = w - s0;  // the unit's place on the line
    const int c_first = cb * COLS, ncolv = min(COLS, p.ncols - c_first);

    int lo_full, hi_full, x_;  // keys that every column of the unit sees
    col_range(p, len, c_first, x_, hi_full);
    col_range(p, len, c_first + ncolv - 1, lo_full, x_);

    // this warp's blocks
    const int nblk = min(ub0 + s1, ub1) - (ub0 + s0);
    const int per_warp = (nblk + kWarps - 1) / kWarps;
    int blk = ub0 + s0 + warp * per_warp;
    const int blk_end = min(ub0 + s0 + nblk, blk + per_warp);

    // pages: the id of the current page and of the next one, read ahead
    int pi = blk / p.blocks_per_page, in_page = blk - pi * p.blocks_per_page;
    const int32_t* trow = p.table + (int64_t)b * p.table_w;
    const int pi_end = (blk_end + p.blocks_per_page - 1) / p.blocks_per_page;
    auto page_id = [&](int i) { return i < pi_end ? __ldg(trow + i) : 0; };
    int id = -1, id_next = 0;
    if (blk < blk_end) {
      id = page_id(pi);
      id_next = page_id(pi + 1);
    }
    BlockRegs<NG> nx;  // the block being fetched
    bool nx_ok = false;
    auto fetch = [&]() {
      nx_ok = id >= 0 && id < p.n_pages;
      if (nx_ok)
        nx.load(p.cache + kv4_block_of(id, in_page, hk, p.Hkv, p.blocks_per_page, NG), lane);
      else if (lane == 0)
        atomicOr(&g_dev_error, DEV_ERR_CACHE_INDEX);
      if (++in_page == p.blocks_per_page) {
        in_page = 0;
        ++pi;
        id = id_next;
        id_next = page_id(pi + 1);
      }
    };
    if (blk < blk_end) fetch();

    // Q as B operand: column 8 nt + g, feature pairs (i, i + 4) of octet t
    uint32_t qf[NT == 1 ? NG : 1][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int col = c_first + 8 * nt + g;
      const bool ok = col < p.ncols;
      const int qi = ok ? col / p.G : 0, qh = hk * p.G + (ok ? col - qi * p.G : 0);
      const __nv_bfloat16* qp = p.q + b * p.sq.b_outer + qi * p.sq.seq + qh * p.sq.head;
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (ok) u = __ldg(reinterpret_cast<const uint4*>(qp + 32 * j + 8 * t));
        const uint32_t f0 = __byte_perm(u.x, u.z, 0x5410), f1 = __byte_perm(u.x, u.z, 0x7632);
        const uint32_t f2 = __byte_perm(u.y, u.w, 0x5410), f3 = __byte_perm(u.y, u.w, 0x7632);
        if constexpr (NT == 1) {
          qf[j][0] = f0;
          qf[j][1] = f1;
          qf[j][2] = f2;
          qf[j][3] = f3;
        } else if (warp == 0) {
          sm_q[(nt * NG + j) * 32 + lane] = make_uint4(f0, f1, f2, f3);
        }
        float s = bf16lo_to_f32(u.x) + bf16hi_to_f32(u.x) + bf16lo_to_f32(u.y) +
                  bf16hi_to_f32(u.y) + bf16lo_to_f32(u.z) + bf16hi_to_f32(u.z) +
                  bf16lo_to_f32(u.w) + bf16hi_to_f32(u.w);
        s += __shfl_xor_sync(0xffffffffu, s, 1);
        s += __shfl_xor_sync(0xffffffffu, s, 2);
        if (warp == 0 && t == 0) sm_qc[nt * NG + j][g] = -136.f * s;
      }
    }
    __syncthreads();

    float m[NT][2], l[NT][2];
    float acc[NT][NG][2][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
      for (int j = 0; j < NG; ++j)
#pragma unroll
        for (int a = 0; a < 2; ++a)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[nt][j][a][e] = 0.f;
    }

    for (; blk < blk_end; ++blk) {
      const BlockRegs<NG> r = nx;
      const bool ok = nx_ok;
      if (blk + 1 < blk_end) fetch();
      if (!ok) continue;
      float x[NT][4];  // (token g, columns 2t, 2t+1), (token g + 8, ...)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[nt][e] = 0.f;
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        uint32_t a[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[2 * i] = nibbles(r.k[0][j], i);
          a[2 * i + 1] = nibbles(r.k[1][j], i);
        }
        const float k0 = scale_of<NG>(r.ks, 0, j), k1 = scale_of<NG>(r.ks, 1, j);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float2 qc = *reinterpret_cast<const float2*>(&sm_qc[nt * NG + j][2 * t]);
          float c[4] = {qc.x, qc.y, qc.x, qc.y};
          if constexpr (NT == 1) {
            mma_bf16(c, a[0], a[1], a[2], a[3], qf[j][0], qf[j][1]);
            mma_bf16(c, a[4], a[5], a[6], a[7], qf[j][2], qf[j][3]);
          } else {
            const uint4 f = sm_q[(nt * NG + j) * 32 + lane];
            mma_bf16(c, a[0], a[1], a[2], a[3], f.x, f.y);
            mma_bf16(c, a[4], a[5], a[6], a[7], f.z, f.w);
          }
          x[nt][0] = fmaf(k0, c[0], x[nt][0]);
          x[nt][1] = fmaf(k0, c[1], x[nt][1]);
          x[nt][2] = fmaf(k1, c[2], x[nt][2]);
          x[nt][3] = fmaf(k1, c[3], x[nt][3]);
        }
      }
      const bool edge = blk * kKv4Tok < lo_full || (blk + 1) * kKv4Tok > hi_full;
      uint32_t hidden = 0;  // bit 4 nt + e
      if (edge) {
        const int key = blk * kKv4Tok + g;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int col = c_first + 8 * nt + 2 * t + (e & 1), kk = key + 8 * (e >> 1);
            int lo, hi;
            col_range(p, len, col, lo, hi);
            if (col >= p.ncols || kk < lo || kk >= hi) {
              hidden |= 1u << (4 * nt + e);
              x[nt][e] = -INFINITY;
            }
          }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < 4; ++e) x[nt][e] *= p.scale_log2;
        const float t0 = fmaxf(x[nt][0], x[nt][2]), t1 = fmaxf(x[nt][1], x[nt][3]);
        if (__any_sync(0xffffffffu, t0 > m[nt][0] + 8.f || t1 > m[nt][1] + 8.f)) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float v = e ? t1 : t0;
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
            v = fmaxf(v, m[nt][e]);
            const float f = m[nt][e] == -INFINITY ? 0.f : exp2f(m[nt][e] - v);
            m[nt][e] = v;
            l[nt][e] *= f;
#pragma unroll
            for (int j = 0; j < NG; ++j)
#pragma unroll
              for (int a = 0; a < 2; ++a) {
                acc[nt][j][a][e] *= f;
                acc[nt][j][a][e + 2] *= f;
              }
          }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // x becomes p
          const float ref = m[nt][e & 1] == -INFINITY ? 0.f : m[nt][e & 1];
          x[nt][e] = fast_exp2(x[nt][e] - ref);
        }
        l[nt][0] += x[nt][0] + x[nt][2];
        l[nt][1] += x[nt][1] + x[nt][3];
      }
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        const float v0 = scale_of<NG>(r.vs, 0, j), v1 = scale_of<NG>(r.vs, 1, j);
        uint32_t a[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[2 * i] = minus136(nibbles(r.v[0][j], i));
          a[2 * i + 1] = minus136(nibbles(r.v[1][j], i));
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float y[4] = {x[nt][0] * v0, x[nt][1] * v0, x[nt][2] * v1, x[nt][3] * v1};
          if (edge) {  // a hidden token's scale may be anything, NaN too
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if ((hidden >> (4 * nt + e)) & 1u) y[e] = 0.f;
          }
          const uint32_t b0 = transpose8x8(pack_bf16x2(y[0], y[1]));
          const uint32_t b1 = transpose8x8(pack_bf16x2(y[2], y[3]));
          mma_bf16(acc[nt][j][0], a[0], a[2], a[1], a[3], b0, b1);
          mma_bf16(acc[nt][j][1], a[4], a[6], a[5], a[7], b0, b1);
        }
      }
    }

    // ---- join the warps: m, l, O of the CTA's part of the unit
    const bool whole = s0 == 0 && s1 == n;
    const int first_cta = (int)(unit_w / share), last_cta = (int)((unit_w + n - 1) / share);
    float* part = p.partials +
                  ((int64_t)blockIdx.x * 2 + ((int)blockIdx.x == first_cta ? 1 : 0)) *
                      p.part_stride;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float v = l[nt][e];
        v += __shfl_xor_sync(0xffffffffu, v, 4);
        v += __shfl_xor_sync(0xffffffffu, v, 8);
        v += __shfl_xor_sync(0xffffffffu, v, 16);
        if (g == 0) {
          sm_m[warp][8 * nt + 2 * t + e] = m[nt][e];
          sm_l[warp][8 * nt + 2 * t + e] = v;
        }
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int cols = min(8, ncolv - 8 * nt);
      if (NT > 1 && cols <= 0) break;
      if (nt > 0) __syncthreads();
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (2 * t + e < cols)
#pragma unroll
          for (int j = 0; j < NG; ++j)
            *reinterpret_cast<float4*>(&sm_o[warp][2 * t + e][32 * j + 4 * g]) =
                make_float4(acc[nt][j][0][e], acc[nt][j][0][e + 2], acc[nt][j][1][e],
                            acc[nt][j][1][e + 2]);
      __syncthreads();
      for (int i = tid; i < cols * (D / 4); i += kThreads) {
        const int c = i / (D / 4), f = (i - c * (D / 4)) * 4, cc = 8 * nt + c;
        float mm = -INFINITY;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) mm = fmaxf(mm, sm_m[k][cc]);
        const float ref = mm == -INFINITY ? 0.f : mm;
        float ll = 0.f;
        float4 oo = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
          const float a = exp2f(sm_m[k][cc] - ref);
          const float4 v = *reinterpret_cast<const float4*>(&sm_o[k][c][f]);
          ll = fmaf(a, sm_l[k][cc], ll);
          oo.x = fmaf(a, v.x, oo.x);
          oo.y = fmaf(a, v.y, oo.y);
          oo.z = fmaf(a, v.z, oo.z);
          oo.w = fmaf(a, v.w, oo.w);
        }
        if (whole) {
          write_out(p, b, hk, c_first + cc, f, oo, ref, ll);
        } else {
          *reinterpret_cast<float4*>(part + cc * D + f) = oo;
          if (f == 0) {
            part[p.part_cols * D + cc] = mm;
            part[p.part_cols * D + p.part_cols + cc] = ll;
          }
        }
      }
    }

    // ---- a unit of several CTAs: the last to arrive joins the parts
    if (!whole) {
      __threadfence();
      __syncthreads();
      if (tid == 0) {
        const unsigned parts = (unsigned)(last_cta - first_cta);  // others than the last
        sm_last = atomicAdd(p.counters + first_cta, 1u) == parts;
        if (sm_last) p.counters[first_cta] = 0u;  // ready for the next call
      }
      __syncthreads();
      if (sm_last) {
        __threadfence();
        auto part_of = [&](int c) {
          return p.partials + ((int64_t)c * 2 + (c == first_cta ? 1 : 0)) * p.part_stride;
        };
        for (int i = tid; i < ncolv * (D / 4); i += kThreads) {
          const int cc = i / (D / 4), f = (i - cc * (D / 4)) * 4;
          float mm = -INFINITY;
          for (int c = first_cta; c <= last_cta; ++c)
            mm = fmaxf(mm, __ldcg(part_of(c) + p.part_cols * D + cc));
          const float ref = mm == -INFINITY ? 0.f : mm;
          float ll = 0.f;
          float4 oo = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int c = first_cta; c <= last_cta; ++c) {
            const float* pp = part_of(c);
            const float a = exp2f(__ldcg(pp + p.part_cols * D + cc) - ref);
            const float4 v = __ldcg(reinterpret_cast<const float4*>(pp + cc * D + f));
            ll = fmaf(a, __ldcg(pp + p.part_cols * D + p.part_cols + cc), ll);
            oo.x = fmaf(a, v.x, oo.x);
            oo.y = fmaf(a, v.y, oo.y);
            oo.z = fmaf(a, v.z, oo.z);
            oo.w = fmaf(a, v.w, oo.w);
          }
          write_out(p, b, hk, c_first + cc, f, oo, ref, ll);
        }
      }
    }
    __syncthreads();  // the unit's shared memory has been read
    w += s1 - s0;
    if (w == seq_base + (long long)per_head * p.Hkv) {
      seq_base = w;
      ++b;
    }
  }
}

bool overlaps(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

// Column blocks of 8, 16 or 32: the fewest passes over the cache; a pass of 16
// or 32 columns unpacks each code once for all of them.
int pick_nt(int64_t ncols) { return ncols <= 8 ? 1 : (ncols <= 16 ? 2 : 4); }

int part_cols(int64_t ncols) {
  const int64_t cols = 8 * pick_nt(ncols);
  return (int)((ncols < cols ? ncols : cols) + 1) & ~1;  // even: rows of floats stay 16-byte
}
int part_stride(int64_t ncols, int d) {  // floats: O, then m, then l
  return (part_cols(ncols) * (d + 2) + 3) & ~3;
}

template <int NG>
void launch(const Kv4AttnParams& p, int nt, int grid, cudaStream_t s) {
  if (nt == 1)
    attn_kv4_kernel<NG, 1><<<grid, kThreads, 0, s>>>(p);
  else if (nt == 2)
    attn_kv4_kernel<NG, 2><<<grid, kThreads, 0, s>>>(p);
  else
    attn_kv4_kernel<NG, 4><<<grid, kThreads, 0, s>>>(p);
}

}  // namespace
}  // namespace iha

extern "C" {

size_t mha_fwd_kv4_workspace_bytes(int B, int Nq, int Hq, int Hkv, int d) {
  if (B <= 0 || Nq <= 0 || Hkv <= 0 || Hq <= 0 || Hq % Hkv || d <= 0) return 0;
  const int64_t ncols = (int64_t)Nq * (Hq / Hkv);
  return sizeof(unsigned) * iha::kMaxCtas +
         (size_t)iha::kMaxCtas * 2 * iha::part_stride(ncols, d) * sizeof(float);
}

iha_status mha_fwd_kv4(const void* q, const void* cache, const int32_t* block_table,
                       const int32_t* seq_lens, void* o, float* lse_out, void* workspace,
                       size_t workspace_bytes, int B, int Nq, int Hq, int Hkv, int d, int n_pages,
                       int page, int table_width, iha_strides sq, iha_strides so, float scale,
                       iha_mask mask_mode, int window, iha_dtype dt, void* stream) {
  using namespace iha;
  const char* name = "mha_fwd_kv4";
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
  iha_status st = kv4_check_cache(name, cache, n_pages, page, Hkv, d);
  if (st != IHA_OK) return st;
  if (dt != IHA_BF16) return fail(IHA_ERR_UNSUPPORTED, "%s: q and o must be bf16", name);
  if (Hq % Hkv)
    return fail(IHA_ERR_INVALID_ARG, "%s: Hq %d is not a multiple of Hkv %d", name, Hq, Hkv);
  if ((int64_t)table_width * page > (1 << 30))
    return fail(IHA_ERR_UNSUPPORTED, "%s: block table longer than 2^30 tokens", name);
  const int G = Hq / Hkv;
  const int64_t ncols = (int64_t)Nq * G;
  const int nt = pick_nt(ncols);
  const int64_t ncb = (ncols + 8 * nt - 1) / (8 * nt);
  if (ncols > (1 << 20) || ncb * ((int64_t)table_width * page / kKv4Tok) > INT32_MAX)
    return fail(IHA_ERR_UNSUPPORTED, "%s: too many new tokens or keys for one launch", name);
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
  if ((sq.b_outer | sq.seq | sq.head | so.b_outer | so.seq | so.head) & 7)
    return fail(IHA_ERR_ALIGNMENT, "%s: strides must be multiples of 8 elements", name);
  if (reinterpret_cast<uintptr_t>(workspace) & 255)
    return fail(IHA_ERR_ALIGNMENT, "%s: workspace must be 256-byte aligned", name);
  const size_t need = mha_fwd_kv4_workspace_bytes(B, Nq, Hq, Hkv, d);
  if (workspace_bytes < need)
    return fail(IHA_ERR_INVALID_ARG, "%s: workspace of %zu bytes, needs %zu", name,
                workspace_bytes, need);
  auto span = [&](const iha_strides& s) {
    return ((int64_t)(B - 1) * s.b_outer + (int64_t)(Nq - 1) * s.seq + (int64_t)(Hq - 1) * s.head +
            d) * 2;
  };
  const int64_t nq = span(sq), no = span(so), nc = (int64_t)n_pages * kv4_page_bytes(page, Hkv, d);
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
  Kv4AttnParams p;
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
  p.counters = static_cast<unsigned*>(workspace);
  p.partials = reinterpret_cast<float*>(p.counters + kMaxCtas);
  p.part_cols = part_cols(ncols);
  p.part_stride = part_stride(ncols, d);
  p.n_pages = n_pages;
  p.page = page;
  p.blocks_per_page = page / kKv4Tok;
  p.table_w = table_width;
  p.mask = mask_mode;
  p.window = window;
  if (!(scale > 0.f)) scale = 1.f / sqrtf((float)d);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.sq = sq;
  p.so = so;
  // every CTA resident at once; no more of them than there can be work
  const int64_t most = (int64_t)B * Hkv * ncb * ((int64_t)table_width * page / kKv4Tok);
  int64_t grid = (int64_t)sm_count() * (nt == 1 ? 4 : (nt == 2 ? 3 : 2));
  if (grid > (most + kMinBlocks - 1) / kMinBlocks) grid = (most + kMinBlocks - 1) / kMinBlocks;
  if (grid > kMaxCtas) grid = kMaxCtas;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (d / kKv4Group) {
    case 1: launch<1>(p, nt, (int)grid, s); break;
    case 2: launch<2>(p, nt, (int)grid, s); break;
    case 3: launch<3>(p, nt, (int)grid, s); break;
    default: launch<4>(p, nt, (int)grid, s); break;
  }
  return check_launch(name);
}

}  // extern "C"
