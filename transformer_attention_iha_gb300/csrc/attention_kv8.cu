// Softmax attention of new queries over a paged cache held in 8 bits
// (mha_fwd_kv8; layout of the cache: kv8.cuh), and the keys' weights in it.
//
//   x_j = scale <q, k_j>,  o = sum_j softmax_j(x) v_j,  k_j = 2^e c
//
// One warp works on blocks of 16 tokens of one key-value head, for 8 NT columns; a
// column is one (new token, query head of the group) pair.
//   S^T [16 tokens x 8 columns] = K Q^T by mma.m16n8k16 on fp16: codes are exact in
//     fp16, Q's row is scaled by a power of two to below 2^15 so that its 8-bit
//     mantissas are too (features below 2^-28 of the largest lose bits).  The block's
//     scale multiplies the fp32 accumulators.
//   O^T [d x 8 columns] += V^T P^T, V's scale inside P: P s F in fp16, with a power of
//     two F per column that keeps the largest of the sum so far between 2^5 and 2^15: F
//     falls when a p s outgrows that, and rises with the softmax reference.  A term is
//     off by 2^-11 of itself or, below 2^-19 of the largest, 2^-30 of that.  V's codes
//     are turned by ldmatrix as pairs of features, P^T by movmatrix.
//   Softmax in the log2 domain, fp32; a column's reference moves only when a score
//     exceeds it, to 8 above that score (a token that weighs alone has p = 2^-8, and
//     its P s exactly); then O and the sum are rescaled.
// Work: the line of kv_attn.cuh; each warp keeps a ring of two stages of two blocks (d =
// 128) that bulk copies fill ahead, codes and tails apart.  Calls with weights keep the scores
// (4 bytes where K and V have 2 d), and a second kernel adds 2^(score - reference) / l up.
//
// What bounds it: long contexts HBM (131071 keys x 80 heads of 128, 2.69 GB: 401 to 411 us,
// 6.5 to 6.7 TB/s; 137 registers, 12 warps an SM, 34 per cent of the issue slots); there the
// SMs come to an end between 302 and 400 us, by their place on the chip.  Ragged batches (16
// sequences of up to 8192 keys, 8 key heads, 103 MB): 32 us with 16 columns, 27 with 4, of
// which 3 until copies are under way, 15 at HBM's rate, the rest imbalance, parts and joins.
// 777 keys x 80 heads: latency, 12.3 us.
#include <cuda_fp16.h>

#include "kv8.cuh"
// Unit cost, on 16 ragged sequences of 1 to 8192 keys and 8 key heads, 16 columns: 2 53.8
// us, 4 43.8, 6 36.2, 9 35.7, 14 35.0; 131071 keys x 80 heads 407 to 411.
#define IHA_KV_UNIT_COST 14
#include "kv_attn.cuh"

namespace iha {
namespace {

constexpr int NB = 2;  // blocks computed together
// The largest F, 2^126 (its reciprocal is a normal number), and its exponent field.
constexpr float kTopF = 8.5070591730234616e37f;
constexpr int kTopFExp = 126 + 127;

// What is written of a row besides O.  A function that is called: in the body of the joins,
// four rows unrolled, it cost 16-column calls 1.2 of 32 us.
__device__ __noinline__ void write_row_stats(float* lse, float2* rows, int64_t row, float ref,
                                             float l, float inv) {
  if (lse != nullptr) lse[row] = lse_of(ref, l);
  if (rows != nullptr) rows[row] = make_float2(ref, inv);
}

struct Kv8AttnParams : KvAttnParams {
  Kv8Pages pages;
  float* scores;  // nullable: [B, Hkv, ncols, table_w * page], log2 domain, -inf where hidden
  // with scores: each row's reference (log2 domain) and 1 / l.  (Not its lse: a sum of both
  // in fp32, let alone turned to natural logarithms and back, is off by 2^-24 of its size, and
  // so are all weights of the row: 1e-4 of themselves for scores about 1000.)
  float2* rows;
  __device__ __forceinline__ void write_row(int64_t row, float ref, float l, float inv) const {
    write_row_stats(lse, rows, row, ref, l, inv);
  }
};

__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 u;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w)
               : "r"(addr)
               : "memory");
  return u;
}

// A warp's softmax state over one unit: 8 NT columns of one head.  ONE: a single
// column, the odd columns of the operands are not computed.
template <int D, int NT, bool ONE>
struct Attend {
  static constexpr int CH = D / 16, BYTES = kv8_block_bytes(D);
  static constexpr int ES = ONE ? 2 : 1;  // step over the columns of a pair
  int lane, g, t;
  uint32_t row_at, row_chunk;  // this lane's row for ldmatrix: its offset, its first chunk
  uint32_t qf[NT == 1 ? CH : 1][2];
  uint2* q_smem;               // NT > 1: [NT * CH * 32]
  float cm[NT][2];             // accumulators of columns 2 t, 2 t + 1 to scores, log2 domain
  // a column's reference: 8 above the maximum when it was last set; mlim is the same,
  // or -inf while no key has been seen (mref = 0)
  float mlim[NT][2], mref[NT][2], l[NT][2], F[NT][2];
  float acc[NT][CH][4];        // (feature 16 c + 2 g, columns 2 t, 2 t + 1), (the next feature, ...)

  __device__ __forceinline__ void init(int lane_, uint2* smem) {
    lane = lane_;
    g = lane >> 2;
    t = lane & 3;
    q_smem = smem;
    const int row = lane & 15;
    row_at = row * D;
    row_chunk = (uint32_t)((lane >> 4) ^ kv8_swap(D, row));
  }

  // Q as B operand: column 8 nt + g, features 16 c + 4 t .. + 3
  __device__ __forceinline__ void load_q(const KvAttnParams& p, int b, int hk, int c_first) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int col = c_first + 8 * nt + g;
      const bool in = col < p.ncols;
      const int qi = in ? token_of(p, col) : 0, qh = hk * p.G + (in ? col - qi * p.G : 0);
      const __nv_bfloat16* qp = p.q + b * p.sq.b_outer + qi * p.sq.seq + qh * p.sq.head + 4 * t;
      uint2 v[CH];
      uint32_t top = 0;
#pragma unroll
      for (int c = 0; c < CH; ++c)
        v[c] = in ? __ldg(reinterpret_cast<const uint2*>(qp + 16 * c)) : make_uint2(0, 0);
#pragma unroll
      for (int c = 0; c < CH; ++c)
        top = __vmaxu2(top, __vmaxu2(v[c].x & 0x7FFF7FFFu, v[c].y & 0x7FFF7FFFu));
      top = max(top & 0xFFFFu, top >> 16);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      // largest |q| in [2^e, 2^(e + 1)): Q is scaled by 2^(14 - e)
      const int e = max((int)(top >> 7) - 127, -112);
      const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
      const float back = ldexpf(p.scale_log2, e - 14);
      cm[nt][0] = __shfl_sync(0xffffffffu, back, 8 * t);
      cm[nt][1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const uint32_t h0 = pack_f16x2(bf16lo_to_f32(v[c].x) * up, bf16hi_to_f32(v[c].x) * up);
        const uint32_t h1 = pack_f16x2(bf16lo_to_f32(v[c].y) * up, bf16hi_to_f32(v[c].y) * up);
        if constexpr (NT == 1) {
          qf[c][0] = h0;
          qf[c][1] = h1;
        } else {
          q_smem[(nt * CH + c) * 32 + lane] = make_uint2(h0, h1);
        }
      }
      mlim[nt][0] = mlim[nt][1] = -INFINITY;
      mref[nt][0] = mref[nt][1] = 0.f;
      l[nt][0] = l[nt][1] = 0.f;
      F[nt][0] = F[nt][1] = kTopF;
#pragma unroll
      for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int e_ = 0; e_ < 4; ++e_) acc[nt][c][e_] = 0.f;
    }
    __syncwarp();
  }

  // A operand of 16 features: K rows (tokens), or V columns turned.
  __device__ __forceinline__ uint32_t at(uint32_t s, int cc) const {
    return s + row_at + ((row_chunk ^ (2 * cc)) << 4);
  }

  // Two blocks in shared memory at s, tails at st, of keys from key0 on.  edge: not all of their keys
  // are visible to every column; gone: a bit per block that no page holds or that lies
  // past the unit's end, past: a bit per block past it.  scores: nullable, of column 0.
  __device__ __forceinline__ void step(const Kv8AttnParams& p, uint32_t s, uint32_t st, int key0,
                                       bool edge, uint32_t gone, uint32_t past, int len,
                                       int c_first, float* scores, int64_t cap) {
    float x[NT][NB][4];  // (token g, columns 2 t, 2 t + 1), (token g + 8, ...)
    float sv[NB];
    uint32_t nan[NB];
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const uint4 tail = lds128(st + b * kKv8TailBytes);
      const float sk = __uint_as_float(tail.x);
      sv[b] = __uint_as_float(tail.y);
      nan[b] = tail.z;
      float c4[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) c4[nt][e] = 0.f;
#pragma unroll
      for (int cc = 0; cc < CH / 2; ++cc) {
        uint32_t w[4];  // rows g, g + 8 of chunk 2 cc, then of 2 cc + 1
        ldmatrix4(at(s + b * BYTES, cc), w);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t a0 = e4m3_to_f16((uint16_t)w[2 * h]);
          const uint32_t a1 = e4m3_to_f16((uint16_t)w[2 * h + 1]);
          const uint32_t a2 = e4m3_to_f16((uint16_t)(w[2 * h] >> 16));
          const uint32_t a3 = e4m3_to_f16((uint16_t)(w[2 * h + 1] >> 16));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if constexpr (NT == 1) {
              mma_f16(c4[nt], a0, a1, a2, a3, qf[2 * cc + h][0], qf[2 * cc + h][1]);
            } else {
              const uint2 f = q_smem[(nt * CH + 2 * cc + h) * 32 + lane];
              mma_f16(c4[nt], a0, a1, a2, a3, f.x, f.y);
            }
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; e += ES) x[nt][b][e] = c4[nt][e] * (sk * cm[nt][e & 1]);
    }
    uint32_t any_nan = 0;
#pragma unroll
    for (int b = 0; b < NB; ++b) any_nan |= nan[b];
    if (any_nan != 0) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 4; e += ES)
            if ((nan[b] >> (g + (e & 2) * 4)) & 1u) x[nt][b][e] = __uint_as_float(0x7FC00000u);
    }
    uint32_t hidden = 0;  // bit 4 (nt NB + b) + e
    if (edge) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; e += ES) {
          const int col = c_first + 8 * nt + 2 * t + e;
          int lo, hi;
          col_range(p, len, col, lo, hi);
          if (col >= p.ncols) hi = 0;
#pragma unroll
          for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int key = key0 + b * kKv8Tok + g + 8 * h;
              if (key < lo || key >= hi || ((gone >> b) & 1u)) {
                hidden |= 1u << (4 * (nt * NB + b) + 2 * h + e);
                x[nt][b][2 * h + e] = -INFINITY;
              }
            }
        }
    }
    if (scores != nullptr) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 2; e += ES) {
          const int col = c_first + 8 * nt + 2 * t + e;
          if (col < p.ncols)
#pragma unroll
            for (int b = 0; b < NB; ++b)
              if (!((past >> b) & 1u)) {
                float* to = scores + col * cap + key0 + b * kKv8Tok + g;
                to[0] = x[nt][b][e];
                to[8] = x[nt][b][e + 2];
              }
        }
    }
    uint32_t pf[NT][NB][2];  // P as B operand
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float top[2];
#pragma unroll
      for (int e = 0; e < 2; e += ES) {
        top[e] = fmaxf(x[nt][0][e], x[nt][0][e + 2]);
#pragma unroll
        for (int b = 1; b < NB; ++b) top[e] = fmax3f(top[e], x[nt][b][e], x[nt][b][e + 2]);
      }
      if (__any_sync(0xffffffffu, top[0] > mlim[nt][0] || (!ONE && top[1] > mlim[nt][1]))) {
#pragma unroll
        for (int e = 0; e < 2; e += ES) {
          float v = top[e];
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
          // a column below its limit keeps its reference
          v = v > mlim[nt][e] ? v + 8.f : mlim[nt][e];
          const float ref = v == -INFINITY ? 0.f : v;
          // the move; 0 from the first reference (nothing to rescale)
          const float up = mlim[nt][e] == -INFINITY ? 0.f : ref - mref[nt][e];
          mlim[nt][e] = v;
          mref[nt][e] = ref;
          l[nt][e] *= exp2f(-up);
          // F rises by the next power of two, as far as its range goes, and O grows by
          // what that is above the move
          const int ef = __float_as_uint(F[nt][e]) >> 23;
          const int to = min(ef + (int)ceilf(fminf(up, 512.f)), kTopFExp);
          F[nt][e] = __uint_as_float((uint32_t)to << 23);
          const float k = exp2f((float)(to - ef) - up);
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            acc[nt][c][e] *= k;
            acc[nt][c][e + 2] *= k;
          }
        }
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
#pragma unroll
        for (int e = 0; e < 4; e += ES) x[nt][b][e] = fast_exp2(x[nt][b][e] - mref[nt][e & 1]);
        l[nt][0] += x[nt][b][0] + x[nt][b][2];
        if (!ONE) l[nt][1] += x[nt][b][1] + x[nt][b][3];
      }
      // x becomes w = p s; P = w F.  When a w F exceeds 2^15, F falls to where the
      // largest of them is 2^5
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int e = 0; e < 4; e += ES) x[nt][b][e] *= sv[b];
      if (edge) {  // the scale of a block that no page holds may be anything
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 4; e += ES)
            if ((hidden >> (4 * (nt * NB + b) + e)) & 1u) x[nt][b][e] = 0.f;
      }
      bool grow = false;
      float wt[2];
#pragma unroll
      for (int e = 0; e < 2; e += ES) {
        wt[e] = fmaxf(x[nt][0][e], x[nt][0][e + 2]);
#pragma unroll
        for (int b = 1; b < NB; ++b) wt[e] = fmax3f(wt[e], x[nt][b][e], x[nt][b][e + 2]);
        grow |= wt[e] * F[nt][e] > 32768.f;
      }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int e = 0; e < 2; e += ES) {
          float v = wt[e];
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
          // 2^(5 - exponent of v), from its bits; v is 0 or positive, infinite at most
          const int ex = __float_as_uint(fmaxf(v, 0.f)) >> 23;
          const float to = __uint_as_float((uint32_t)min(259 - ex, kTopFExp) << 23);
          if (to < F[nt][e]) {
            const float f = to / F[nt][e];
            F[nt][e] = to;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
              acc[nt][c][e] *= f;
              acc[nt][c][e + 2] *= f;
            }
          }
        }
      }
      if (any_nan != 0) {  // a visible V row of NaN makes all of O NaN
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int e = 0; e < 4; e += ES)
            if (((nan[b] >> (16 + g + (e & 2) * 4)) & 1u) &&
                !((hidden >> (4 * (nt * NB + b) + e)) & 1u))
              x[nt][b][e] = __uint_as_float(0x7FC00000u);
      }
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        pf[nt][b][0] = transpose8x8(
            pack_f16x2(x[nt][b][0] * F[nt][0], ONE ? 0.f : x[nt][b][1] * F[nt][1]));
        pf[nt][b][1] = transpose8x8(
            pack_f16x2(x[nt][b][2] * F[nt][0], ONE ? 0.f : x[nt][b][3] * F[nt][1]));
      }
    }
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      if ((gone >> b) & 1u) continue;  // whatever is there may be NaN, and 0 NaN is
#pragma unroll
      for (int cc = 0; cc < CH / 2; ++cc) {
        uint32_t w[4];  // tokens 2 t, 2 t + 1 of each half, features 2 g, 2 g + 1 of two chunks
        ldmatrix4_trans(at(s + b * BYTES + kKv8Tok * D, cc), w);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // (token, token') of the first feature in the low half, of the second in the high
          const uint32_t u0 = __byte_perm(w[2 * h], 0, 0x3120);
          const uint32_t u1 = __byte_perm(w[2 * h + 1], 0, 0x3120);
          const uint32_t a0 = e4m3_to_f16((uint16_t)u0), a1 = e4m3_to_f16((uint16_t)(u0 >> 16));
          const uint32_t a2 = e4m3_to_f16((uint16_t)u1), a3 = e4m3_to_f16((uint16_t)(u1 >> 16));
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_f16(acc[nt][2 * cc + h], a0, a1, a2, a3, pf[nt][b][0], pf[nt][b][1]);
        }
      }
    }
  }

  // Sums over the warp's lanes; put(column, feature, two features' O, lim, ref, l).
  template <typename Put>
  __device__ __forceinline__ void finish(int ncolv, Put put) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 4);
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 8);
        l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 16);
        const int cc = 8 * nt + 2 * t + e;
        const float f = 1.f / F[nt][e];
        if (cc < ncolv)
#pragma unroll
          for (int c = 0; c < CH; ++c)
            put(cc, 16 * c + 2 * g, make_float2(acc[nt][c][e] * f, acc[nt][c][e + 2] * f),
                mlim[nt][e], mref[nt][e], l[nt][e]);
      }
  }
};

// ---- the line of work.  (The 4-bit attention has the same in its kernel's body: as
// functions they cost it 0.5 to 2.5 per cent, 4 x 32768 keys of 4 columns 56.3 -> 57.7 us.)

// What a CTA keeps in shared memory of its place in the line.
struct LineSmem {
  long long scan[kWarps], base[kWarps];
  int seq[kWarps];
  // units that span warps: at each end of a warp's stretch, {sequence, head,
  // column block, first and last warp (-1, kWarps: in other CTAs), blocks (0: none),
  // CTAs it began before this one, CTAs it ends behind this one}
  int span[kWarps + 1][8];
  int last[2], of[2][2];  // unit at each end of the stretch: joined here, its CTAs
  int abort;
};

// The stretch of the line that this warp has: the length of every warp's share and of
// this one's, and the unit it begins in.  False if the CTA has none (all threads call; a
// length out of range is flagged).
template <int COLS>
__device__ __forceinline__ bool find_stretch(const KvAttnParams& p, LineSmem& sm,
                                             int& share, int& stretch, Unit& u) {
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  // positions of this thread's sequence, and of all; batches longer than the
  // CTA are summed first and scanned in a second pass
  auto positions = [&](int b, bool check) {
    if (b >= p.B) return 0ll;
    const int raw = __ldg(p.lens + b), len = min(max(raw, 0), p.table_w * p.page);
    if (check && blockIdx.x == 0 && raw != len) atomicOr(&g_dev_error, DEV_ERR_CACHE_INDEX);
    return (long long)head_positions<COLS>(p, len) * p.Hkv;
  };
  auto scan = [&](long long v, long long& all) {  // inclusive sum over the CTA's threads
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, v, k);
      if (lane >= k) v += x;
    }
    if (lane == 31) sm.scan[warp] = v;
    __syncthreads();
    all = 0;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      if (k < warp) v += sm.scan[k];
      all += sm.scan[k];
    }
    return v;
  };
  long long v = positions(tid, true), all, incl = scan(v, all), total = all;
  for (int b0 = kThreads; b0 < p.B; b0 += kThreads) {
    long long more;
    __syncthreads();
    scan(positions(b0 + tid, true), more);
    total += more;
  }
  const long long workers = gridDim.x * kWarps;
  share = max(kMinShare, (int)((total + workers - 1) / workers));
  const long long w_cta = (long long)share * (blockIdx.x * kWarps), w = w_cta + share * warp;
  if (w_cta >= total) return false;
  stretch = (int)min((long long)share, max(0ll, total - w));
  // the sequence that holds position w, for each warp
  for (long long base = 0, b0 = 0;;) {
    const long long lo = base + incl - v, hi = base + incl;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) {
      const long long wk = w_cta + share * k;
      if (wk >= lo && wk < hi) {
        sm.seq[k] = (int)b0 + tid;
        sm.base[k] = lo;
      }
    }
    base += all;
    b0 += kThreads;
    __syncthreads();
    if (b0 >= p.B || base > w_cta + share * (kWarps - 1)) break;  // the same everywhere
    v = positions((int)b0 + tid, false);
    incl = scan(v, all);
  }
  if (stretch > 0) {
    u.b = sm.seq[warp];
    u.len = seq_len(p, u.b);
    const int per_head = head_positions<COLS>(p, u.len);
    const long long rel = w - sm.base[warp];
    u.hk = (rel >> 31) == 0 ? (int)((unsigned)rel / (unsigned)per_head) : (int)(rel / per_head);
    int s = (int)(rel - (long long)u.hk * per_head);
    for (u.cb = 0;; ++u.cb) {
      unit_blocks<COLS>(p, u.len, u.cb, u.b0, u.n);
      if (s < u.n + kUnitCost || u.cb == p.ncb - 1) break;
      s -= u.n + kUnitCost;
    }
    u.at = -s;
  }
  return true;
}

// A warp's ring of blocks in shared memory: STAGES stages of up to RUN blocks of one
// unit, filled ahead by bulk copies in runs inside a page; the page id of the run after
// the current one is read ahead.
template <int BYTES, int RUN, int STAGES, int COLS>
struct BlockRing {
  struct Run {
    int id, head, in_page, cnt;  // cnt blocks of the page, 0: no more
    int left;                    // blocks of the unit from this run on
  };
  Unit pu;
  int pr, pr_end, stretch, lane;
  bool more;
  Run run, run_next;
  const uint8_t *src, *src_tail;  // the run's next block and its tail; null: no such page
  // bit per block of the ring: no such page; bit per stage: copies under way, and the
  // parity of its barrier
  uint32_t bad, flying, phase, ring, tails, bars;

  __device__ __forceinline__ Run next_run(const Kv8AttnParams& p) {
    Run r = {0, 0, 0, 0, 0};
    while (more && pr >= pr_end) {
      more = pu.at + pu.n + kUnitCost < stretch && next_unit<COLS>(p, pu);
      if (more) my_blocks(pu, stretch, pr, pr_end);
    }
    if (more) {
      const int blk = pu.b0 + pr, pi = blk / p.blocks_per_page;
      r.in_page = blk - pi * p.blocks_per_page;
      r.left = pr_end - pr;
      r.cnt = min(p.blocks_per_page - r.in_page, r.left);
      r.head = pu.hk;
      r.id = __ldg(p.table + (int64_t)pu.b * p.table_w + pi);
      pr += r.cnt;
    }
    return r;
  }
  __device__ __forceinline__ void take_run(const Kv8AttnParams& p) {
    run = run_next;
    if (run.cnt > 0) {
      run_next = next_run(p);
      const bool in = run.id >= 0 && run.id < p.n_pages;
      if (!in && lane == 0) atomicOr(&g_dev_error, DEV_ERR_CACHE_INDEX);
      src = in ? p.cache + p.pages.block(run.id, run.head, run.in_page, BYTES / 32) : nullptr;
      src_tail = in ? p.cache + p.pages.tail(run.id, run.head, run.in_page) : nullptr;
    }
  }
  __device__ __forceinline__ void start(const Kv8AttnParams& p, const Unit& u, int stretch_,
                                        int lane_, uint32_t ring_, uint32_t tails_,
                                        uint32_t bars_) {
    pu = u;
    stretch = stretch_;
    lane = lane_;
    ring = ring_;
    tails = tails_;
    bars = bars_;
    more = true;
    bad = flying = phase = 0;
    src = src_tail = nullptr;
    my_blocks(pu, stretch, pr, pr_end);
    run_next = next_run(p);
    take_run(p);
#pragma unroll 1
    for (int i = 0; i < STAGES; ++i) fetch(p, i);
  }
  __device__ __forceinline__ void fetch(const Kv8AttnParams& p, int stage) {
    bad &= ~(((1u << RUN) - 1u) << (stage * RUN));
    flying &= ~(1u << stage);
    if (run.cnt == 0) return;
    const int want = min(RUN, run.left);
    uint32_t bytes = 0;
    int have = 0;
    do {
      const int c = min(want - have, run.cnt);
      if (src != nullptr) {
        if (lane == 0) {
          bulk_load(ring + (stage * RUN + have) * BYTES, src, c * BYTES, bars + 8 * stage);
          bulk_load(tails + (stage * RUN + have) * kKv8TailBytes, src_tail, c * kKv8TailBytes,
                    bars + 8 * stage);
        }
        bytes += c * (BYTES + kKv8TailBytes);
        src += c * BYTES;
        src_tail += c * kKv8TailBytes;
      } else {
        bad |= ((1u << c) - 1u) << (stage * RUN + have);
      }
      have += c;
      run.cnt -= c;
      run.left -= c;
      if (run.cnt == 0) take_run(p);
    } while (have < want);
    if (lane == 0) mbar_arrive_expect_tx(bars + 8 * stage, bytes);
    flying |= 1u << stage;
  }
  __device__ __forceinline__ bool wait(const Kv8AttnParams& p, int stage, volatile int* abort_flag) {
    if (!mbar_wait_warp(bars + 8 * stage, (phase >> stage) & 1u, abort_flag, p.wait_ns))
      return false;
    phase ^= 1u << stage;
    return true;
  }
  // After a wait that gave up: what is in flight lands before the memory goes away.
  __device__ __forceinline__ void drain(const Kv8AttnParams& p) {
    volatile int no_abort = 0;
    for (int i = 0; i < STAGES; ++i)
      if ((flying >> i) & 1u) mbar_wait(bars + 8 * i, (phase >> i) & 1u, &no_abort, p.wait_ns);
  }
};

// Notes where the part of a unit that a warp leaves belongs: with its first and last
// warp and CTA (one lane calls, for a unit that goes on behind the warp, or began before
// the CTA).
__device__ __forceinline__ void note_span(LineSmem& sm, const Unit& u, int warp, int share, int r0,
                                          int r1) {
  const int p0 = share * warp + u.at + kUnitCost;  // of the unit's first block, in the CTA
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (k ? r1 < u.n : (r0 > 0 && warp == 0)) {
      int* sp = sm.span[k ? warp + 1 : 0];
      sp[0] = u.b;
      sp[1] = u.hk;
      sp[2] = u.cb;
      sp[3] = p0 >= 0 ? p0 / share : -1;
      sp[4] = min((p0 + u.n - 1) / share, kWarps);
      sp[5] = u.n;
      // (in 32 bits: a 64-bit division is a call, and costs the loop registers)
      sp[6] = p0 >= 0 ? 0 : (-p0 + share * kWarps - 1) / (share * kWarps);
      sp[7] = (p0 + u.n - 1) / (share * kWarps);
    }
}

// join_ctas for units of many columns: I items of a thread, U parts of each, on their way
// together (a join waits for memory: 16 columns of 128 features, 7 parts, ...).
template <int D, int COLS>
__device__ __forceinline__ void join_wide(const Kv8AttnParams& p, const int* span, const int* of,
                                          float* scratch) {
  const int c_first = span[2] * COLS, first = of[0], last = of[1];
  const int items = min(COLS, p.ncols - c_first) * (D / 4);
  if (COLS * D / 4 <= kThreads || items <= kThreads) {
    join_ctas<D, COLS>(p, span, of, scratch);
    return;
  }
  constexpr int I = COLS * D / 4 > 2 * kThreads ? 4 : 2, U = I == 4 ? 4 : 8;
  for (int i0 = threadIdx.x; i0 < items; i0 += I * kThreads) {
    Joined a[I];
#pragma unroll
    for (int i = 0; i < I; ++i) a[i].clear();
    for (int c0 = first; c0 <= last; c0 += U) {
      float m[I][U], l[I][U];
      float4 o[I][U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int c = min(c0 + k, last);
        const float* pp = p.parts + ((int64_t)c * kCtaParts + (c == first ? 1 : 0)) * p.part_stride;
#pragma unroll
        for (int i = 0; i < I; ++i) {
          const int at = min(i0 + i * kThreads, items - 1), cc = at / (D / 4);
          m[i][k] = c0 + k <= last ? __ldcg(pp + p.part_cols * D + cc) : -INFINITY;
          l[i][k] = c0 + k <= last ? __ldcg(pp + p.part_cols * D + p.part_cols + cc) : 0.f;
          o[i][k] = __ldcg(reinterpret_cast<const float4*>(pp + 4 * at));
        }
      }
#pragma unroll
      for (int i = 0; i < I; ++i) a[i].add(m[i], l[i], o[i]);
    }
#pragma unroll
    for (int i = 0; i < I; ++i) {
      const int at = i0 + i * kThreads, cc = at / (D / 4);
      if (at < items) a[i].write(p, span, c_first + cc, (at - cc * (D / 4)) * 4);
    }
  }
}

// Units that span warps: joins this CTA's parts, and, of a unit that spans CTAs, all of
// them in the CTA that arrives last (all threads call).  head_of, tail_of: a warp's part
// of a unit that ends in its stretch after beginning before it, and of one that goes on.
template <int D, int COLS, typename Head, typename Tail>
__device__ __forceinline__ void join_units(const Kv8AttnParams& p, LineSmem& sm, Head head_of,
                                           Tail tail_of, float* cta_parts, float* scratch) {
  const int tid = threadIdx.x;
  __syncthreads();
  if (sm.abort) return;
  auto same_unit = [&](int i, int k) {
    return sm.span[i][5] != 0 && sm.span[i][0] == sm.span[k][0] && sm.span[i][1] == sm.span[k][1] &&
           sm.span[i][2] == sm.span[k][2];
  };
#pragma unroll 1
  for (int k = 0; k <= kWarps; ++k) {
    const int* span = sm.span[k];
    const int first = span[3], last = span[4];
    if (span[5] == 0 || (k > 0 && same_unit(k - 1, k))) continue;
    const int c_first = span[2] * COLS, ncolv = min(COLS, p.ncols - c_first);
    const int lo = max(first, 0), hi = min(last, kWarps - 1);
    float* to = cta_parts + (first >= 0 ? 1 : 0) * p.part_stride;
    constexpr int I = COLS * D / 4 > 2 * kThreads ? 4 : COLS * D / 4 > kThreads ? 2 : 1;
    const int items = ncolv * (D / 4);
    for (int i0 = tid; i0 < items; i0 += I * kThreads) {  // I items of a thread at once
      Joined a[I];
#pragma unroll
      for (int i = 0; i < I; ++i) a[i].clear();
      for (int x = lo; x <= hi; ++x) {
        const float* pp = x == last ? head_of(x) : tail_of(x);
        float m[I], l[I];
        float4 o[I];
#pragma unroll
        for (int i = 0; i < I; ++i) {
          const int at = min(i0 + i * kThreads, items - 1), cc = at / (D / 4);
          m[i] = pp[p.part_cols * D + cc];
          l[i] = pp[p.part_cols * D + p.part_cols + cc];
          o[i] = *reinterpret_cast<const float4*>(pp + 4 * at);
        }
#pragma unroll
        for (int i = 0; i < I; ++i) a[i].add(m[i], l[i], o[i]);
      }
#pragma unroll
      for (int i = 0; i < I; ++i) {
        const int at = i0 + i * kThreads, cc = at / (D / 4), f = (at - cc * (D / 4)) * 4;
        if (at >= items) break;
        if (first >= 0 && last < kWarps) {
          a[i].write(p, span, c_first + cc, f);
        } else {
          *reinterpret_cast<float4*>(to + cc * D + f) = a[i].o;
          if (f == 0) {
            to[p.part_cols * D + cc] = a[i].m;
            to[p.part_cols * D + p.part_cols + cc] = a[i].l;
          }
        }
      }
    }
  }
  // units that span CTAs, the one the CTA begins in and the one it ends in
  __syncthreads();
  if (tid < 2) {
    const int* span = sm.span[tid == 0 ? 0 : kWarps];
    bool join = span[5] != 0 && (tid == 0 || !same_unit(0, kWarps));
    if (join) {
      // CTAs of the unit's first and last block
      const int first = blockIdx.x - span[6], last = blockIdx.x + span[7];
      join = first != last && arrive(p.counters + first) == (unsigned)(last - first);
      if (join) p.counters[first] = 0u;  // ready for the next call
      sm.of[tid][0] = first;
      sm.of[tid][1] = last;
    }
    sm.last[tid] = join;
  }
  __syncthreads();
#pragma unroll 1
  for (int k = 0; k < 2; ++k)
    if (sm.last[k]) join_wide<D, COLS>(p, sm.span[k == 0 ? 0 : kWarps], sm.of[k], scratch);
}

// ---- the kernel
// A warp's ring: stages of up to run_of blocks.
constexpr int kStages = 2;
__host__ __device__ constexpr int run_of(int d) { return d >= 96 ? 2 : d == 64 ? 4 : 8; }

template <int D, int NT>
struct Smem {
  // a warp's ring; when it has run out, the part of the unit its stretch ends in
  alignas(128) uint8_t ring[kWarps][kStages][run_of(D)][kv8_block_bytes(D)];
  alignas(16) uint8_t tails[kWarps][kStages][run_of(D)][kKv8TailBytes];
  uint2 q[NT > 1 ? kWarps : 1][NT > 1 ? NT * (D / 16) * 32 : 1];
  uint64_t full[kWarps][kStages];
  LineSmem line;
};

template <int D, int NT, bool ONE>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(NT))
    attn_kv8_kernel(const Kv8AttnParams p) {
  constexpr int COLS = 8 * NT, BYTES = kv8_block_bytes(D), RUN = run_of(D);
  extern __shared__ __align__(128) uint8_t smem_raw[];
  Smem<D, NT>& sm = *reinterpret_cast<Smem<D, NT>*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // the same in the warp, for the compiler too
  volatile int* abort_flag = &sm.line.abort;
  if (lane == 0)
    for (int i = 0; i < kStages; ++i)
      mbar_init(smem_u32(&sm.full[warp][i]), p.withhold && blockIdx.x == 0 && i == 0 ? 2 : 1);
  if (tid <= kWarps) sm.line.span[tid][5] = 0;
  if (tid == 0) sm.line.abort = 0;
  mbar_init_fence();
  int share, stretch;
  Unit u;
  if (!find_stretch<COLS>(p, sm.line, share, stretch, u)) return;

  // where a warp of this CTA leaves its part of a unit that ends in its stretch
  // after beginning before it, and of one that goes on after it
  float* const cta_parts = p.parts + (int64_t)blockIdx.x * kCtaParts * p.part_stride;
  auto head_of = [&](int w) { return cta_parts + (2 + w) * p.part_stride; };
  auto tail_of = [&](int w) { return reinterpret_cast<float*>(sm.ring[w]); };
  if (stretch > 0) {
    const int g = lane >> 2, t = lane & 3;
    // Q of the unit this warp comes to next, on its way while the unit before is computed
    auto prefetch_q = [&](const Unit& n) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int col = n.cb * COLS + 8 * nt + g;
        if (col < p.ncols && t < (D + 63) / 64) {  // lines of 128 bytes: 64 features
          const int qi = token_of(p, col), qh = n.hk * p.G + col - qi * p.G;
          const __nv_bfloat16* qp =
              p.q + n.b * p.sq.b_outer + qi * p.sq.seq + qh * p.sq.head + 64 * t;
          asm volatile("prefetch.L1 [%0];" ::"l"(qp));
        }
      }
    };
    prefetch_q(u);
    BlockRing<BYTES, RUN, kStages, COLS> ring;
    ring.start(p, u, stretch, lane, smem_u32(sm.ring[warp]), smem_u32(sm.tails[warp]),
               smem_u32(sm.full[warp]));
    Attend<D, NT, ONE> a;
    a.init(lane, sm.q[NT > 1 ? warp : 0]);
    const int64_t cap = (int64_t)p.table_w * p.page;
    int stage = 0;
    bool ok = true;

    // ---- units of the stretch
    for (;;) {
      int r0, r1;
      my_blocks(u, stretch, r0, r1);
      const int empty_at = u.at + kUnitCost - 1;  // an empty unit belongs to this position
      const bool empty = u.n == 0 && empty_at >= 0 && empty_at < stretch;
      if (r0 < r1 || empty) {
        const int c_first = u.cb * COLS, ncolv = min(COLS, p.ncols - c_first);
        int lo_full, hi_full, x_;  // keys that every column of the unit sees
        col_range(p, u.len, c_first, x_, hi_full);
        col_range(p, u.len, c_first + ncolv - 1, lo_full, x_);
        a.load_q(p, u.b, u.hk, c_first);
        {
          Unit n = u;
          if (u.at + u.n + kUnitCost < stretch && next_unit<COLS>(p, n)) prefetch_q(n);
        }
        float* scores =
            p.scores ? p.scores + ((int64_t)u.b * p.Hkv + u.hk) * p.ncols * cap : nullptr;
        // blocks r with rf0 <= r - b0 < rf0 + rf_n are visible to every column
        const int rf0 = (lo_full + kKv8Tok - 1) / kKv8Tok - u.b0;
        const unsigned rf_n = (unsigned)max(0, (hi_full >> 4) - u.b0 - rf0);
#pragma unroll 1
        for (int r = r0; r < r1; r += RUN) {
          if (!ring.wait(p, stage, abort_flag)) {
            ok = false;
            break;
          }
          // blocks of the stage that no page holds, or past the stretch, are computed
          // like the others and hidden
          const uint32_t past = r1 - r < RUN ? ~0u << (r1 - r) : 0u;
          const uint32_t gone = ((ring.bad >> (stage * RUN)) & ((1u << RUN) - 1u)) | past;
#pragma unroll 1
          for (int k0 = 0; k0 < RUN; k0 += NB) {
            const int rk = r + k0;
            if (rk >= r1) break;
            const uint32_t gk = (gone >> k0) & ((1u << NB) - 1u);
            const bool edge = (unsigned)(rk - rf0) >= rf_n || (unsigned)(rk + NB - 1 - rf0) >= rf_n ||
                              gk != 0;
            a.step(p, ring.ring + (stage * RUN + k0) * BYTES,
                   ring.tails + (stage * RUN + k0) * kKv8TailBytes, (u.b0 + rk) * kKv8Tok, edge, gk,
                   past >> k0, u.len, c_first, scores, cap);
          }
          __syncwarp();  // the stage has been read
          ring.fetch(p, stage);
          stage = stage + 1 == kStages ? 0 : stage + 1;
        }
        if (!ok) break;

        // ---- the unit's rows, or this warp's part of them
        const bool whole = r0 <= 0 && r1 >= u.n;
        // r1 < u.n: the unit goes on in the next warp, and this one is done
        float* part = r1 < u.n ? tail_of(warp) : head_of(warp);
        a.finish(ncolv, [&](int cc, int f, float2 o, float lim, float ref, float l) {
          if (whole) {
            write_out(p, u.b, u.hk, c_first + cc, f, o, ref, l);
          } else {
            *reinterpret_cast<float2*>(part + cc * D + f) = o;
            if (f == 0) {
              part[p.part_cols * D + cc] = lim;
              part[p.part_cols * D + p.part_cols + cc] = l;
            }
          }
        });
        if (!whole && lane == 0) note_span(sm.line, u, warp, share, r0, r1);
      }
      if (u.at + u.n + kUnitCost >= stretch || !next_unit<COLS>(p, u)) break;
    }
    if (!ok) {  // a copy never came: report it, let what is in flight land
      *abort_flag = 1;
      if (lane == 0) {
        atomicOr(&g_dev_error, DEV_ERR_WAIT_TIMEOUT);
        p.counters[kGaveUp] = 1u;  // the weights' kernel then leaves them alone
      }
      ring.drain(p);
    }
  }
  launch_dependents();  // the weights' CTAs may come; they wait for this grid's end
  join_units<D, COLS>(p, sm.line, head_of, tail_of, cta_parts, reinterpret_cast<float*>(sm.ring));
}

struct WeighParams {
  KvAttnParams a;
  const float *scores, *weights;
  const float2* rows;
  float* out;
  int64_t cap;
  int chunks;  // CTAs of a head
};

constexpr int kWeighKeys = 1024;  // keys that a CTA takes at a time

// out[b, h, j] = weights[b, h, j] + the sum over columns of 2^(score - reference) / l, four
// neighbouring keys a thread (VEC: as vectors).  Launched behind the attention: the first
// weights are on their way while that ends.  (1 token over 4 ragged sequences of up to
// 32768 keys x 20 heads: 5 to 8 us behind the attention's 74.)
template <bool VEC>
__global__ void __launch_bounds__(kWeighKeys / 4) kv8_weigh_kernel(const WeighParams p) {
  const int plane = blockIdx.x / p.chunks, b = plane / p.a.Hkv, hk = plane - b * p.a.Hkv;
  const int chunk = (int)blockIdx.x - plane * p.chunks;
  const int len = seq_len(p.a, b);
  // behind the last key weights are copied; in place there is nothing to do
  const int64_t end = p.weights == p.out ? len : p.cap;
  float w[4] = {0.f, 0.f, 0.f, 0.f};
  auto load = [&](int64_t j) {
    const float* from = p.weights + plane * p.cap + j;
    if (VEC) {
      const float4 v = *reinterpret_cast<const float4*>(from);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = from[i];
    }
  };
  const int64_t first = (int64_t)chunk * kWeighKeys + 4 * (int)threadIdx.x;
  if (first < end) load(first);
  wait_for_grid();
  // an attention that gave up left scores and rows unwritten, in all of its units perhaps
  const bool gave_up = __ldcg(p.a.counters + kGaveUp) != 0u;
  for (int64_t j64 = first; j64 < end; j64 += (int64_t)p.chunks * kWeighKeys) {
    const int j = (int)j64;
    if (j64 != first) load(j64);
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int col = 0; j < len && col < p.a.ncols; ++col) {
      int lo, hi;
      col_range(p.a, len, col, lo, hi);
      if (j + 4 <= lo || j >= hi) continue;
      const int qi = token_of(p.a, col), qh = hk * p.a.G + (col - qi * p.a.G);
      // (scores, references and 1 / l: not through the read-only path)
      const float4 v = __ldcg(reinterpret_cast<const float4*>(
          p.scores + (plane * (int64_t)p.a.ncols + col) * p.cap + j));
      const float x[4] = {v.x, v.y, v.z, v.w};
      const int64_t row = ((int64_t)b * p.a.Hq + qh) * p.a.Nq + qi;
      const float2 r = __ldcg(p.rows + row);
#pragma unroll
      for (int i = 0; i < 4; ++i)  // outside [lo, hi) the score may be anything
        if (j + i >= lo && j + i < hi && x[i] != -INFINITY)
          sum[i] += exp2f(x[i] - r.x) * r.y;
    }
    if (gave_up) return;
    float* to = p.out + plane * p.cap + j;
    if (VEC) {
      *reinterpret_cast<float4*>(to) =
          make_float4(w[0] + sum[0], w[1] + sum[1], w[2] + sum[2], w[3] + sum[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) to[i] = w[i] + sum[i];
    }
  }
}

template <int D, int NT, bool ONE>
iha_status launch_nt(const Kv8AttnParams& p, int grid, cudaStream_t s) {
  static_assert((sizeof(Smem<D, NT>) + 1024) * ctas_per_sm(NT) <= 228 * 1024,
                "8-bit attention: the CTAs of an SM do not fit its shared memory");
  static_assert(sizeof(Smem<D, NT>::ring) >= kThreads * 6 * sizeof(float), "scratch of the join");
  static_assert(sizeof(Smem<D, NT>::ring) / kWarps >= 8 * NT * (D + 2) * sizeof(float),
                "a warp's part of a unit goes into its ring");
  static SmemLimit limit;
  const cudaError_t e = limit.ensure(attn_kv8_kernel<D, NT, ONE>, (int)sizeof(Smem<D, NT>));
  if (e != cudaSuccess)
    return fail(IHA_ERR_CUDA, "mha_fwd_kv8 (smem attribute): %s", cudaGetErrorString(e));
  attn_kv8_kernel<D, NT, ONE><<<grid, kThreads, sizeof(Smem<D, NT>), s>>>(p);
  return check_launch("mha_fwd_kv8");
}
template <int D>
iha_status launch(const Kv8AttnParams& p, int nt, int grid, cudaStream_t s) {
  if (p.ncols == 1) return launch_nt<D, 1, true>(p, grid, s);
  return nt == 1 ? launch_nt<D, 1, false>(p, grid, s) : launch_nt<D, 2, false>(p, grid, s);
}

size_t part_bytes(int64_t ncols, int d) {
  const int ctas = kMaxCtas * ctas_per_sm(pick_nt(ncols)) / ctas_per_sm(1);
  return (size_t)ctas * kCtaParts * part_stride(ncols, d) * sizeof(float);
}

size_t row_floats(int B, int Hq, int Nq) {  // one a row; what follows starts on 16 bytes
  return ((size_t)B * Hq * Nq + 3) & ~(size_t)3;
}

constexpr int kMaxWeighed = 64;  // columns whose scores a call with weights keeps

}  // namespace
}  // namespace iha

extern "C" {

size_t mha_fwd_kv8_workspace_bytes(int B, int Nq, int Hq, int Hkv, int d, int weight_keys) {
  if (B <= 0 || Nq <= 0 || Hkv <= 0 || Hq <= 0 || Hq % Hkv || d <= 0 || weight_keys < 0) return 0;
  const int64_t ncols = (int64_t)Nq * (Hq / Hkv);
  // counters, parts; with weights two floats a row (one of them counts without weights
  // too), the rows' scores
  size_t n = iha::kCounterBytes + iha::part_bytes(ncols, d) +
             iha::row_floats(B, Hq, Nq) * sizeof(float);
  if (weight_keys > 0 && (double)B * Hkv * ncols * weight_keys > 1e15) return 0;  // no such
  if (weight_keys > 0)
    n += (iha::row_floats(B, Hq, Nq) + (size_t)B * Hkv * ncols * weight_keys) * sizeof(float);
  return n;
}

iha_status mha_fwd_kv8(const void* q, const void* cache, const int32_t* block_table,
                       const int32_t* seq_lens, void* o, float* lse_out, const float* weights,
                       float* weights_out, void* workspace, size_t workspace_bytes, int B, int Nq,
                       int Hq, int Hkv, int d, int n_pages, int page, int table_width,
                       iha_strides sq, iha_strides so, float scale, iha_mask mask_mode, int window,
                       iha_dtype dt, void* stream) {
  using namespace iha;
  const char* name = "mha_fwd_kv8";
  const int64_t cap = (int64_t)table_width * page;
  if ((weights == nullptr) != (weights_out == nullptr))
    return fail(IHA_ERR_INVALID_ARG, "%s: weights and weights_out go together", name);
  const int keys = weights && cap > 0 && cap <= (1 << 30) ? (int)cap : 0;
  if (keys > 0 && Nq > 0 && Hkv > 0 && (double)B * Hq * Nq * keys > 1e15)
    return fail(IHA_ERR_UNSUPPORTED, "%s: too many scores", name);
  Kv8AttnParams p;
  int nt, grid;
  iha_status st = kv_attn_setup(
      name, p, nt, grid, kv8_check_cache, kv8_page_bytes(page, Hkv, d),
      mha_fwd_kv8_workspace_bytes(B, Nq, Hq, Hkv, d, keys), q, cache, block_table, seq_lens, o,
      lse_out, workspace, workspace_bytes, B, Nq, Hq, Hkv, d, n_pages, page, table_width, sq, so,
      scale, mask_mode, window, dt);
  if (st != IHA_OK) return st;
  p.pages.set(page, Hkv, d);
  p.scores = nullptr;
  p.rows = nullptr;
  if (weights) {
    if (p.ncols > kMaxWeighed)
      return fail(IHA_ERR_UNSUPPORTED, "%s: weights of more than %d rows of a key head", name,
                  kMaxWeighed);
    if ((reinterpret_cast<uintptr_t>(weights) | reinterpret_cast<uintptr_t>(weights_out)) & 3)
      return fail(IHA_ERR_ALIGNMENT, "%s: weights must be 4-byte aligned", name);
    bool neg;
    auto span_of = [&](const iha_strides& t) { return view_bytes(t, B, 1, Nq, Hq, d, 2, &neg); };
    if ((int64_t)B * Hkv > (1 << 26))
      return fail(IHA_ERR_UNSUPPORTED, "%s: weights of more than 2^26 heads", name);
    const int64_t nw = (int64_t)B * Hkv * cap * 4, no = span_of(p.so);
    if ((weights != weights_out && overlaps(weights, nw, weights_out, nw)) ||
        overlaps(weights_out, nw, q, span_of(p.sq)) ||
        overlaps(weights_out, nw, cache, (int64_t)n_pages * (int64_t)kv8_page_bytes(page, Hkv, d)) ||
        overlaps(weights_out, nw, block_table, (int64_t)B * table_width * 4) ||
        overlaps(weights_out, nw, seq_lens, (int64_t)B * 4) ||
        overlaps(weights_out, nw, workspace, (int64_t)workspace_bytes) ||
        overlaps(weights, nw, workspace, (int64_t)workspace_bytes) ||
        overlaps(weights_out, nw, o, no) || overlaps(weights, nw, o, no) ||
        (lse_out && (overlaps(weights_out, nw, lse_out, (int64_t)B * Hq * Nq * 4) ||
                     overlaps(weights, nw, lse_out, (int64_t)B * Hq * Nq * 4))))
      return fail(IHA_ERR_INVALID_ARG, "%s: weights overlap another tensor", name);
    float* own = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kCounterBytes +
                                          part_bytes(p.ncols, d));
    p.rows = reinterpret_cast<float2*>(own);
    p.scores = own + 2 * row_floats(B, Hq, Nq);
  }
  p.wait_ns = wait_limit_for_next_launch();
  p.withhold = withhold_for_this_launch() ? 1 : 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  IHA_KV8_D_SWITCH(d, st = launch<kD>(p, nt, grid, s))
  if (st != IHA_OK || !weights) return st;
  // CTAs of a head: for all of its keys, but no more than fill the GPU (the table may be
  // far wider than the sequences)
  const int64_t all = (cap + kWeighKeys - 1) / kWeighKeys;
  const int64_t fill = (8 * (int64_t)sm_count() + (int64_t)B * Hkv - 1) / ((int64_t)B * Hkv);
  const WeighParams w = {p,           p.scores, weights, p.rows,
                         weights_out, cap,      (int)(all < fill ? all : fill)};
  const unsigned ctas = (unsigned)(B * Hkv * w.chunks);
  return launch_behind(name, aligned16(weights) && aligned16(weights_out) ? kv8_weigh_kernel<true>
                                                                          : kv8_weigh_kernel<false>,
                       ctas, kWeighKeys / 4, s, w);
}

}  // extern "C"
