// Softmax attention of new queries over a paged cache held in 4 bits
// (mha_fwd_kv4; layout of the cache: kv4.cuh).
//
//   x_j = scale <q, k_j>,  o = sum_j softmax_j(x) v_j,  k_j = s c per group
//
// One warp works on a block of 16 tokens of one key-value head at a time, for
// 8 columns; a column is one (new token, query head of the group) pair.
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
// once, straight into the registers of the lanes that use them.
#include <math.h>

#include "kv4.cuh"

namespace iha {
namespace {

IHA_DEVICE_ERROR_WORD(attention_kv4)

constexpr int kWarps = 4;
constexpr int kCols = 8;  // columns (new token x query head) of a CTA

struct Kv4AttnParams {
  const __nv_bfloat16* q;
  const uint8_t* cache;
  const int32_t* table;
  const int32_t* lens;
  __nv_bfloat16* o;
  float* lse;
  int B, Nq, Hq, Hkv, G, ncols;  // ncols = Nq * G columns of a key-value head
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

template <int NG>
__global__ void __launch_bounds__(32 * kWarps) attn_kv4_kernel(const Kv4AttnParams p) {
  constexpr int D = 32 * NG;
  __shared__ float sm_m[kWarps][kCols], sm_l[kWarps][kCols];
  __shared__ float sm_o[kWarps][kCols][D + 4];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int hk = blockIdx.x % p.Hkv, cb = blockIdx.x / p.Hkv, b = blockIdx.y;
  int len = __ldg(p.lens + b);
  if (len < 0 || len > p.table_w * p.page) {
    if (tid == 0) atomicOr(&g_dev_error, DEV_ERR_CACHE_INDEX);
    len = len < 0 ? 0 : p.table_w * p.page;
  }
  // visible keys [lo, hi) of a column's new token; none: all
  auto col_range = [&](int col, int& lo, int& hi) {
    const int i = len - p.Nq + col / p.G;  // position of the new token
    hi = p.mask == IHA_MASK_NONE ? len : min(len, i + 1);
    lo = p.mask == IHA_MASK_CAUSAL_WINDOW && i >= p.window ? i - p.window + 1 : 0;
    if (col >= p.ncols) hi = lo = 0;
  };
  const int c_first = cb * kCols, c_last = min(p.ncols, c_first + kCols) - 1;
  int lo_all, hi_all, lo_full, hi_full;  // union and intersection over the columns
  col_range(c_first, lo_all, hi_full);
  col_range(c_last, lo_full, hi_all);
  int col_lo[2], col_hi[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) col_range(c_first + 2 * t + e, col_lo[e], col_hi[e]);

  // Q as B operand: column g, feature pairs (i, i + 4) of octet t of each group
  uint32_t qf[NG][4];
  float qc[NG][2];  // -136 * sum of the group's q, columns 2 t and 2 t + 1
  {
    const int col = c_first + g;
    const bool ok = col < p.ncols;
    const int qi = ok ? col / p.G : 0, qh = hk * p.G + (ok ? col % p.G : 0);
    const __nv_bfloat16* qp = p.q + b * p.sq.b_outer + qi * p.sq.seq + qh * p.sq.head;
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (ok) u = __ldg(reinterpret_cast<const uint4*>(qp + 32 * j + 8 * t));
      qf[j][0] = __byte_perm(u.x, u.z, 0x5410);
      qf[j][1] = __byte_perm(u.x, u.z, 0x7632);
      qf[j][2] = __byte_perm(u.y, u.w, 0x5410);
      qf[j][3] = __byte_perm(u.y, u.w, 0x7632);
      float s = bf16lo_to_f32(u.x) + bf16hi_to_f32(u.x) + bf16lo_to_f32(u.y) +
                bf16hi_to_f32(u.y) + bf16lo_to_f32(u.z) + bf16hi_to_f32(u.z) +
                bf16lo_to_f32(u.w) + bf16hi_to_f32(u.w);
      s += __shfl_xor_sync(0xffffffffu, s, 1);
      s += __shfl_xor_sync(0xffffffffu, s, 2);
      qc[j][0] = -136.f * __shfl_sync(0xffffffffu, s, 8 * t);
      qc[j][1] = -136.f * __shfl_sync(0xffffffffu, s, 8 * t + 4);
    }
  }

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float acc[NG][2][4];
#pragma unroll
  for (int j = 0; j < NG; ++j)
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][a][e] = 0.f;

  const int blk0 = lo_all / kKv4Tok, blk1 = (hi_all + kKv4Tok - 1) / kKv4Tok;
  for (int blk = blk0 + warp; blk < blk1; blk += kWarps) {
    const int pi = blk / p.blocks_per_page;
    const int id = __ldg(p.table + (int64_t)b * p.table_w + pi);
    if (id < 0 || id >= p.n_pages) {
      if (lane == 0) atomicOr(&g_dev_error, DEV_ERR_CACHE_INDEX);
      continue;
    }
    BlockRegs<NG> r;
    r.load(p.cache + kv4_block_of(id, blk - pi * p.blocks_per_page, hk, p.Hkv, p.blocks_per_page,
                                  NG),
           lane);
    float x[4] = {0.f, 0.f, 0.f, 0.f};  // (token g, columns 2t, 2t+1), (token g + 8, ...)
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      float c[4] = {qc[j][0], qc[j][1], qc[j][0], qc[j][1]};
      mma_bf16(c, nibbles(r.k[0][j], 0), nibbles(r.k[1][j], 0), nibbles(r.k[0][j], 1),
               nibbles(r.k[1][j], 1), qf[j][0], qf[j][1]);
      mma_bf16(c, nibbles(r.k[0][j], 2), nibbles(r.k[1][j], 2), nibbles(r.k[0][j], 3),
               nibbles(r.k[1][j], 3), qf[j][2], qf[j][3]);
      const float s0 = scale_of<NG>(r.ks, 0, j), s1 = scale_of<NG>(r.ks, 1, j);
      x[0] = fmaf(s0, c[0], x[0]);
      x[1] = fmaf(s0, c[1], x[1]);
      x[2] = fmaf(s1, c[2], x[2]);
      x[3] = fmaf(s1, c[3], x[3]);
    }
    const int key = blk * kKv4Tok + g;
    const bool edge = blk * kKv4Tok < lo_full || (blk + 1) * kKv4Tok > hi_full;
    bool vis[4] = {true, true, true, true};
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] *= p.scale_log2;
    if (edge) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int kk = key + 8 * (e >> 1);
        vis[e] = kk >= col_lo[e & 1] && kk < col_hi[e & 1];
        if (!vis[e]) x[e] = -INFINITY;
      }
    }
    const float t0 = fmaxf(x[0], x[2]), t1 = fmaxf(x[1], x[3]);
    if (__any_sync(0xffffffffu, t0 > m[0] + 8.f || t1 > m[1] + 8.f)) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float n = e ? t1 : t0;
        n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 4));
        n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 8));
        n = fmaxf(n, __shfl_xor_sync(0xffffffffu, n, 16));
        n = fmaxf(n, m[e]);
        const float f = m[e] == -INFINITY ? 0.f : exp2f(m[e] - n);
        m[e] = n;
        l[e] *= f;
#pragma unroll
        for (int j = 0; j < NG; ++j)
#pragma unroll
          for (int a = 0; a < 2; ++a) {
            acc[j][a][e] *= f;
            acc[j][a][e + 2] *= f;
          }
      }
    }
    float pr[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float ref = m[e & 1] == -INFINITY ? 0.f : m[e & 1];
      pr[e] = fast_exp2(x[e] - ref);
    }
    l[0] += pr[0] + pr[2];
    l[1] += pr[1] + pr[3];
#pragma unroll
    for (int j = 0; j < NG; ++j) {
      const float s0 = scale_of<NG>(r.vs, 0, j), s1 = scale_of<NG>(r.vs, 1, j);
      float w[4] = {pr[0] * s0, pr[1] * s0, pr[2] * s1, pr[3] * s1};
      if (edge) {  // a hidden token's scale may be anything, NaN too
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!vis[e]) w[e] = 0.f;
      }
      const uint32_t b0 = transpose8x8(pack_bf16x2(w[0], w[1]));
      const uint32_t b1 = transpose8x8(pack_bf16x2(w[2], w[3]));
#pragma unroll
      for (int a = 0; a < 2; ++a)
        mma_bf16(acc[j][a], minus136(nibbles(r.v[0][j], 2 * a)),
                 minus136(nibbles(r.v[0][j], 2 * a + 1)), minus136(nibbles(r.v[1][j], 2 * a)),
                 minus136(nibbles(r.v[1][j], 2 * a + 1)), b0, b1);
    }
  }

  // join the warps
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 4);
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 8);
    l[e] += __shfl_xor_sync(0xffffffffu, l[e], 16);
    if (g == 0) {
      sm_m[warp][2 * t + e] = m[e];
      sm_l[warp][2 * t + e] = l[e];
    }
#pragma unroll
    for (int j = 0; j < NG; ++j)
      *reinterpret_cast<float4*>(&sm_o[warp][2 * t + e][32 * j + 4 * g]) =
          make_float4(acc[j][0][e], acc[j][0][e + 2], acc[j][1][e], acc[j][1][e + 2]);
  }
  __syncthreads();
  for (int i = tid; i < kCols * D / 4; i += 32 * kWarps) {
    const int c = i / (D / 4), f = (i - c * (D / 4)) * 4;
    const int col = c_first + c;
    if (col >= p.ncols) continue;
    float mm = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm_m[w][c]);
    const float ref = mm == -INFINITY ? 0.f : mm;
    float ll = 0.f;
    float4 oo = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float a = exp2f(sm_m[w][c] - ref);
      const float4 v = *reinterpret_cast<const float4*>(&sm_o[w][c][f]);
      ll = fmaf(a, sm_l[w][c], ll);
      oo.x = fmaf(a, v.x, oo.x);
      oo.y = fmaf(a, v.y, oo.y);
      oo.z = fmaf(a, v.z, oo.z);
      oo.w = fmaf(a, v.w, oo.w);
    }
    const float inv = ll == 0.f ? 0.f : 1.f / ll;
    const int qi = col / p.G, qh = hk * p.G + col % p.G;
    uint2 u;
    u.x = pack_bf16x2(oo.x * inv, oo.y * inv);
    u.y = pack_bf16x2(oo.z * inv, oo.w * inv);
    *reinterpret_cast<uint2*>(p.o + b * p.so.b_outer + qi * p.so.seq + qh * p.so.head + f) = u;
    if (p.lse && f == 0)
      p.lse[((int64_t)b * p.Hq + qh) * p.Nq + qi] =
          ll == 0.f ? -INFINITY : (ref + log2f(ll)) * 0.6931471805599453f;
  }
}

bool overlaps(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

}  // namespace
}  // namespace iha

extern "C" {

size_t mha_fwd_kv4_workspace_bytes(int B, int Nq, int Hq, int Hkv, int d) {
  (void)B, (void)Nq, (void)Hq, (void)Hkv, (void)d;
  return 256;
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
  const int64_t ncols = (int64_t)Nq * G, ncb = (ncols + kCols - 1) / kCols;
  if (ncols > (1 << 24) || ncb * Hkv > INT32_MAX || B > 65535)
    return fail(IHA_ERR_UNSUPPORTED, "%s: too many heads, rows or sequences for one launch", name);
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
  const int64_t nt = (int64_t)B * table_width * 4;
  auto clash = [&](const void* a, int64_t na) {
    return overlaps(a, na, q, nq) || overlaps(a, na, cache, nc) ||
           overlaps(a, na, block_table, nt) || overlaps(a, na, seq_lens, (int64_t)B * 4);
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
  const dim3 grid((unsigned)(ncb * Hkv), (unsigned)B);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (d / kKv4Group) {
    case 1: attn_kv4_kernel<1><<<grid, 32 * kWarps, 0, s>>>(p); break;
    case 2: attn_kv4_kernel<2><<<grid, 32 * kWarps, 0, s>>>(p); break;
    case 3: attn_kv4_kernel<3><<<grid, 32 * kWarps, 0, s>>>(p); break;
    default: attn_kv4_kernel<4><<<grid, 32 * kWarps, 0, s>>>(p); break;
  }
  return check_launch(name);
}

}  // extern "C"
