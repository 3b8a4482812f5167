// Softmax attention of new queries over a paged cache held in 4 bits
// (mha_fwd_kv4; layout of the cache: kv4.cuh).
//
//   x_j = scale <q, k_j>,  o = sum_j softmax_j(x) v_j,  k_j = s c per group
//
// One warp works on a block of 16 tokens of one key-value head at a time, for
// 8 NT columns; a column is one (new token, query head of the group) pair.
//   S^T [16 tokens x 8 columns] = K Q^T: per group of 32 features two
//     mma.m16n8k16 on fp16, with the codes as the A operand.  A nibble n masked
//     in place is the fp16 subnormal n 2^-24 (or 16 n 2^-24 from the upper half
//     of a byte; those features of Q are divided by 16): one AND a pair.  The
//     accumulator starts at -8 2^-24 sum_f q_f, so it ends at 2^-24 sum_f q_f
//     c_f, and the group's scale multiplies it in fp32.  Q's row is scaled by a
//     power of two to below 2^15, so that its 8-bit mantissas are exact in fp16
//     (features below 2^-28 of the largest lose bits).
//   O^T [d x 8 columns] += V^T P^T, the scale of a token and group inside P:
//     up to 2 columns (one token of unshared heads, the common case): the 8
//       columns of the operand hold the 2 columns four times, once per group,
//       each with its group's scale, so P is scaled, rounded and turned once
//       instead of four times; up to 4 columns, twice, for two groups.  P s F in
//       fp16 with a power of two F per column and group that keeps the largest of
//       the sum so far between 2^5 and 2^15: F falls when a p s outgrows that, and
//       rises with the softmax reference, so it follows what is left of a token
//       that later ones overtake.  A term is off by 2^-11 of itself or, if it is
//       below 2^-19 of the largest, 2^-30 of that.  Codes as for K; -8 sum P comes
//       from one more MMA with a constant A operand (the same rounded P) and leaves
//       O every kFlush blocks.
//     more columns: P s in bf16 (2^-8 a term, as P has in the bf16 attention),
//       the codes as bf16 (128 + n) - 136, exact.
//     P^T turns from accumulator to B operand by movmatrix.
//   Softmax in the log2 domain, fp32; a column's reference moves only when a
//   score exceeds it, to 8 above that score (a token that weighs alone has p = 2^-8,
//   and its P s exactly); then O and the sum are rescaled.
// Codes are never expanded in memory: 36 NG bytes per token and head are read
// once, by bulk copies of whole blocks into a ring that each warp owns, and
// unpacked in the registers of the lanes that use them.
//
// Work is one line of positions: sequence by sequence, head by head, column
// block by column block (a unit); a unit takes one position per block of 16
// tokens it sees and kUnitCost for what a unit costs by itself (its Q, its
// output).  Every warp of the grid takes an equal contiguous stretch of the
// line, whatever the lengths of the sequences: one long sequence, a ragged
// batch and many short ones all fill the GPU, and a warp's ring runs on across
// units.  Lengths are read on the device (each CTA sums them up), so a captured
// call replays with other lengths.  A unit that lies in one warp's stretch is
// finished by that warp; one that spans several is joined from the warps' parts
// (m, l, O in fp32), first inside each CTA, then, if it spans CTAs, through the
// workspace by the CTA that arrives last.  The order of the join follows from the
// lengths and the grid (with few columns every n-th part, then the n sums), never from
// timing.
//
// What bounds it: long contexts of one column, HBM and instruction issue about
// alike (131071 keys x 80 heads of 128, 1.51 GB: 246 us, 6.15 TB/s; the same
// kernel without its arithmetic 219 us; 244 warp instructions a block of 16
// tokens, 80 of them the unpacking).  More columns: issue (8 columns 50 us where
// 1 takes 42; 32 columns 116).  Short work: latency, 11.6 to 12.6 us for 777 keys x 80
// heads: lengths and stretch 1.7, page ids and first copies 1.5, Q 0.6, blocks 2,
// joining 2 to 4.
// Unit cost, on a ragged batch (16 sequences of 1 to 8192 keys, 8 key heads): 2 31 us, 4
// 23.6, 6 23.1; on 131071 keys x 80 heads they differ by 1 per cent.
#define IHA_KV_UNIT_COST 6
#include "kv_attn.cuh"

namespace iha {
namespace {

// A warp's ring: stages of up to kRun blocks.  Longer stages spread the
// cost of a wait and a refill; 12 warps of 2 x 4 blocks measured better than 16
// of 2 x 2 (131071 keys x 80 heads: 241 against 260 us; 8 warps: 256).
constexpr int kStages = 2;
constexpr int kRun = 4;
// FEW: the codes' offset leaves O after this many blocks (256 tokens): it costs
// 32 FMAs, and O has grown by 8 s per unit of probability until then.
constexpr int kFlush = 16;
// FEW: the largest F, 2^126 (its reciprocal is a normal number), and its exponent field.
constexpr float kTopF = 8.5070591730234616e37f;
constexpr int kTopFExp = 126 + 127;
// What a caller zeroes of a workspace.  Parts are written before they are read.
constexpr int kZeroBytes = 4096;
static_assert(kCounterBytes <= kZeroBytes, "4-bit attention: counters within the zeroed bytes");
// The four nibble pairs of a word (nibble i of each half) as fp16 subnormals:
// n 2^-24 for i = 0, 2 and 16 n 2^-24 for i = 1, 3.
__device__ __forceinline__ void nibbles_f16(uint32_t w, uint32_t (&v)[4]) {
  const uint32_t h = w >> 8;
  v[0] = w & 0x000F000Fu;
  v[1] = w & 0x00F000F0u;
  v[2] = h & 0x000F000Fu;
  v[3] = h & 0x00F000F0u;
}
// Nibble i of each half of w as the bf16 pair (128 + n, 128 + n').
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

// NG words of one lane (contiguous, 4 NG-byte aligned shared memory).
template <int NG>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[NG]) {
  if constexpr (NG == 4) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    w[0] = u.x;
    w[1] = u.y;
    w[2] = u.z;
    w[3] = u.w;
  } else if constexpr (NG == 2) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    w[0] = u.x;
    w[1] = u.y;
  } else {
#pragma unroll
    for (int j = 0; j < NG; ++j) w[j] = reinterpret_cast<const uint32_t*>(p)[j];
  }
}

// Scale of token half c, group j, from a lane's NG scale words.
template <int NG>
__device__ __forceinline__ float scale_of(const uint32_t (&w)[NG], int c, int j) {
  const int h = c * NG + j;
  return (h & 1) ? bf16hi_to_f32(w[h >> 1]) : bf16lo_to_f32(w[h >> 1]);
}

// A part of a unit's result: O [columns][D], then m, then l, of up to COLS columns.
template <int NG, int NT>
struct Part {
  static constexpr int D = 32 * NG, COLS = 8 * NT, FLOATS = COLS * (D + 2);
};

template <int NG, int NT>
struct Smem {
  // a warp's ring; when it has run out, the part of the unit its stretch ends in
  uint8_t ring[kWarps][kStages][kRun][kv4_block_bytes(NG)];
  uint4 q[NT > 1 ? kWarps : 1][NT > 1 ? NT * NG * 32 : 1];
  // -8 2^-24 sum of a group's q of columns 2 t and 2 t + 1, twice: an accumulator's start
  float4 qc[kWarps][NT * NG][4];
  uint64_t full[kWarps][kStages];
  long long scan[kWarps], base[kWarps];
  int seq[kWarps];
  // units that span warps: at each end of a warp's stretch, {sequence, head,
  // column block, first and last warp (-1, kWarps: in other CTAs), blocks (0: none),
  // CTAs it began before this one, CTAs it ends behind this one}
  int span[kWarps + 1][8];
  int last[2], of[2][2];  // unit at each end of the stretch: joined here, its CTAs
  int abort;
};

// GC: groups that share a P operand (4, 2: see above; 1: none).  ONE: a single
// column, the odd columns of the operands are not computed.
template <int NG, int NT, int GC, bool ONE>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(NT))
    attn_kv4_kernel(const KvAttnParams p) {
  constexpr int D = 32 * NG, COLS = 8 * NT, BYTES = kv4_block_bytes(NG);
  constexpr int NB = 2;            // blocks computed together
  constexpr int ES = ONE ? 2 : 1;      // step over the columns of a pair
  constexpr bool FEW = GC > 1;
  constexpr int REAL = FEW ? 8 / GC : 8;           // columns of a B operand that differ
  constexpr int SH = FEW ? (NG + GC - 1) / GC : 1;  // P operands of a block
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Smem<NG, NT>& sm = *reinterpret_cast<Smem<NG, NT>*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, g = lane >> 2, t = lane & 3;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // the same in the warp, for the compiler too
  volatile int* abort_flag = &sm.abort;
  const int vl = kv4_v_lane(g, t);
  // FEW: of operand s, columns 2 t, 2 t + 1 are columns tc, tc + 1 scaled for group GC s + tg
  const int tg = FEW ? 2 * t / REAL : 0, tc = FEW ? 2 * t % REAL : 2 * t;

  // ---- this warp's stretch of the line
  if (lane == 0)
    for (int i = 0; i < kStages; ++i)
      mbar_init(smem_u32(&sm.full[warp][i]),
                p.withhold && blockIdx.x == 0 && i == 0 ? 2 : 1);
  if (tid <= kWarps) sm.span[tid][5] = 0;
  if (tid == 0) sm.abort = 0;
  mbar_init_fence();
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
      const long long u = __shfl_up_sync(0xffffffffu, v, k);
      if (lane >= k) v += u;
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
  const int share = max(kMinShare, (int)((total + workers - 1) / workers));
  const long long w_cta = (long long)share * (blockIdx.x * kWarps), w = w_cta + share * warp;
  if (w_cta >= total) return;  // the whole CTA
  const int stretch = (int)min((long long)share, max(0ll, total - w));
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

  // where a warp of this CTA leaves its part of a unit that ends in its stretch
  // after beginning before it, and of one that goes on after it
  float* const cta_parts = p.parts + (int64_t)blockIdx.x * kCtaParts * p.part_stride;
  auto head_of = [&](int w) { return cta_parts + (2 + w) * p.part_stride; };
  auto tail_of = [&](int w) { return reinterpret_cast<float*>(sm.ring[w]); };
  bool ok = true;
  if (stretch > 0) {
    Unit u;
    u.b = sm.seq[warp];
    u.len = seq_len(p, u.b);
    {
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

    // Q of the unit this warp comes to next, on its way while the unit before is computed
    auto prefetch_q = [&](const Unit& n) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int col = n.cb * COLS + 8 * nt + g % REAL;
        if (col < p.ncols && t < (NG + 1) / 2) {  // lines of 128 bytes: 64 features
          const int qi = token_of(p, col), qh = n.hk * p.G + col - qi * p.G;
          const __nv_bfloat16* qp =
              p.q + n.b * p.sq.b_outer + qi * p.sq.seq + qh * p.sq.head + 64 * t;
          asm volatile("prefetch.L1 [%0];" ::"l"(qp));
        }
      }
    };
    prefetch_q(u);

    // ---- the ring: stages of up to kRun blocks of one unit, kStages ahead, copied
    // in runs inside a page; the page id of the run after the current one is
    // read ahead
    Unit pu = u;
    int pr, pr_end;
    my_blocks(pu, stretch, pr, pr_end);
    bool more = true;
    struct Run {
      int id, head, in_page, cnt;  // cnt blocks of the page, 0: no more
      int left;                    // blocks of the unit from this run on
    };
    auto next_run = [&]() {
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
    };
    Run run, run_next = next_run();
    const uint8_t* src = nullptr;  // the run's next block; null: no such page
    auto take_run = [&]() {
      run = run_next;
      if (run.cnt > 0) {
        run_next = next_run();
        const bool in = run.id >= 0 && run.id < p.n_pages;
        if (!in && lane == 0) atomicOr(&g_dev_error, DEV_ERR_CACHE_INDEX);
        src = in ? p.cache + kv4_block_of(run.id, run.in_page, run.head, p.Hkv, p.blocks_per_page,
                                          NG)
                 : nullptr;
      }
    };
    take_run();
    // bit per block of the ring: no such page; bit per stage: copies under way,
    // and the parity of its barrier
    uint32_t bad = 0, flying = 0, phase = 0;
    const uint32_t ring = smem_u32(sm.ring[warp]), bars = smem_u32(sm.full[warp]);
    auto fetch = [&](int stage) {
      bad &= ~(((1u << kRun) - 1u) << (stage * kRun));
      flying &= ~(1u << stage);
      if (run.cnt == 0) return;
      const int want = min(kRun, run.left);
      uint32_t bytes = 0;
      int have = 0;
      do {
        const int c = min(want - have, run.cnt);
        if (src != nullptr) {
          if (lane == 0)
            bulk_load(ring + (stage * kRun + have) * BYTES, src, c * BYTES, bars + 8 * stage);
          bytes += c * BYTES;
          src += c * BYTES;
        } else {
          bad |= ((1u << c) - 1u) << (stage * kRun + have);
        }
        have += c;
        run.cnt -= c;
        run.left -= c;
        if (run.cnt == 0) take_run();
      } while (have < want);
      if (lane == 0) mbar_arrive_expect_tx(bars + 8 * stage, bytes);
      flying |= 1u << stage;
    };
#pragma unroll 1
    for (int i = 0; i < kStages; ++i) fetch(i);
    int stage = 0;

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

        // Q as B operand: column 8 nt + g (FEW: column g % REAL), feature pairs
        // (i, i + 4) of octet t, those of odd i divided by 16
        uint32_t qf[NT == 1 ? NG : 1][4];
        float cm[NT][2];  // accumulators of columns 2 t, 2 t + 1 to scores, log2 domain
        __syncwarp();     // the Q of the unit before has been read
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int col = c_first + 8 * nt + g % REAL;
          const bool in = col < p.ncols;
          const int qi = in ? token_of(p, col) : 0, qh = u.hk * p.G + (in ? col - qi * p.G : 0);
          const __nv_bfloat16* qp =
              p.q + u.b * p.sq.b_outer + qi * p.sq.seq + qh * p.sq.head + 8 * t;
          uint4 v[NG];
          uint32_t top = 0;
#pragma unroll
          for (int j = 0; j < NG; ++j)
            v[j] = in ? __ldg(reinterpret_cast<const uint4*>(qp + 32 * j)) : make_uint4(0, 0, 0, 0);
#pragma unroll
          for (int j = 0; j < NG; ++j) {
            top = __vmaxu2(top, __vmaxu2(v[j].x & 0x7FFF7FFFu, v[j].y & 0x7FFF7FFFu));
            top = __vmaxu2(top, __vmaxu2(v[j].z & 0x7FFF7FFFu, v[j].w & 0x7FFF7FFFu));
          }
          top = max(top & 0xFFFFu, top >> 16);
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
          top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
          // largest |q| in [2^e, 2^(e + 1)): Q is scaled by 2^(14 - e)
          const int e = max((int)(top >> 7) - 127, -112);
          const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
          // above 0: a hidden score is -inf times this
          const float back = fmaxf(ldexpf(p.scale_log2, e + 10), 1.1754944e-38f);
          cm[nt][0] = __shfl_sync(0xffffffffu, back, 8 * t);
          cm[nt][1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
#pragma unroll
          for (int j = 0; j < NG; ++j) {
            const float f0 = bf16lo_to_f32(v[j].x) * up, f1 = bf16hi_to_f32(v[j].x) * up;
            const float f2 = bf16lo_to_f32(v[j].y) * up, f3 = bf16hi_to_f32(v[j].y) * up;
            const float f4 = bf16lo_to_f32(v[j].z) * up, f5 = bf16hi_to_f32(v[j].z) * up;
            const float f6 = bf16lo_to_f32(v[j].w) * up, f7 = bf16hi_to_f32(v[j].w) * up;
            const uint32_t h0 = pack_f16x2(f0, f4), h1 = pack_f16x2(f1 * 0.0625f, f5 * 0.0625f);
            const uint32_t h2 = pack_f16x2(f2, f6), h3 = pack_f16x2(f3 * 0.0625f, f7 * 0.0625f);
            if constexpr (NT == 1) {
              qf[j][0] = h0;
              qf[j][1] = h1;
              qf[j][2] = h2;
              qf[j][3] = h3;
            } else {
              sm.q[warp][(nt * NG + j) * 32 + lane] = make_uint4(h0, h1, h2, h3);
            }
            float s = ((f0 + f1) + (f2 + f3)) + ((f4 + f5) + (f6 + f7));
            s += __shfl_xor_sync(0xffffffffu, s, 1);
            s += __shfl_xor_sync(0xffffffffu, s, 2);
            if (t == 0) {  // column g of the pair (g & ~1, g | 1)
              float* c = reinterpret_cast<float*>(&sm.qc[warp][nt * NG + j][g >> 1]) + (g & 1);
              c[0] = c[2] = -4.76837158203125e-07f * s;  // -8 2^-24
            }
          }
        }
        __syncwarp();
        {
          Unit n = u;
          if (u.at + u.n + kUnitCost < stretch && next_unit<COLS>(p, n)) prefetch_q(n);
        }

        // a column's reference: 8 above the maximum when it was last set, so that
        // p = 2^(x - mref) stays below 1 (p times a scale then cannot overflow);
        // mlim is the same, or -inf while no key has been seen (mref = 0)
        float mlim[NT][2], mref[NT][2], l[NT][2];
        float off[SH][4];        // FEW: -8 2^-24 sum P since the last flush
        float F[SH][2];          // FEW: the power of two of a column and group, see below
#pragma unroll
        for (int s = 0; s < SH; ++s) {
          off[s][0] = off[s][1] = off[s][2] = off[s][3] = 0.f;
          F[s][0] = F[s][1] = kTopF;
        }
        float acc[NT][NG][2][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mlim[nt][0] = mlim[nt][1] = -INFINITY;
          mref[nt][0] = mref[nt][1] = 0.f;
          l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
          for (int j = 0; j < NG; ++j)
#pragma unroll
            for (int a = 0; a < 2; ++a)
#pragma unroll
              for (int e = 0; e < 4; ++e) acc[nt][j][a][e] = 0.f;
        }

        auto flush = [&]() {  // take the codes' offset out of O
#pragma unroll
          for (int j = 0; j < NG; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                acc[0][j][h][e] += off[j / GC % SH][e];
                acc[0][j][h][e + 2] = fmaf(16.f, off[j / GC % SH][e], acc[0][j][h][e + 2]);
              }
#pragma unroll
          for (int s = 0; s < SH; ++s) off[s][0] = off[s][1] = off[s][2] = off[s][3] = 0.f;
        };
        // blocks r with rf0 <= r - b0 < rf0 + rf_n are visible to every column
        const int rf0 = (lo_full + kKv4Tok - 1) / kKv4Tok - u.b0;
        const unsigned rf_n = (unsigned)max(0, (hi_full >> 4) - u.b0 - rf0);
#pragma unroll 1
        for (int r = r0; r < r1; r += kRun) {
          if (!mbar_wait_warp(bars + 8 * stage, (phase >> stage) & 1u, abort_flag, p.wait_ns)) {
            ok = false;
            break;
          }
          phase ^= 1u << stage;
          // blocks of the stage that no page holds, or past the unit's end, are
          // computed like the others and hidden
          uint32_t gone = (bad >> (stage * kRun)) & ((1u << kRun) - 1u);
          if (r1 - r < kRun) gone |= ~0u << (r1 - r);
#pragma unroll 1
          for (int k0 = 0; k0 < kRun; k0 += NB) {
            const int rk = r + k0;
            if (rk >= r1) break;
            const uint8_t* blk_s = sm.ring[warp][stage][k0];
            float x[NT][NB][4];  // (token g, columns 2t, 2t+1), (token g + 8, ...)
#pragma unroll
            for (int b = 0; b < NB; ++b) {
              uint32_t kw[2][NG], ks[NG];
              load_words<NG>(blk_s + b * BYTES + lane * 4 * NG, kw[0]);
              load_words<NG>(blk_s + b * BYTES + (32 + lane) * 4 * NG, kw[1]);
              load_words<NG>(blk_s + b * BYTES + kv4_scales(NG) + g * 8 * NG, ks);
#pragma unroll
              for (int j = 0; j < NG; ++j) {
                uint32_t a[4], c8[4];  // rows g and g + 8
                nibbles_f16(kw[0][j], a);
                nibbles_f16(kw[1][j], c8);
                const float k0_ = scale_of<NG>(ks, 0, j), k1_ = scale_of<NG>(ks, 1, j);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  const float4 q4 = sm.qc[warp][nt * NG + j][t];
                  const float c0[4] = {q4.x, q4.y, q4.z, q4.w};
                  float c[4], d[4];
                  if constexpr (NT == 1) {
                    mma_f16(c, a[0], c8[0], a[1], c8[1], qf[j][0], qf[j][1], c0);
                    mma_f16(d, a[2], c8[2], a[3], c8[3], qf[j][2], qf[j][3], c);
                  } else {
                    const uint4 f = sm.q[warp][(nt * NG + j) * 32 + lane];
                    mma_f16(c, a[0], c8[0], a[1], c8[1], f.x, f.y, c0);
                    mma_f16(d, a[2], c8[2], a[3], c8[3], f.z, f.w, c);
                  }
#pragma unroll
                  for (int e = 0; e < 4; e += ES)
                    x[nt][b][e] = j == 0 ? (e < 2 ? k0_ : k1_) * d[e]
                                         : fmaf(e < 2 ? k0_ : k1_, d[e], x[nt][b][e]);
                }
              }
            }

            const bool edge = (unsigned)(rk - rf0) >= rf_n || (unsigned)(rk + NB - 1 - rf0) >= rf_n ||
                              ((gone >> k0) & ((1u << NB) - 1u)) != 0;
            uint32_t hidden = 0;  // bit 4 (nt NB + b) + e
            if (edge) {
              const int key = (u.b0 + rk) * kKv4Tok + g;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; e += ES) {
                  const int col = c_first + 8 * nt + tc + e;
                  int lo, hi;
                  col_range(p, u.len, col, lo, hi);
                  if (col >= p.ncols) hi = 0;
#pragma unroll
                  for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                      const int kk = key + b * kKv4Tok + 8 * h;
                      if (kk < lo || kk >= hi || ((gone >> (k0 + b)) & 1u)) {
                        hidden |= 1u << (4 * (nt * NB + b) + 2 * h + e);
                        x[nt][b][2 * h + e] = -INFINITY;
                      }
                    }
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float top[2];
#pragma unroll
              for (int e = 0; e < 2; e += ES) {
                top[e] = fmaxf(x[nt][0][e], x[nt][0][e + 2]);
#pragma unroll
                for (int b = 1; b < NB; ++b)
                  top[e] = fmax3f(top[e], x[nt][b][e], x[nt][b][e + 2]);
                top[e] *= cm[nt][e];
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
                  const float f = exp2f(-up);
                  mlim[nt][e] = v;
                  mref[nt][e] = ref;
                  l[nt][e] *= f;
#pragma unroll
                  for (int s = 0; s < SH; ++s) {
                    // FEW: F rises by the next power of two, as far as its range goes, and
                    // O grows by what that is above the move (less than 2; each move is by
                    // 2^8 at least, so F is at its top after 32 of them, if no p s lowers it)
                    float k = f;
                    if constexpr (FEW) {
                      const int ef = __float_as_uint(F[s][e]) >> 23;
                      const int to = min(ef + (int)ceilf(fminf(up, 512.f)), kTopFExp);
                      F[s][e] = __uint_as_float((uint32_t)to << 23);
                      k = exp2f((float)(to - ef) - up);
                      off[s][e] *= k;
                    }
#pragma unroll
                    for (int j = FEW ? GC * s : 0; j < (FEW && GC * (s + 1) < NG ? GC * (s + 1) : NG);
                         ++j)
#pragma unroll
                      for (int a = 0; a < 2; ++a) {
                        acc[nt][j][a][e] *= k;
                        acc[nt][j][a][e + 2] *= k;
                      }
                  }
                }
              }
#pragma unroll
              for (int b = 0; b < NB; ++b) {
#pragma unroll
                for (int e = 0; e < 4; e += ES)  // x becomes p
                  x[nt][b][e] = fast_exp2(fmaf(x[nt][b][e], cm[nt][e & 1], -mref[nt][e & 1]));
                l[nt][0] += x[nt][b][0] + x[nt][b][2];
                if (!ONE) l[nt][1] += x[nt][b][1] + x[nt][b][3];
              }
            }
            if constexpr (FEW) {
              // w = p s of this lane's group; P = w F.  F starts at the top of its
              // range; when a w F exceeds 2^15, F falls to where the largest of them is
              // 2^5 (p grows by up to 2^9 until the reference moves, and with it F).
              float w[SH][NB][4];
              bool grow = false;
              float top[SH][2];
#pragma unroll
              for (int s = 0; s < SH; ++s) {
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                  float f0 = 0.f, f1 = 0.f;  // scales of tokens g, g + 8 in this lane's group
                  if (GC * (s + 1) <= NG || GC * s + tg < NG) {
                    const uint16_t* sp = reinterpret_cast<const uint16_t*>(
                        blk_s + b * BYTES + kv4_scales(NG) + g * 8 * NG + 4 * NG) + GC * s + tg;
                    f0 = __uint_as_float((uint32_t)sp[0] << 16);
                    f1 = __uint_as_float((uint32_t)sp[NG] << 16);
                  }
#pragma unroll
                  for (int e = 0; e < 4; e += ES) w[s][b][e] = x[0][b][e] * (e < 2 ? f0 : f1);
                }
                if (edge) {  // a hidden token's scale may be anything, NaN too
#pragma unroll
                  for (int b = 0; b < NB; ++b)
#pragma unroll
                    for (int e = 0; e < 4; e += ES)
                      if ((hidden >> (4 * b + e)) & 1u) w[s][b][e] = 0.f;
                }
#pragma unroll
                for (int e = 0; e < 2; e += ES) {
                  top[s][e] = fmaxf(w[s][0][e], w[s][0][e + 2]);
#pragma unroll
                  for (int b = 1; b < NB; ++b)
                    top[s][e] = fmax3f(top[s][e], w[s][b][e], w[s][b][e + 2]);
                  grow |= top[s][e] * F[s][e] > 32768.f;
                }
              }
              if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int s = 0; s < SH; ++s)
#pragma unroll
                  for (int e = 0; e < 2; e += ES) {
                    float v = top[s][e];
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
                    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
                    // 2^(5 - exponent of v), from its bits; v is 0 or positive, infinite at most
                    const int ex = __float_as_uint(v) >> 23;
                    const float to = __uint_as_float((uint32_t)min(259 - ex, kTopFExp) << 23);
                    if (to < F[s][e]) {
                      const float f = to / F[s][e];
                      F[s][e] = to;
                      off[s][e] *= f;
#pragma unroll
                      for (int j = GC * s; j < (GC * (s + 1) < NG ? GC * (s + 1) : NG); ++j)
#pragma unroll
                        for (int a = 0; a < 2; ++a) {
                          acc[0][j][a][e] *= f;
                          acc[0][j][a][e + 2] *= f;
                        }
                    }
                  }
              }
#pragma unroll
              for (int b = 0; b < NB; ++b) {
                uint32_t vw[2][NG];
                load_words<NG>(blk_s + b * BYTES + kv4_v_codes(NG) + vl * 4 * NG, vw[0]);
                load_words<NG>(blk_s + b * BYTES + kv4_v_codes(NG) + (32 + vl) * 4 * NG, vw[1]);
#pragma unroll
                for (int s = 0; s < SH; ++s) {
                  const uint32_t b0 =
                      transpose8x8(pack_f16x2(w[s][b][0] * F[s][0], ONE ? 0.f : w[s][b][1] * F[s][1]));
                  const uint32_t b1 =
                      transpose8x8(pack_f16x2(w[s][b][2] * F[s][0], ONE ? 0.f : w[s][b][3] * F[s][1]));
#pragma unroll
                  for (int j = GC * s; j < (GC * (s + 1) < NG ? GC * (s + 1) : NG); ++j) {
                    uint32_t a[4], c8[4];  // tokens 2 t, 2 t + 1 of each half
                    nibbles_f16(vw[0][j], a);
                    nibbles_f16(vw[1][j], c8);
#pragma unroll
                    for (int h = 0; h < 2; ++h)  // feature rows i = 2 h and 2 h + 1 (16 times)
                      mma_f16(acc[0][j][h], a[2 * h], a[2 * h + 1], c8[2 * h], c8[2 * h + 1], b0,
                              b1);
                  }
                  mma_f16(off[s], 0x80088008u, 0x80088008u, 0x80088008u, 0x80088008u, b0, b1);
                }
              }
              if (((rk - r0) & (kFlush - NB)) == kFlush - NB) flush();
            } else {
#pragma unroll
              for (int b = 0; b < NB; ++b) {
                uint32_t vw[2][NG], vs[NG];
                load_words<NG>(blk_s + b * BYTES + kv4_v_codes(NG) + vl * 4 * NG, vw[0]);
                load_words<NG>(blk_s + b * BYTES + kv4_v_codes(NG) + (32 + vl) * 4 * NG, vw[1]);
                load_words<NG>(blk_s + b * BYTES + kv4_scales(NG) + g * 8 * NG + 4 * NG, vs);
#pragma unroll
                for (int j = 0; j < NG; ++j) {
                  const float v0 = scale_of<NG>(vs, 0, j), v1 = scale_of<NG>(vs, 1, j);
                  uint32_t a[8];
#pragma unroll
                  for (int i = 0; i < 4; ++i) {
                    a[2 * i] = minus136(nibbles(vw[0][j], i));
                    a[2 * i + 1] = minus136(nibbles(vw[1][j], i));
                  }
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt) {
                    float y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = x[nt][b][e] * (e < 2 ? v0 : v1);
                    if (edge) {
#pragma unroll
                      for (int e = 0; e < 4; ++e)
                        if ((hidden >> (4 * (nt * NB + b) + e)) & 1u) y[e] = 0.f;
                    }
                    const uint32_t b0 = transpose8x8(pack_bf16x2(y[0], y[1]));
                    const uint32_t b1 = transpose8x8(pack_bf16x2(y[2], y[3]));
                    mma_bf16(acc[nt][j][0], a[0], a[2], a[1], a[3], b0, b1);
                    mma_bf16(acc[nt][j][1], a[4], a[6], a[5], a[7], b0, b1);
                  }
                }
              }
            }
          }
          __syncwarp();  // the stage has been read
          fetch(stage);
          stage = stage + 1 == kStages ? 0 : stage + 1;
        }
        if (!ok) break;

        // ---- the unit's rows, or this warp's part of them
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 4);
            l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 8);
            l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], 16);
          }
        const bool whole = r0 <= 0 && r1 >= u.n;
        // r1 < u.n: the unit goes on in the next warp, and this one is done
        float* part = r1 < u.n ? tail_of(warp) : head_of(warp);
        // features 32 j + 4 g .. + 3 of column cc
        auto put = [&](int cc, int j, float4 o, float lim, float ref, float ll) {
          if (whole) {
            write_out(p, u.b, u.hk, c_first + cc, 32 * j + 4 * g, o, ref, ll);
          } else {
            *reinterpret_cast<float4*>(part + cc * D + 32 * j + 4 * g) = o;
            if (j == 0 && g == 0) {
              part[p.part_cols * D + cc] = lim;
              part[p.part_cols * D + p.part_cols + cc] = ll;
            }
          }
        };
        if constexpr (FEW) {  // a lane holds the groups GC s + tg, columns tc and tc + 1
          flush();
#pragma unroll
          for (int s = 0; s < SH; ++s)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int j = GC * s; j < (GC * (s + 1) < NG ? GC * (s + 1) : NG); ++j)
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  o[k] = __uint_as_float(sel_u32(GC * s + tg == j,
                                                 __float_as_uint(acc[0][j][k >> 1][2 * (k & 1) + e]),
                                                 __float_as_uint(o[k])));
              // 2^24 / F as two factors: together they can leave the range of fp32
              const float f = 1.f / F[s][e];
              if (GC * s + tg < NG && tc + e < ncolv)
                put(tc + e, GC * s + tg,
                    make_float4(o[0] * 16777216.f * f, o[1] * 1048576.f * f,
                                o[2] * 16777216.f * f, o[3] * 1048576.f * f),
                    mlim[0][e], mref[0][e], l[0][e]);
            }
        } else {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int cc = 8 * nt + 2 * t + e;
              if (cc < ncolv)
#pragma unroll
                for (int j = 0; j < NG; ++j)
                  put(cc, j,
                      make_float4(acc[nt][j][0][e], acc[nt][j][0][e + 2], acc[nt][j][1][e],
                                  acc[nt][j][1][e + 2]),
                      mlim[nt][e], mref[nt][e], l[nt][e]);
            }
        }
        if (!whole) {
          if (lane == 0) {
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
        }
      }
      if (u.at + u.n + kUnitCost >= stretch || !next_unit<COLS>(p, u)) break;
    }
    if (!ok) {  // a copy never came: report it, let what is in flight land
      *abort_flag = 1;
      if (lane == 0) atomicOr(&g_dev_error, DEV_ERR_WAIT_TIMEOUT);
      volatile int no_abort = 0;
      for (int i = 0; i < kStages; ++i)
        if ((flying >> i) & 1u) mbar_wait(bars + 8 * i, (phase >> i) & 1u, &no_abort, p.wait_ns);
    }
  }

  // ---- units that span warps: join this CTA's parts
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
    for (int i = tid; i < ncolv * (D / 4); i += kThreads) {
      const int cc = i / (D / 4), f = (i - cc * (D / 4)) * 4;
      Joined a;
      a.clear();
      for (int x = lo; x <= hi; ++x) {
        const float* pp = x == last ? head_of(x) : tail_of(x);
        a.add(pp[p.part_cols * D + cc], pp[p.part_cols * D + p.part_cols + cc],
              *reinterpret_cast<const float4*>(pp + cc * D + f));
      }
      if (first >= 0 && last < kWarps) {
        a.write(p, span, c_first + cc, f);
      } else {
        *reinterpret_cast<float4*>(to + cc * D + f) = a.o;
        if (f == 0) {
          to[p.part_cols * D + cc] = a.m;
          to[p.part_cols * D + p.part_cols + cc] = a.l;
        }
      }
    }
  }
  // ---- units that span CTAs, the one the CTA begins in and the one it ends in:
  // the CTA that arrives last joins them
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
    if (sm.last[k])
      join_ctas<D, COLS>(p, sm.span[k == 0 ? 0 : kWarps], sm.of[k],
                         reinterpret_cast<float*>(sm.ring));
}

template <int NG, int NT, int GC, bool ONE>
iha_status launch_nt(const KvAttnParams& p, int grid, cudaStream_t s) {
  static_assert((sizeof(Smem<NG, NT>) + 1024) * ctas_per_sm(NT) <= 228 * 1024,
                "4-bit attention: the CTAs of an SM do not fit its shared memory");
  static_assert(sizeof(Smem<NG, NT>::ring) >= kThreads * 6 * sizeof(float), "scratch of the join");
  static_assert(sizeof(Smem<NG, NT>::ring) / kWarps >= Part<NG, NT>::FLOATS * sizeof(float),
                "a warp's part of a unit goes into its ring");
  static SmemLimit limit;
  const cudaError_t e = limit.ensure(attn_kv4_kernel<NG, NT, GC, ONE>, (int)sizeof(Smem<NG, NT>));
  if (e != cudaSuccess)
    return fail(IHA_ERR_CUDA, "mha_fwd_kv4 (smem attribute): %s", cudaGetErrorString(e));
  attn_kv4_kernel<NG, NT, GC, ONE><<<grid, kThreads, sizeof(Smem<NG, NT>), s>>>(p);
  return check_launch("mha_fwd_kv4");
}
template <int NG>
iha_status launch(const KvAttnParams& p, int nt, int grid, cudaStream_t s) {
  if (p.ncols == 1) return launch_nt<NG, 1, 4, true>(p, grid, s);
  if (p.ncols == 2) return launch_nt<NG, 1, 4, false>(p, grid, s);
  if (p.ncols <= 4) return launch_nt<NG, 1, 2, false>(p, grid, s);
  return nt == 1 ? launch_nt<NG, 1, 1, false>(p, grid, s) : launch_nt<NG, 2, 1, false>(p, grid, s);
}

}  // namespace
}  // namespace iha

extern "C" {

size_t mha_fwd_kv4_workspace_bytes(int B, int Nq, int Hq, int Hkv, int d) {
  if (B <= 0 || Nq <= 0 || Hkv <= 0 || Hq <= 0 || Hq % Hkv || d <= 0) return 0;
  const int64_t ncols = (int64_t)Nq * (Hq / Hkv);
  const int ctas = iha::kMaxCtas * iha::ctas_per_sm(iha::pick_nt(ncols)) / iha::ctas_per_sm(1);
  return iha::kCounterBytes +
         (size_t)ctas * iha::kCtaParts * iha::part_stride(ncols, d) * sizeof(float);
}

iha_status mha_fwd_kv4(const void* q, const void* cache, const int32_t* block_table,
                       const int32_t* seq_lens, void* o, float* lse_out, void* workspace,
                       size_t workspace_bytes, int B, int Nq, int Hq, int Hkv, int d, int n_pages,
                       int page, int table_width, iha_strides sq, iha_strides so, float scale,
                       iha_mask mask_mode, int window, iha_dtype dt, void* stream) {
  using namespace iha;
  KvAttnParams p;
  int nt, grid;
  const iha_status st = kv_attn_setup(
      "mha_fwd_kv4", p, nt, grid, kv4_check_cache, kv4_page_bytes(page, Hkv, d),
      mha_fwd_kv4_workspace_bytes(B, Nq, Hq, Hkv, d), q, cache, block_table, seq_lens, o, lse_out,
      workspace, workspace_bytes, B, Nq, Hq, Hkv, d, n_pages, page, table_width, sq, so, scale,
      mask_mode, window, dt);
  if (st != IHA_OK) return st;
  p.wait_ns = wait_limit_for_next_launch();
  p.withhold = withhold_for_this_launch() ? 1 : 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  switch (d / kKv4Group) {
    case 1: return launch<1>(p, nt, grid, s);
    case 2: return launch<2>(p, nt, grid, s);
    case 3: return launch<3>(p, nt, grid, s);
    default: return launch<4>(p, nt, grid, s);
  }
}

}  // extern "C"
