// Rotary positions of query and key rows (iha_rope_fwd) and of their gradients
// (iha_rope_bwd).
//
//   (y_a, y_b) = gain (x_a cos - x_b sin, x_b cos + x_a sin),  angle = position w_i
//
// for pair i of the first rot features: (i, i + rot / 2) or (2 i, 2 i + 1); the other
// features are copied.  The backward pass turns the other way.
//
// Angles: a pair's frequency is held as turns per position in 64-bit fixed point,
// turn = w / 2 pi * 2^64 mod 2^64, so position * turn in 64-bit integers is the angle
// in turns modulo 1 for any position, without the loss of a 32-bit product (position
// 2^20 in fp32 is off by 2^-4 radians).  The table is right to its last bit.  Of the product's
// upper 32 bits the nearest quarter of a turn is taken off, the rest goes through sincospif:
// off by about 2^-24 in all.
//
// A thread takes 32 bytes of a row, 8 pairs of bf16 or 4 of fp32, works out their
// sines once and applies them to up to `hg` heads of its token.
//
// Bound by HBM: 32768 tokens x 40 heads of 128, bf16, 671 MB: 103 us, 6.5 TB/s (CTAs of
// 256 threads 110), into the same buffers again 99; half of each head rotated 98, 8192 x 160
// heads 101, 6.6.  Halves off 16 bytes: 50 of 80 features 2.8 to 3.2, 100 of 128 3.9 (pair by
// pair from memory 1.8 and 2.3).
#include <math.h>

#include "kv4.cuh"

namespace iha {
namespace {

constexpr int kMaxPairs = 128;
constexpr int kRopeThreads = 128;
constexpr int kBatch = 4;  // heads whose rows a thread loads at once

struct RopeParams {
  const void *q, *k;
  void *yq, *yk;
  const int32_t* pos;  // null: the place in the sequence
  iha_strides sq, sk, tq, tk;
  FastDiv units, groups, N;  // units of a row, groups of heads of a token, tokens of a sequence
  int items;                 // threads (warps) with work
  int turning;               // units that turn, the rest copy (vectors that hold turned ones)
  int copy_step;             // features between a copying unit's two vectors; 0: it has one
  int Hq, H, hg;             // heads of q, of both, of a group
  int rot;
  float gain, sign;
  uint64_t turn[kMaxPairs];
};

template <typename T>
__device__ __forceinline__ void unpack(uint4 v, float (&f)[16 / sizeof(T)]);
template <>
__device__ __forceinline__ void unpack<__nv_bfloat16>(uint4 v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16lo_to_f32(w[i]);
    f[2 * i + 1] = bf16hi_to_f32(w[i]);
  }
}
template <>
__device__ __forceinline__ void unpack<float>(uint4 v, float (&f)[4]) {
  f[0] = __uint_as_float(v.x);
  f[1] = __uint_as_float(v.y);
  f[2] = __uint_as_float(v.z);
  f[3] = __uint_as_float(v.w);
}
__device__ __forceinline__ uint4 repack(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ uint4 repack(const float (&f)[4]) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                    __float_as_uint(f[3]));
}
// The sine and cosine of a pair at a position, each times its factor.
__device__ __forceinline__ void turn_of(int64_t pos, uint64_t turn, float gain, float sign,
                                        float& sn, float& cs) {
  // q quarters of a turn and a rest of up to an eighth, which fp32 holds to 2^-28 turns
  const uint32_t part = (uint32_t)(((uint64_t)pos * turn) >> 32);
  const uint32_t q = (part + 0x20000000u) >> 30;
  float sr, cr;
  sincospif((float)(int32_t)(part - (q << 30)) * 4.656612873077393e-10f, &sr, &cr);  // 2^-31
  sn = __uint_as_float(__float_as_uint(q & 1u ? cr : sr) ^ (q & 2u) << 30) * sign;
  cs = __uint_as_float(__float_as_uint(q & 1u ? sr : cr) ^ ((q + 1u) & 2u) << 30) * gain;
}
__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void narrow(float* p, float x) { *p = x; }
__device__ __forceinline__ void narrow(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// Rows of q, then of k, of one token.
template <typename T>
struct TokenRows {
  const T *q, *k;
  T *yq, *yk;
  __device__ __forceinline__ TokenRows(const RopeParams& p, int b, int n)
      : q(static_cast<const T*>(p.q) + b * p.sq.b_outer + n * p.sq.seq),
        k(static_cast<const T*>(p.k) + (p.k ? b * p.sk.b_outer + n * p.sk.seq : 0)),
        yq(static_cast<T*>(p.yq) + b * p.tq.b_outer + n * p.tq.seq),
        yk(static_cast<T*>(p.yk) + (p.k ? b * p.tk.b_outer + n * p.tk.seq : 0)) {}
  __device__ __forceinline__ const T* in(const RopeParams& p, int h) const {
    return h < p.Hq ? q + h * p.sq.head : k + (h - p.Hq) * p.sk.head;
  }
  __device__ __forceinline__ T* out(const RopeParams& p, int h) const {
    return h < p.Hq ? yq + h * p.tq.head : yk + (h - p.Hq) * p.tk.head;
  }
};

template <typename T, bool INTER>
__global__ void __launch_bounds__(kRopeThreads)
    rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int V = 16 / sizeof(T);  // features of a vector, pairs of a thread
  __shared__ uint64_t turn[kMaxPairs];
  for (int i = threadIdx.x; i < p.rot / 2; i += kRopeThreads) turn[i] = p.turn[i];
  __syncthreads();
  const int id = blockIdx.x * kRopeThreads + threadIdx.x;
  if (id >= p.items) return;
  const int rest = p.units.div(id), u = id - rest * p.units.d;
  const int tok = p.groups.div(rest), head0 = (rest - tok * p.groups.d) * p.hg;
  const int b = p.N.div(tok), n = tok - b * p.N.d;
  const int head1 = min(head0 + p.hg, p.H);
  const bool turns = u < p.turning;
  // the thread's two vectors in a row
  int at0, at1;
  if (!turns) {
    at0 = p.rot + (u - p.turning) * V;
    at1 = at0 + p.copy_step;
  } else if (INTER) {
    at0 = u * 2 * V;
    at1 = at0 + V;
  } else {
    at0 = u * V;
    at1 = p.rot / 2 + at0;
  }
  float cs[V], sn[V];
  if (turns) {
    const int64_t pos = p.pos ? __ldg(p.pos + tok) : n;
#pragma unroll
    for (int i = 0; i < V; ++i) turn_of(pos, turn[u * V + i], p.gain, p.sign, sn[i], cs[i]);
  }
  const TokenRows<T> rows(p, b, n);
  // all of a batch's loads before its first store (a row turned in place is read and
  // written by the same thread)
#pragma unroll 1
  for (int h0 = head0; h0 < head1; h0 += kBatch) {
    uint4 v[kBatch][2];
#pragma unroll
    for (int j = 0; j < kBatch; ++j)
      if (h0 + j < head1) {
        const T* x = rows.in(p, h0 + j);
        v[j][0] = *reinterpret_cast<const uint4*>(x + at0);
        v[j][1] = *reinterpret_cast<const uint4*>(x + at1);  // (copying one: the same again)
      }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      if (h0 + j >= head1) break;
      T* y = rows.out(p, h0 + j);
      if (!turns) {
        *reinterpret_cast<uint4*>(y + at0) = v[j][0];
        *reinterpret_cast<uint4*>(y + at1) = v[j][1];
        continue;
      }
      float f[2][V], g[2][V];
      unpack<T>(v[j][0], f[0]);
      unpack<T>(v[j][1], f[1]);
#pragma unroll
      for (int i = 0; i < V; ++i) {
        // element i of a pair list: (vector, place) of its two features
        const int va = INTER ? 2 * i / V : 0, ia = INTER ? 2 * i % V : i;
        const int vb = INTER ? va : 1, ib = INTER ? ia + 1 : i;
        const float a = f[va][ia], c = f[vb][ib];
        g[va][ia] = a * cs[i] - c * sn[i];
        g[vb][ib] = c * cs[i] + a * sn[i];
      }
      *reinterpret_cast<uint4*>(y + at0) = repack(g[0]);
      *reinterpret_cast<uint4*>(y + at1) = repack(g[1]);
    }
  }
}

// Pairs whose halves do not start on 16 bytes: a warp takes a token's rows, puts their
// vectors that hold turned features into shared memory, turns pair by pair there and writes
// whole vectors back.
template <typename T, bool INTER>
__global__ void __launch_bounds__(kRopeThreads)
    rope_rows_kernel(const __grid_constant__ RopeParams p) {
  constexpr int V = 16 / sizeof(T), MOST = 2 * kMaxPairs / V;  // vectors that hold turned ones
  constexpr int LANE_PAIRS = kMaxPairs / 32;
  __shared__ uint64_t turn[kMaxPairs];
  __shared__ uint4 held[kRopeThreads / 32][kBatch][MOST];
  for (int i = threadIdx.x; i < p.rot / 2; i += kRopeThreads) turn[i] = p.turn[i];
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int id = blockIdx.x * (kRopeThreads / 32) + warp;
  if (id >= p.items) return;
  const int tok = p.groups.div(id), head0 = (id - tok * p.groups.d) * p.hg;
  const int b = p.N.div(tok), n = tok - b * p.N.d;
  const int head1 = min(head0 + p.hg, p.H);
  float cs[LANE_PAIRS], sn[LANE_PAIRS];
  const int64_t pos = p.pos ? __ldg(p.pos + tok) : n;
#pragma unroll
  for (int i = 0; i < LANE_PAIRS; ++i)
    if (32 * i + lane < p.rot / 2)
      turn_of(pos, turn[32 * i + lane], p.gain, p.sign, sn[i], cs[i]);
  const TokenRows<T> rows(p, b, n);
  const int held_n = p.turning, all_n = p.units.d;  // vectors to hold, of a row
#pragma unroll 1
  for (int h0 = head0; h0 < head1; h0 += kBatch) {
    const int nrows = min(kBatch, head1 - h0);
    for (int i = lane; i < nrows * all_n; i += 32) {
      const int r = p.units.div(i), c = i - r * all_n;
      const uint4 v = reinterpret_cast<const uint4*>(rows.in(p, h0 + r))[c];
      if (c < held_n)
        held[warp][r][c] = v;
      else
        reinterpret_cast<uint4*>(rows.out(p, h0 + r))[c] = v;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < LANE_PAIRS; ++i) {
      const int pair = 32 * i + lane;
      if (pair >= p.rot / 2) break;
      const int at0 = INTER ? 2 * pair : pair, at1 = INTER ? at0 + 1 : pair + p.rot / 2;
      for (int r = 0; r < nrows; ++r) {
        T* x = reinterpret_cast<T*>(held[warp][r]);
        const float a = widen(x[at0]), c = widen(x[at1]);
        narrow(x + at0, a * cs[i] - c * sn[i]);
        narrow(x + at1, c * cs[i] + a * sn[i]);
      }
    }
    __syncwarp();
    for (int i = lane; i < nrows * held_n; i += 32) {
      const int r = i / held_n, c = i - r * held_n;
      reinterpret_cast<uint4*>(rows.out(p, h0 + r))[c] = held[warp][r][c];
    }
    __syncwarp();
  }
}

template <typename T, bool INTER>
void launch(const RopeParams& p, bool vec, unsigned blocks, cudaStream_t s) {
  if (vec)
    rope_kernel<T, INTER><<<blocks, kRopeThreads, 0, s>>>(p);
  else
    rope_rows_kernel<T, INTER><<<blocks, kRopeThreads, 0, s>>>(p);
}

iha_status rotate(const char* name, bool back, const void* q, const void* k,
                  const int32_t* positions, void* yq, void* yk, const iha_rope* rope, int B, int N,
                  int Hq, int Hk, int d, iha_strides sq, iha_strides sk, iha_strides tq,
                  iha_strides tk, iha_dtype dt, void* stream) {
  if (!q || !yq || !rope) return fail(IHA_ERR_INVALID_ARG, "%s: null pointer", name);
  if ((k == nullptr) != (yk == nullptr) || (k == nullptr) != (Hk == 0))
    return fail(IHA_ERR_INVALID_ARG, "%s: k, its output and Hk > 0 go together", name);
  if (B <= 0 || N <= 0 || Hq <= 0 || Hk < 0 || d <= 0)
    return fail(IHA_ERR_INVALID_ARG, "%s: sizes must be positive", name);
  if (dt != IHA_BF16 && dt != IHA_F32) return fail(IHA_ERR_INVALID_ARG, "%s: bad dtype", name);
  if (rope->rot < 2 || rope->rot > 2 * kMaxPairs || (rope->rot & 1) || !(rope->mul > 0.f))
    return fail(IHA_ERR_INVALID_ARG, "%s: rope is not as iha_rope_init leaves it", name);
  if (rope->rot > d)
    return fail(IHA_ERR_INVALID_ARG, "%s: %d rotated features of %d", name, rope->rot, d);
  const int es = dt == IHA_BF16 ? 2 : 4, V = 16 / es;
  if (d % V)
    return fail(IHA_ERR_UNSUPPORTED, "%s: d %d is not a multiple of %d", name, d, V);
  for (iha_strides* t : {&sq, &tq, &sk, &tk}) {  // the stride of an extent of 1 is never used
    const bool isq = t == &sq || t == &tq;
    if (B == 1) t->b_outer = 0;
    if (N == 1) t->seq = 0;
    if ((isq ? Hq : Hk) <= 1) t->head = 0;
    if (!isq && Hk == 0) *t = iha_strides{0, 0, 0, 0};
    if (t->b_outer < 0 || t->seq < 0 || t->head < 0)
      return fail(IHA_ERR_INVALID_ARG, "%s: negative stride", name);
    if (t->b_outer % V || t->seq % V || t->head % V)
      return fail(IHA_ERR_ALIGNMENT, "%s: strides must be multiples of 16 bytes", name);
  }
  if (!aligned16(q) || !aligned16(yq) || !aligned16(k) || !aligned16(yk))
    return fail(IHA_ERR_ALIGNMENT, "%s: tensors must be 16-byte aligned", name);
  if (reinterpret_cast<uintptr_t>(positions) & 3)
    return fail(IHA_ERR_ALIGNMENT, "%s: positions must be 4-byte aligned", name);
  const int64_t toks = (int64_t)B * N;
  if (toks > (1 << 30))
    return fail(IHA_ERR_UNSUPPORTED, "%s: more than 2^30 tokens in one call", name);

  // outputs: rows apart from one another, from the other output and from the inputs,
  // but for a tensor turned in place
  struct Tensor {
    const void* p;
    int H;
    iha_strides s;
  };
  const Tensor in[2] = {{q, Hq, sq}, {k, Hk, sk}}, out[2] = {{yq, Hq, tq}, {yk, Hk, tk}};
  const int nt = k ? 2 : 1;
  auto view = [&](const Tensor& t) {
    return Kv4View{3, {B, N, t.H}, {t.s.b_outer, t.s.seq, t.s.head}};
  };
  auto bytes = [&](const Tensor& t) {
    return ((int64_t)(B - 1) * t.s.b_outer + (int64_t)(N - 1) * t.s.seq +
            (int64_t)(t.H - 1) * t.s.head + d) * es;
  };
  auto meet = [&](const Tensor& a, const Tensor& b) {
    if (!overlaps(a.p, bytes(a), b.p, bytes(b))) return false;
    const int64_t apart = static_cast<const char*>(b.p) - static_cast<const char*>(a.p);
    return kv4_views_meet(view(a), view(b), apart / es, d, false);
  };
  for (int i = 0; i < nt; ++i) {
    const Tensor& o = out[i];
    if ((B > 1 && o.s.b_outer == 0) || (N > 1 && o.s.seq == 0) || (o.H > 1 && o.s.head == 0) ||
        kv4_views_meet(view(o), view(o), 0, d, true))
      return fail(IHA_ERR_INVALID_ARG, "%s: rows of an output overlap one another", name);
    if (positions && overlaps(o.p, bytes(o), positions, toks * 4))
      return fail(IHA_ERR_INVALID_ARG, "%s: an output overlaps positions", name);
    for (int j = 0; j < nt; ++j) {
      const bool in_place = i == j && o.p == in[j].p && o.s.b_outer == in[j].s.b_outer &&
                            o.s.seq == in[j].s.seq && o.s.head == in[j].s.head;
      if (!in_place && meet(o, in[j]))
        return fail(IHA_ERR_INVALID_ARG, "%s: an output overlaps an input it is not in place of",
                    name);
    }
  }
  if (nt == 2 && meet(out[0], out[1]))
    return fail(IHA_ERR_INVALID_ARG, "%s: the outputs overlap one another", name);

  RopeParams p;
  p.q = q;
  p.k = k;
  p.yq = yq;
  p.yk = yk;
  p.pos = positions;
  p.sq = sq;
  p.sk = sk;
  p.tq = tq;
  p.tk = tk;
  p.Hq = Hq;
  p.H = Hq + Hk;
  p.rot = rope->rot;
  p.gain = rope->mul;
  p.sign = back ? -rope->mul : rope->mul;
  for (int i = 0; i < rope->rot / 2; ++i) p.turn[i] = rope->turn[i];
  // vectors where both halves of a turn start on 16 bytes
  const bool vec = rope->rot / 2 % V == 0;
  p.hg = 1;
  p.copy_step = 0;
  const int64_t sms = sm_count();
  int64_t items;
  if (vec) {
    p.turning = rope->rot / 2 / V;
    int copying = (d - rope->rot) / V;
    if (copying % 2 == 0 && copying > 0) {
      copying /= 2;
      p.copy_step = copying * V;
    }
    const int units = p.turning + copying;
    // heads of a thread: its sines cost about as much as four heads' rows, so as many as
    // leave half of the GPU's threads (32768 tokens x 40 heads of 128: one head a thread 222
    // us, 8 110, 16 112; 3003 tokens x 40 heads of 96, fp32: two full waves left 26, half
    // a wave 18)
    while (p.hg < 8 && toks * p.H * units / (2 * p.hg) >= 1024 * sms) p.hg *= 2;
    p.units.set(units);
    items = toks * ((p.H + p.hg - 1) / p.hg) * units;
  } else {  // a warp for some heads of a token; likewise
    p.turning = (rope->rot + V - 1) / V;
    p.units.set(d / V);
    while (p.hg < 16 && toks * p.H / (2 * p.hg) >= 32 * sms) p.hg *= 2;
    items = toks * ((p.H + p.hg - 1) / p.hg);
  }
  if (items > (1 << 30) || d / V > (1 << 20))
    return fail(IHA_ERR_UNSUPPORTED, "%s: too many rows in one call", name);
  p.groups.set((p.H + p.hg - 1) / p.hg);
  p.N.set(N);
  p.items = (int)items;
  const int per = vec ? kRopeThreads : kRopeThreads / 32;  // items of a CTA
  const unsigned blocks = (unsigned)((p.items + per - 1) / per);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dt == IHA_BF16) {
    if (rope->interleaved)
      launch<__nv_bfloat16, true>(p, vec, blocks, s);
    else
      launch<__nv_bfloat16, false>(p, vec, blocks, s);
  } else {
    if (rope->interleaved)
      launch<float, true>(p, vec, blocks, s);
    else
      launch<float, false>(p, vec, blocks, s);
  }
  return check_launch(name);
}

// ---- the table.  A turn is fixed to 2^-64, and far positions take up all of its bits (53 of
// them, a double's, leave 2^-25 turns at position 2^31), so it is worked out on sums of two
// doubles, some 104 bits: Knuth's and Dekker's sums and products without error, a product's
// rest by fma.  (Where a compiler joins a product and a sum, bits only move between hi and lo.)
struct Pair {
  double hi, lo;
};
Pair two_sum(double a, double b) {
  const double s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
Pair operator+(Pair a, Pair b) {
  const Pair s = two_sum(a.hi, b.hi), t = two_sum(a.lo, b.lo);
  const Pair u = two_sum(s.hi, s.lo + t.hi);
  return two_sum(u.hi, u.lo + t.lo);
}
Pair operator-(Pair a, Pair b) { return a + Pair{-b.hi, -b.lo}; }
Pair operator*(Pair a, Pair b) {
  const double p = a.hi * b.hi;
  return two_sum(p, fma(a.hi, b.lo, fma(a.lo, b.hi, fma(a.hi, b.hi, -p))));
}
Pair operator/(Pair a, Pair b) {
  const double q = a.hi / b.hi;
  const Pair r = a - Pair{q, 0.0} * b;
  const double q2 = r.hi / b.hi;
  const Pair r2 = r - Pair{q2, 0.0} * b;
  return two_sum(q, q2) + Pair{r2.hi / b.hi, 0.0};
}
// x^(-1 / n), 1 <= n < 2^7: a double's root and a step of Newton's method; x is brought to
// below 2^n, so that no power leaves its range.
Pair inverse_root(double x, int n) {
  const int k = ilogb(x) / n;
  const double m = ldexp(x, -n * k), y = pow(m, 1.0 / n);
  Pair p = {y, 0.0};  // y^n
  for (int i = 1; i < n; ++i) p = p * Pair{y, 0.0};
  const Pair rest = Pair{m, 0.0} - p;
  const Pair root = two_sum(y, y * (rest.hi / p.hi / n));
  return Pair{ldexp(1.0, -k), 0.0} / root;
}

}  // namespace
}  // namespace iha

extern "C" {

iha_status iha_rope_init(iha_rope* r) {
  using namespace iha;
  const char* name = "iha_rope_init";
  if (!r) return fail(IHA_ERR_INVALID_ARG, "%s: null pointer", name);
  if (r->rot < 2 || (r->rot & 1))
    return fail(IHA_ERR_INVALID_ARG, "%s: rot %d is not an even number above 0", name, r->rot);
  if (r->rot > 2 * kMaxPairs)
    return fail(IHA_ERR_UNSUPPORTED, "%s: more than %d rotated features", name, 2 * kMaxPairs);
  if (r->interleaved != 0 && r->interleaved != 1)
    return fail(IHA_ERR_INVALID_ARG, "%s: interleaved is 0 or 1", name);
  if (!(r->base > 1.0) || !isfinite(r->base))
    return fail(IHA_ERR_INVALID_ARG, "%s: base must be finite and above 1", name);
  if (!(r->gain >= 0.0) || !(r->gain < 1e30))
    return fail(IHA_ERR_INVALID_ARG, "%s: gain must be positive, or 0 for the usual one", name);
  if (r->scaling < IHA_ROPE_NONE || r->scaling > IHA_ROPE_PARTS)
    return fail(IHA_ERR_INVALID_ARG, "%s: bad scaling %d", name, r->scaling);
  const double f = r->factor;
  if (r->scaling != IHA_ROPE_NONE && (!(f >= 1.0) || !(f < 1e30)))
    return fail(IHA_ERR_INVALID_ARG, "%s: factor must be at least 1", name);
  if (r->scaling == IHA_ROPE_BASE && r->rot == 2)
    return fail(IHA_ERR_INVALID_ARG, "%s: a scaled base needs rot > 2", name);
  if (r->scaling == IHA_ROPE_PARTS &&
      (r->trained < 1 || !(r->slow >= 0.0) || !(r->fast > r->slow) || !isfinite(r->fast)))
    return fail(IHA_ERR_INVALID_ARG, "%s: parts needs trained >= 1 and 0 <= slow < fast", name);
  const Pair per_turn = {0x1.45f306dc9c883p-3, -0x1.6b01ec5417056p-57};  // 1 / 2 pi
  const Pair one = {1.0, 0.0}, zero = {0.0, 0.0}, by = {f, 0.0};
  // base^(-2 i / rot), with a scaled base times f^(-2 i / (rot - 2))
  Pair ratio = inverse_root(r->base, r->rot / 2), turns = per_turn;
  if (r->scaling == IHA_ROPE_BASE) ratio = ratio * inverse_root(f, r->rot / 2 - 1);
  for (int i = 0; i < r->rot / 2; ++i, turns = turns * ratio) {
    Pair t = turns;  // per position, below 1 / 6
    if (r->scaling == IHA_ROPE_LINEAR) t = t / by;
    if (r->scaling == IHA_ROPE_PARTS) {
      Pair g = (Pair{(double)r->trained, 0.0} * t - Pair{r->slow, 0.0}) /
               two_sum(r->fast, -r->slow);
      if (g.hi < 0.0) g = zero;
      if (g.hi >= 1.0) g = one;
      t = t * (g + (one - g) / by);
    }
    const double hi = ldexp(t.hi, 64), whole = floor(hi);
    const double rest = floor((hi - whole) + ldexp(t.lo, 64) + 0.5);
    r->turn[i] = (uint64_t)((int64_t)whole + (int64_t)rest);
  }
  r->mul = (float)(r->gain > 0.0 ? r->gain
                                 : r->scaling == IHA_ROPE_PARTS ? 0.1 * log(f) + 1.0 : 1.0);
  if (!(r->mul > 0.f)) return fail(IHA_ERR_INVALID_ARG, "%s: gain is 0 in fp32", name);
  return IHA_OK;
}

iha_status iha_rope_fwd(const void* q, const void* k, const int32_t* positions, void* yq, void* yk,
                        const iha_rope* rope, int B, int N, int Hq, int Hk, int d, iha_strides sq,
                        iha_strides sk, iha_strides syq, iha_strides syk, iha_dtype dt,
                        void* stream) {
  return iha::rotate("iha_rope_fwd", false, q, k, positions, yq, yk, rope, B, N, Hq, Hk, d, sq, sk,
                     syq, syk, dt, stream);
}

iha_status iha_rope_bwd(const void* dyq, const void* dyk, const int32_t* positions, void* dq,
                        void* dk, const iha_rope* rope, int B, int N, int Hq, int Hk, int d,
                        iha_strides sdyq, iha_strides sdyk, iha_strides sdq, iha_strides sdk,
                        iha_dtype dt, void* stream) {
  return iha::rotate("iha_rope_bwd", true, dyq, dyk, positions, dq, dk, rope, B, N, Hq, Hk, d,
                     sdyq, sdyk, sdq, sdk, dt, stream);
}

}  // extern "C"
