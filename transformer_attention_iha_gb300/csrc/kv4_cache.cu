// The 4-bit key-value cache: rows quantised as they are written (kv4_store)
// and read back (kv4_load).  Layout and format: kv4.cuh.
//
// Both are byte movers.  Writing a token and head of d features reads 2 d
// values (4 d bytes of bf16) and writes d + d / 8 bytes; reading back moves
// the same bytes the other way.
//
// Store: a thread owns 8 neighbouring features of K and of V (the four threads
// of a group of 32 find its maximum with two shuffles), a half-warp a token, a
// warp two tokens of the call next to each other.  Where these go to an even
// slot and the next (a prompt), the halves exchange their V codes, so that V is
// written in whole words like K.
//
// Rounding x / s without a division per value: y = x * (1 / s) is off by at
// most 2^-19 (|y| < 7.1, a reciprocal good to an ulp), and x / s of a bf16 x
// and a bf16 s is either exactly half-way between two codes or at least 1 / 512
// away from it (2 x and (2 k + 1) s are 8-bit integers times powers of two, so
// they differ by at least the smaller unit or not at all).  So y is first
// rounded to a multiple of 2^-14 by adding 776 in the same FMA (776 = 768 + 8
// also shifts the code to its nibble), which puts half-way cases exactly
// half-way, and then to an integer, ties to even, by adding 1.5 * 2^23; the low
// byte of the sum is the nibble.  Likewise bf16(top / 7) is bf16(top * fl(1/7)):
// top / 7 of an 8-bit mantissa stays 2^-12 away from every bf16 tie.
//
// Load: eight threads a row, each with half of a K octet's words (whole lines
// over the row) and one g of V.  bf16 output: codes as bf16 (128 + n) - 136,
// exact, times s in one rounding multiply; f32: s * c, exact.
//
// Both are bound by HBM.  8192 tokens x 80 heads of 128, bf16, in order, 430 MB:
// store 72 us (6.0 TB/s; the quantiser's arithmetic keeps the issue slots 69 per
// cent busy), load 66 us (6.6 TB/s).  16384 rows read in random order: 163 us, 5.3
// TB/s of what is asked for and 6 of what moves (a V row alone moves its
// partner's bytes too).
#include "kv4.cuh"

namespace iha {
namespace {

IHA_DEVICE_ERROR_WORD(kv4_cache)

// n / d for 0 <= n < 2^31 by multiplication: inv = ceil(2^64 / d) is too large
// by less than d / 2^64 of itself, so the product by less than 1 / d.
struct FastDiv {
  uint64_t inv;
  int d;
  __host__ void set(int x) {
    d = x;
    inv = x > 1 ? ~0ull / (unsigned)x + 1 : 0;
  }
  __device__ __forceinline__ int div(int n) const {
    return d == 1 ? n : (int)__umul64hi((uint64_t)(unsigned)n, inv);
  }
};

struct Kv4Geom {
  FastDiv N, Bi, page, units;  // tokens of a batch row; inner batch; page; head units of a warp
  int toks, H, n_units, blocks_per_page;
  int n_slots;  // n_pages * page
};

// Where token i of the call lies in a strided view.
__device__ __forceinline__ int64_t view_of(const Kv4Geom& g, const iha_strides& s, int i) {
  const int b = g.N.div(i), n = i - b * g.N.d, bo = g.Bi.div(b), bi = b - bo * g.Bi.d;
  return bo * s.b_outer + bi * s.b_inner + n * s.seq;
}

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
  const float s = __bfloat162float(__float2bfloat16_rn(top * (1.f / 7.f)));
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  uint32_t r[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 x = make_float2(bf16lo_to_f32(v[i]), bf16hi_to_f32(v[i]));
    x = __ffma2_rn(x, make_float2(inv, inv), make_float2(776.f, 776.f));
    x = __fadd2_rn(x, make_float2(12582912.f, 12582912.f));
    r[2 * i] = __float_as_uint(x.x);
    r[2 * i + 1] = __float_as_uint(x.y);
  }
  const uint32_t even = __byte_perm(__byte_perm(r[0], r[2], 0x0040),
                                    __byte_perm(r[4], r[6], 0x0040), 0x5410);
  const uint32_t odd = __byte_perm(__byte_perm(r[1], r[3], 0x0040),
                                   __byte_perm(r[5], r[7], 0x0040), 0x5410);
  uint32_t word = even | (odd << 4);
  scale_bits = __float_as_uint(s) >> 16;
  if (m >= 0x7F80u || top < kKv4Tiny) {  // the same in the group's lanes
    word = 0x88888888u;
    scale_bits = m >= 0x7F80u ? 0x7FC0u : 0u;
  }
  return word;
}

// A warp: two tokens, UN head units of 16 / (lanes of a row) heads each.  All
// rows of a thread are on their way before the first is quantised.
template <typename T, int NG, int UN>
__global__ void __launch_bounds__(256)
    kv4_store_kernel(const T* __restrict__ k, const T* __restrict__ v,
                     const int32_t* __restrict__ slots, uint8_t* __restrict__ cache, Kv4Geom g,
                     iha_strides sk, iha_strides sv) {
  constexpr int LPR = NG == 3 ? 16 : 4 * NG, HPW = 16 / LPR;  // lanes of a row, heads of a unit
  const int lane = threadIdx.x & 31;
  const int id = blockIdx.x * 8 + (threadIdx.x >> 5);  // (token pair, head units)
  const int pair = g.units.div(id), unit = id - pair * g.n_units;
  const int tok = 2 * pair + (lane >> 4), head0 = unit * UN * HPW + (lane & 15) / LPR;
  const int o = (lane & 15) % LPR;  // octet of the row
  const bool live = tok < g.toks && o < 4 * NG;
  const int slot = live ? __ldg(slots + tok) : -1;
  const bool in = slot >= 0 && slot < g.n_slots;
  if (!in && slot != -1) atomicOr(&g_dev_error, DEV_ERR_CACHE_INDEX);
  uint32_t xk[UN][4], xv[UN][4];
  {
    const int b = g.N.div(tok), n = tok - b * g.N.d, bo = g.Bi.div(b), bi = b - bo * g.Bi.d;
    const T* pk = k + bo * sk.b_outer + bi * sk.b_inner + n * sk.seq + head0 * sk.head + o * 8;
    const T* pv = v + bo * sv.b_outer + bi * sv.b_inner + n * sv.seq + head0 * sv.head + o * 8;
#pragma unroll
    for (int u = 0; u < UN; ++u) {
#pragma unroll
      for (int i = 0; i < 4; ++i) xk[u][i] = xv[u][i] = 0;
      if (in && head0 + u * HPW < g.H) {
        load8<T>(pk, xk[u]);
        load8<T>(pv, xv[u]);
      }
      pk += HPW * sk.head;
      pv += HPW * sv.head;
    }
  }
  // the partner's token lies in the other half of this token's words?
  const int other = __shfl_xor_sync(0xffffffffu, slot, 16);
  const bool paired = in && other == (slot ^ 1);
  const bool odd = slot & 1;
  const int pg = in ? g.page.div(slot) : 0, off = in ? slot - pg * g.page.d : 0;
  const int tk = off % kKv4Tok, j = o >> 2, t = o & 3;
  uint8_t* blk = cache + kv4_block_of(pg, off / kKv4Tok, head0, g.H, g.blocks_per_page, NG);
  const int64_t next = (int64_t)HPW * g.blocks_per_page * kv4_block_bytes(NG);
#pragma unroll
  for (int u = 0; u < UN; ++u, blk += next) {
    uint32_t ks, vs;
    const uint32_t kw = quantise8(xk[u], ks), vw = quantise8(xv[u], vs);
    // of the words of features 4 (2 t) .. and 4 (2 t + 1) .., the even slot's lane
    // writes the first, the odd slot's the second
    const uint32_t got = __shfl_xor_sync(0xffffffffu, odd ? vw : vw >> 16, 16);
    if (in && head0 + u * HPW < g.H) {
      *reinterpret_cast<uint32_t*>(blk + kv4_k_word(NG, tk, t, j)) = kw;
      if (paired) {
        const uint32_t w = odd ? __byte_perm(got, vw, 0x7610) : __byte_perm(vw, got, 0x5410);
        *reinterpret_cast<uint32_t*>(blk + kv4_v_half(NG, tk & ~1, 2 * t + (odd ? 1 : 0), j)) = w;
      } else {
        *reinterpret_cast<uint16_t*>(blk + kv4_v_half(NG, tk, 2 * t, j)) = (uint16_t)vw;
        *reinterpret_cast<uint16_t*>(blk + kv4_v_half(NG, tk, 2 * t + 1, j)) = (uint16_t)(vw >> 16);
      }
      if (t < 2)
        *reinterpret_cast<uint16_t*>(blk + kv4_scale(NG, t, tk, j)) = (uint16_t)(t == 0 ? ks : vs);
    }
  }
}

// Nibbles 0, 1 (low, high half) of 4-bit fields in the low halves' order -> values.
__device__ __forceinline__ uint32_t scaled_pair(uint32_t nib, uint32_t s2) {
  uint32_t x = nib | 0x43004300u;  // bf16 128 + n, exact
  const uint32_t o = 0x43084308u;  // 136
  __nv_bfloat162 v = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&x),
                             *reinterpret_cast<const __nv_bfloat162*>(&o));
  v = __hmul2(v, *reinterpret_cast<__nv_bfloat162*>(&s2));
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ float scaled(uint32_t nib, float s) {
  return s * (__uint_as_float(nib | 0x4B000000u) - 8388616.f);  // 2^23 + n - (2^23 + 8)
}

// 8 features of a K word, 4 of a V half-word (low 16 bits), times the scale.
__device__ __forceinline__ void write_k(__nv_bfloat16* p, uint32_t w, uint32_t sc) {
  const uint32_t s2 = sc | (sc << 16);
  uint32_t v[4];  // features (i, i + 4)
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = scaled_pair((w >> (4 * i)) & 0x000F000Fu, s2);
  *reinterpret_cast<uint4*>(p) =
      make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410),
                 __byte_perm(v[0], v[1], 0x7632), __byte_perm(v[2], v[3], 0x7632));
}
__device__ __forceinline__ void write_v(__nv_bfloat16* p, uint32_t h, uint32_t sc) {
  const uint32_t s2 = sc | (sc << 16), hi = h >> 8;
  *reinterpret_cast<uint2*>(p) = make_uint2(scaled_pair((h | (h << 12)) & 0x000F000Fu, s2),
                                            scaled_pair((hi | (hi << 12)) & 0x000F000Fu, s2));
}
__device__ __forceinline__ void write_k(float* p, uint32_t w, uint32_t sc) {
  const float s = __uint_as_float(sc << 16);
#pragma unroll
  for (int q = 0; q < 2; ++q, w >>= 16)
    reinterpret_cast<float4*>(p)[q] =
        make_float4(scaled(w & 15u, s), scaled((w >> 4) & 15u, s), scaled((w >> 8) & 15u, s),
                    scaled((w >> 12) & 15u, s));
}
__device__ __forceinline__ void write_v(float* p, uint32_t h, uint32_t sc) {
  const float s = __uint_as_float(sc << 16);
  *reinterpret_cast<float4*>(p) =
      make_float4(scaled(h & 15u, s), scaled((h >> 4) & 15u, s), scaled((h >> 8) & 15u, s),
                  scaled((h >> 12) & 15u, s));
}

// Eight threads a row of a token and head.
template <typename T, int NG>
__global__ void __launch_bounds__(256)
    kv4_load_kernel(const uint8_t* __restrict__ cache, const int32_t* __restrict__ slots,
                    T* __restrict__ k, T* __restrict__ v, Kv4Geom g, iha_strides sk,
                    iha_strides sv) {
  constexpr int HALF = (NG + 1) / 2;  // K words of a thread
  const int64_t row64 = (int64_t)blockIdx.x * 32 + (threadIdx.x >> 3);
  if (row64 >= (int64_t)g.toks * g.H) return;
  const int row = (int)row64, i = threadIdx.x & 7;
  const int tok = g.units.div(row), head = row - tok * g.H;
  const int slot = __ldg(slots + tok);
  const bool in = slot >= 0 && slot < g.n_slots;
  if (!in && slot != -1) atomicOr(&g_dev_error, DEV_ERR_CACHE_INDEX);
  const int t = i >> 1, j0 = (i & 1) * HALF;
  uint32_t kw[HALF], vh[NG], ks[HALF], vs[NG];
#pragma unroll
  for (int q = 0; q < HALF; ++q) kw[q] = ks[q] = 0;
#pragma unroll
  for (int j = 0; j < NG; ++j) vh[j] = vs[j] = 0;
  if (in) {
    const int pg = g.page.div(slot), off = slot - pg * g.page.d, tk = off % kKv4Tok;
    const uint8_t* blk =
        cache + kv4_block_of(pg, off / kKv4Tok, head, g.H, g.blocks_per_page, NG);
    const uint8_t* vp = blk + kv4_v_half(NG, tk & ~1, i, 0);  // words of the token and its partner
    const int sh = (tk & 1) * 16;
    if constexpr (NG == 4) {
      const uint2 a = *reinterpret_cast<const uint2*>(blk + kv4_k_word(NG, tk, t, j0));
      const uint4 b = *reinterpret_cast<const uint4*>(vp);
      const uint32_t c = *reinterpret_cast<const uint32_t*>(blk + kv4_scale(NG, 0, tk, j0));
      const uint2 e = *reinterpret_cast<const uint2*>(blk + kv4_scale(NG, 1, tk, 0));
      kw[0] = a.x, kw[1] = a.y;
      vh[0] = b.x, vh[1] = b.y, vh[2] = b.z, vh[3] = b.w;
      ks[0] = c & 0xFFFFu, ks[1] = c >> 16;
      vs[0] = e.x & 0xFFFFu, vs[1] = e.x >> 16, vs[2] = e.y & 0xFFFFu, vs[3] = e.y >> 16;
    } else {
#pragma unroll
      for (int q = 0; q < HALF; ++q)
        if (j0 + q < NG) {
          kw[q] = *reinterpret_cast<const uint32_t*>(blk + kv4_k_word(NG, tk, t, j0 + q));
          ks[q] = *reinterpret_cast<const uint16_t*>(blk + kv4_scale(NG, 0, tk, j0 + q));
        }
#pragma unroll
      for (int j = 0; j < NG; ++j) {
        vh[j] = reinterpret_cast<const uint32_t*>(vp)[j];
        vs[j] = *reinterpret_cast<const uint16_t*>(blk + kv4_scale(NG, 1, tk, j));
      }
    }
#pragma unroll
    for (int j = 0; j < NG; ++j) vh[j] = (vh[j] >> sh) & 0xFFFFu;
  }
  T* pk = k + view_of(g, sk, tok) + head * sk.head;
  T* pv = v + view_of(g, sv, tok) + head * sv.head;
#pragma unroll
  for (int q = 0; q < HALF; ++q)
    if (j0 + q < NG) write_k(pk + 32 * (j0 + q) + 8 * t, kw[q], ks[q]);
#pragma unroll
  for (int j = 0; j < NG; ++j) write_v(pv + 32 * j + 4 * i, vh[j], vs[j]);
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

// Coefficients lo .. hi of a stride; the least and the most that this one and the
// smaller ones reach.
struct Step {
  int64_t s, lo, hi, least, most;
};

// Is there a choice of coefficients with |at + sum c s| < d?  Steps in falling order
// of their strides, so each level has few coefficients that the rest can still undo.
bool reaches(const Step* t, int n, int64_t at, int d, int& budget) {
  if (--budget < 0) return true;
  if (n == 0) return at < d && at > -d;
  const int64_t least = n > 1 ? t[1].least : 0, most = n > 1 ? t[1].most : 0;
  // at + c s + [least, most] has to meet (-d, d)
  const int64_t a = 1 - d - most - at, b = d - 1 - least - at;
  int64_t c0 = a / t->s + (a > 0 && a % t->s != 0), c1 = b / t->s - (b < 0 && b % t->s != 0);
  if (c0 < t->lo) c0 = t->lo;
  if (c1 > t->hi) c1 = t->hi;
  for (int64_t c = c0; c <= c1; ++c)
    if (reaches(t + 1, n - 1, at + c * t->s, d, budget)) return true;
  return false;
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

// Head units of a warp.  Few rows: one, for the most warps.  Many bf16 rows: four,
// which spreads the address arithmetic over them (8192 tokens x 80 heads of 128:
// 72 against 101 us, 5.96 TB/s).  f32 rows carry twice the bytes a value and are
// bound by them with one (8192 x 40: 60 us, 6.3 TB/s, against 70 with four).
constexpr int kStoreUnits = 4;
constexpr int64_t kStoreMany = 32768;  // rows (a token and head)

template <typename T, int NG>
void launch_store(int un, unsigned blocks, cudaStream_t s, const void* k, const void* v,
                  const int32_t* slots, uint8_t* cache, const Kv4Geom& g, iha_strides sk,
                  iha_strides sv) {
  const T* tk = static_cast<const T*>(k);
  const T* tv = static_cast<const T*>(v);
  if constexpr (sizeof(T) == 2) {
    if (un > 1) {
      kv4_store_kernel<T, NG, kStoreUnits><<<blocks, 256, 0, s>>>(tk, tv, slots, cache, g, sk, sv);
      return;
    }
  }
  kv4_store_kernel<T, NG, 1><<<blocks, 256, 0, s>>>(tk, tv, slots, cache, g, sk, sv);
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
  if (toks > INT32_MAX - 1 || rows > INT32_MAX)
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
    if (overlaps(k, bk, slots, toks * 4) || overlaps(v, bv, slots, toks * 4))
      return fail(IHA_ERR_INVALID_ARG, "%s: an output overlaps another tensor", name);
    for (const iha_strides* t : {&sk, &sv})
      if ((B_outer > 1 && t->b_outer == 0) || (B_inner > 1 && t->b_inner == 0) ||
          (N > 1 && t->seq == 0) || (Hkv > 1 && t->head == 0))
        return fail(IHA_ERR_INVALID_ARG, "%s: an output repeats rows (stride 0)", name);
    const Kv4View wk = {4, {B_outer, B_inner, N, Hkv}, {sk.b_outer, sk.b_inner, sk.seq, sk.head}};
    const Kv4View wv = {4, {B_outer, B_inner, N, Hkv}, {sv.b_outer, sv.b_inner, sv.seq, sv.head}};
    if (kv4_views_meet(wk, wk, 0, d, true) || kv4_views_meet(wv, wv, 0, d, true))
      return fail(IHA_ERR_INVALID_ARG, "%s: rows of an output overlap one another", name);
    const int64_t apart = static_cast<const char*>(v) - static_cast<const char*>(k);
    if (overlaps(k, bk, v, bv) && kv4_views_meet(wk, wv, apart / es, d, false))
      return fail(IHA_ERR_INVALID_ARG, "%s: the outputs overlap one another", name);
  }
  const int ng = d / kKv4Group;
  const int heads_of_warp = ng == 3 ? 1 : 4 / ng;
  Kv4Geom g;
  g.N.set(N);
  g.Bi.set(B_inner);
  g.page.set(page);
  g.toks = (int)toks;
  g.H = Hkv;
  g.blocks_per_page = page / kKv4Tok;
  g.n_slots = n_pages * page;
  const int un = store && dt == IHA_BF16 && rows >= kStoreMany ? kStoreUnits : 1;
  g.n_units = store ? (Hkv + heads_of_warp * un - 1) / (heads_of_warp * un) : Hkv;
  g.units.set(g.n_units);
  // store: 8 warps a CTA, a warp per token pair and head unit; load: 32 rows a CTA
  const int64_t blocks = store ? ((toks + 1) / 2 * g.n_units + 7) / 8 : (rows + 31) / 32;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  uint8_t* c = static_cast<uint8_t*>(const_cast<void*>(cache));
  IHA_NG_SWITCH(ng, {
    if (store) {
      if (dt == IHA_BF16)
        launch_store<__nv_bfloat16, kNG>(un, (unsigned)blocks, s, k, v, slots, c, g, sk, sv);
      else
        launch_store<float, kNG>(un, (unsigned)blocks, s, k, v, slots, c, g, sk, sv);
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

bool kv4_views_meet(const Kv4View& a, const Kv4View& b, int64_t delta, int d, bool self) {
  Step t[8];
  int n = 0;
  auto add = [&](int64_t s, int64_t lo, int64_t hi) {  // kept in falling order of s
    int i = 0;
    while (i < n && t[i].s > s) ++i;
    if (i < n && t[i].s == s) {
      t[i].lo += lo;
      t[i].hi += hi;
      return;
    }
    for (int k = n++; k > i; --k) t[k] = t[k - 1];
    t[i].s = s;
    t[i].lo = lo;
    t[i].hi = hi;
  };
  auto sums = [&](int last) {
    int64_t least = 0, most = 0;
    for (int i = n - 1; i >= last; --i) {
      t[i].least = least += t[i].lo * t[i].s;
      t[i].most = most += t[i].hi * t[i].s;
    }
  };
  int budget = 1 << 20;
  if (self) {
    bool zero = false;
    for (int i = 0; i < a.dims; ++i)
      if (a.n[i] > 1) {
        if (a.s[i] == 0) zero = true;
        for (int k = 0; k < n; ++k)
          if (t[k].s == a.s[i]) zero = true;  // rows (1, 0) and (0, 1) are one
        add(a.s[i], -(a.n[i] - 1), a.n[i] - 1);
      }
    if (zero) return true;
    bool nested = true;  // each stride steps over all that the smaller ones reach
    int64_t reach = d;
    for (int i = n - 1; i >= 0; --i) {
      nested = nested && t[i].s >= reach;
      reach += t[i].hi * t[i].s;
    }
    if (nested) return false;
    for (int i = 0; i < n; ++i) {  // two rows that differ in t[i] and smaller strides only
      t[i].lo = 1;
      sums(i);
      if (reaches(t + i, n - i, 0, d, budget)) return true;
    }
    return false;
  }
  for (int i = 0; i < a.dims; ++i)
    if (a.n[i] > 1 && a.s[i] > 0) add(a.s[i], -(a.n[i] - 1), 0);
  for (int i = 0; i < b.dims; ++i)
    if (b.n[i] > 1 && b.s[i] > 0) add(b.s[i], 0, b.n[i] - 1);
  sums(0);
  return reaches(t, n, delta, d, budget);
}

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
