// The 8-bit key-value cache: its layout, shared by the kernels that write it, read
// it back, attend over it and copy from it.
//
// 16 positions of a sequence that share a block hold, per key-value head, K and V
// rows of d features (d = 32, 64, 96, 128) as e4m3 codes with one scale 2^e each for
// K and for V: e is the smallest with every |x| <= 448 * 2^e, at least -100.  A power
// of two, so that codes rounded again at another scale lose bits only where they
// become subnormal: rows that are moved or whose block grows keep their values.
//
// Pages hold `page` tokens (a multiple of 16) of every head, K and V together:
//   codes    [head][token / 16] blocks of 32 d bytes, K [16][d] and V [16][d]: a row's
//            16-byte chunks c lie at c ^ swap(row), so that eight rows' chunks of the same
//            c are in different banks (ldmatrix of either, transposed for V, without
//            conflicts).  Rows of 128 features are whole lines: with the tails between
//            the blocks a row alone moved half as much again (rows gathered from
//            32768 x 80 heads: 288 MB read for 168).
//   tails    [head][token / 16] 16 bytes: scale of K, scale of V (fp32), one bit per row of
//            K (low half) and of V whose values were not all finite: it stands for NaN
//            throughout, its codes are 0.  No code is ever NaN, so hidden rows are
//            harmless as operands.
// A page is a multiple of 128 bytes.
#pragma once

#include <cuda_fp16.h>

#include "kv4.cuh"

namespace iha {

constexpr int kKv8Tok = 16;      // tokens of a block
constexpr int kKv8LowestE = -100;  // smallest e
constexpr int kKv8HighestE = 120;  // the largest that finite rows need

__host__ __device__ constexpr int kv8_block_bytes(int d) { return 32 * d; }  // of codes
constexpr int kKv8TailBytes = 16;
// What a row's chunk numbers are XORed with.
__host__ __device__ constexpr int kv8_swap(int d, int row) {
  return d == 128 ? row & 7 : d == 64 ? (row >> 1) & 3 : (row >> 2) & 1;
}

struct alignas(16) Kv8Tail {
  float scale[2];  // of K, of V
  uint32_t nan;    // bit row: K, bit 16 + row: V
  uint32_t unused;
};

// Where a page's blocks and tails are.
struct Kv8Pages {
  int64_t bytes, tails;  // of a page; from its start to its tails
  int bpp;               // blocks of a head in a page
  void set(int page, int heads, int d) {
    bpp = page / kKv8Tok;
    tails = (int64_t)heads * bpp * kv8_block_bytes(d);
    bytes = (tails + (int64_t)heads * bpp * kKv8TailBytes + 127) & ~(int64_t)127;
  }
#if defined(__CUDACC__)
  // Byte offsets (64 bits: a cache can be far longer than 4 GB) of a block, and of its tail.
  __device__ __forceinline__ int64_t block(int page_id, int head, int blk, int d) const {
    return page_id * bytes + (int64_t)(head * bpp + blk) * kv8_block_bytes(d);
  }
  __device__ __forceinline__ int64_t tail(int page_id, int head, int blk) const {
    return page_id * bytes + tails + (int64_t)(head * bpp + blk) * kKv8TailBytes;
  }
#endif
};

#if defined(__CUDACC__)
__device__ __forceinline__ Kv8Tail kv8_tail(const uint8_t* at) {
  const uint4 u = *reinterpret_cast<const uint4*>(at);
  Kv8Tail t;
  t.scale[0] = __uint_as_float(u.x);
  t.scale[1] = __uint_as_float(u.y);
  t.nan = u.z;
  t.unused = 0;
  return t;
}
// e of a scale, within its range whatever the bits (a page that was never written).
__device__ __forceinline__ int kv8_exponent(float scale) {
  return min(max((int)((__float_as_uint(scale) >> 23) & 255u) - 127, kKv8LowestE), kKv8HighestE);
}
__device__ __forceinline__ float kv8_two(int e) {  // 2^e; 0 below fp32's normal numbers
  return e < -126 ? 0.f : __uint_as_float((uint32_t)(127 + e) << 23);
}
// Two codes (low byte first) from fp32, to values as fp16.
__device__ __forceinline__ uint16_t e4m3_pair(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_to_f16(uint16_t c) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
// Four codes times a power of two, rounded again.
__device__ __forceinline__ uint32_t e4m3_rescale(uint32_t w, float f) {
  uint32_t out = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t h = e4m3_to_f16((uint16_t)(w >> (16 * i)));
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&h));
    out |= (uint32_t)e4m3_pair(x.x * f, x.y * f) << (16 * i);
  }
  return out;
}
#endif

// Host checks shared by the cache's entry points.
iha_status kv8_check_cache(const char* name, const void* cache, int n_pages, int page, int Hkv,
                           int d);

#define IHA_KV8_D_SWITCH(d, ...)                              \
  switch (d) {                                                \
    case 32: { constexpr int kD = 32; __VA_ARGS__; } break;   \
    case 64: { constexpr int kD = 64; __VA_ARGS__; } break;   \
    case 96: { constexpr int kD = 96; __VA_ARGS__; } break;   \
    default: { constexpr int kD = 128; __VA_ARGS__; } break;  \
  }

}  // namespace iha
