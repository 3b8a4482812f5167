// The 4-bit key-value cache: its layout, shared by the kernels that write it,
// read it back and attend over it.
//
// A cached row of d features (d = 32 NG) is NG groups of 32 neighbours; group
// j has a bf16 scale s = bf16(max |x| / 7) and codes c = round(x / s), ties to
// even, |c| <= 7, held as the nibble n = c + 8.  It stands for s * c.
//
// Pages hold `page` tokens (a multiple of 16) of every head, K and V together:
//   cache[page id][head][token / 16] = one block of 16 tokens, 576 NG bytes.
// A block is laid out in the order in which the 32 lanes of a warp feed it to
// mma.m16n8k16 (lane = 4 g + t), so the attention loads it with one coalesced
// 4 NG-byte access per lane and plane and unpacks it with shifts and masks:
//   K codes   [token / 8][g = token % 8][t][j]  32-bit words: nibble e is
//             feature 32 j + 8 t + e.  Lane (g, t) owns token rows g and g + 8
//             of the A operand; (w >> 4 i) & 0x000F000F is the feature pair
//             (i, i + 4), and Q's B operand pairs its features the same way.
//   V codes   [token / 8][t = token % 8 / 2][g ^ 2 t][j]  32-bit words: the low
//             half is token 2 t, the high half token 2 t + 1; nibble i of a half
//             is feature 32 j + 4 g + i.  (w >> 4 i) & 0x000F000F is the token
//             pair the transposed A operand (features x tokens) wants.  A pair of
//             tokens is 32 NG contiguous bytes (a row read alone moves twice its
//             bytes, not four times as with t innermost); the XOR keeps the
//             attention's reads from shared memory free of bank conflicts.
//   scales    [g = token % 8][K, V][token / 8][j] bf16: both rows of a token in
//             one 32-byte sector.
#pragma once

#include "common.cuh"

namespace iha {

constexpr int kKv4Tok = 16;    // tokens per block
constexpr int kKv4Group = 32;  // features per scale

// A page or slot index out of range: the access is skipped and flagged.
enum : unsigned { DEV_ERR_CACHE_INDEX = 8u };

// Group maxima below this are stored as zero (their reciprocal scale would
// leave the normal fp32 range).
constexpr float kKv4Tiny = 7.8886090522101181e-31f;  // 2^-100

// Bytes of the whole block and of its planes, for NG groups.
__host__ __device__ constexpr int kv4_block_bytes(int ng) { return 576 * ng; }
__host__ __device__ constexpr int kv4_v_codes(int ng) { return 256 * ng; }
__host__ __device__ constexpr int kv4_scales(int ng) { return 512 * ng; }

// Byte offset inside a block of the K word of token tok (0..15), octet t, group j.
__host__ __device__ constexpr int kv4_k_word(int ng, int tok, int t, int j) {
  return (((tok >> 3) * 32 + (tok & 7) * 4 + t) * ng + j) * 4;
}
// Place of lane (g, t) among the 32 of a half's V words.
__host__ __device__ constexpr int kv4_v_lane(int g, int t) { return t * 8 + (g ^ (2 * t)); }
// ... of the V half-word (4 features 32 j + 4 g ..) of token tok.
__host__ __device__ constexpr int kv4_v_half(int ng, int tok, int g, int j) {
  return kv4_v_codes(ng) +
         (((tok >> 3) * 32 + kv4_v_lane(g, (tok & 7) >> 1)) * ng + j) * 4 + (tok & 1) * 2;
}
// ... of the scale of token tok, group j, of K (v = 0) or V (v = 1).
__host__ __device__ constexpr int kv4_scale(int ng, int v, int tok, int j) {
  return kv4_scales(ng) + ((((tok & 7) * 2 + v) * 2 + (tok >> 3)) * ng + j) * 2;
}

#if defined(__CUDACC__)
// Byte offset of block blk_in_page of `head` in page `page_id` (64 bits: a
// cache can be far longer than 4 GB).
__device__ __forceinline__ int64_t kv4_block_of(int page_id, int blk_in_page, int head, int heads,
                                                int blocks_per_page, int ng) {
  return (((int64_t)page_id * heads + head) * blocks_per_page + blk_in_page) *
         (int64_t)kv4_block_bytes(ng);
}
#endif

// Two strided views of rows of d elements (extents n, strides s in elements, none
// negative; view b starts `delta` elements after view a): does a row of one lie on
// a row of the other?  With self, delta is 0 and a row does not meet itself.  Exact,
// except that layouts that take more than 2^20 steps to tell apart count as meeting.
struct Kv4View {
  int dims;
  int64_t n[4], s[4];
};
bool kv4_views_meet(const Kv4View& a, const Kv4View& b, int64_t delta, int d, bool self);

// Host checks shared by the cache's entry points.
iha_status kv4_check_cache(const char* name, const void* cache, int n_pages, int page, int Hkv,
                           int d);

}  // namespace iha
