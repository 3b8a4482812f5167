/*
 * iha.h — C ABI of the GB300 (sm_103a) library for the Interleaved Head
 * Attention (IHA) attention-layer hot path and Hiera mask-unit attention.
 *
 * Operations and where they are defined:
 *   iha_premix_fwd / iha_premix_bwd_dx / iha_premix_bwd_dw
 *     "IHA-CUDA: Interleaved Head Attention Kernels for Hopper GPUs",
 *     section "Pseudo-Token Mixing (Triton Premix Kernels)": the mix
 *     Out[h,p] = sum_s W[h,p,s] * X[s] at every (batch, position, feature),
 *     its input gradient dX = W^T dY and its weight gradient
 *     dW = sum over (b, n, d) of dY * X^T, with optional fused RoPE.
 *   mha_fwd
 *     same page, sections "Kernel Design" and "FLOP Matching": softmax
 *     attention over the H*P pseudo-heads with a causal sliding window of
 *     W = WSL + 1 keys; "hiera-optim 0.1.0", file
 *     hiera_optim/attention/mask_unit.py (MaskUnitAttentionFast.forward):
 *     unmasked attention inside each mask unit, read in Hiera's
 *     (T outer, num_windows inner) token layout.
 *   mu_gather / mu_scatter
 *     "hiera-optim 0.1.0", README, "optimize(model) does two things", item 2:
 *     boolean mask indexing of the kept mask units replaced by gather and
 *     scatter.
 *
 *   kv4_store / kv4_load / mha_fwd_kv4 / iha_premix_fwd_qkv_at
 *     serving: a paged key-value cache held in 4 bits, the attention of new
 *     tokens over it and the premix of tokens that continue a sequence (no
 *     counterpart in the pages).
 *   iha_rope_fwd / iha_rope_bwd, kv8_append / kv8_load / mha_fwd_kv8 / kv8_evict
 *     rotary positions as operators of their own; the same kind of cache held in
 *     8 bits, and its eviction by the attention weight that keys gather (likewise).
 *
 * Conventions shared by every entry point:
 *   - Pointers named x, y, q, ... are DEVICE pointers owned by the caller.
 *     The library allocates nothing, keeps no pointer after return and never
 *     writes outside the output buffers named in each call.
 *   - Work is enqueued asynchronously on `stream` (a cudaStream_t; NULL is the
 *     legacy default stream).  All argument checks happen on the host before
 *     any launch; a failed check returns an error and launches nothing.
 *   - IHA_ERR_CUDA means a CUDA runtime call failed (details in
 *     iha_last_error()).  Errors that only the GPU can see (an out-of-range
 *     keep index, an internal wait that gave up) set a device error word
 *     that iha_device_error() reads; the offending accesses are skipped.
 *   - Tensors are dense in their last dimension; byte strides of 16-bit
 *     tensors must be multiples of 16 and base pointers 16-byte aligned
 *     (IHA_ERR_ALIGNMENT otherwise).
 */
#ifndef IHA_H_
#define IHA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  IHA_OK = 0,
  IHA_ERR_INVALID_ARG = 1,   /* null pointer, non-positive size, bad enum   */
  IHA_ERR_UNSUPPORTED = 2,   /* valid but outside what the kernels handle   */
  IHA_ERR_ALIGNMENT = 3,     /* base pointer or stride not 16-byte aligned  */
  IHA_ERR_CUDA = 4           /* a CUDA runtime call or launch failed        */
} iha_status;

typedef enum { IHA_F32 = 0, IHA_BF16 = 1 } iha_dtype;

typedef enum {
  IHA_MASK_NONE = 0,           /* every key visible                          */
  IHA_MASK_CAUSAL = 1,         /* key j visible to query i iff j <= i         */
  IHA_MASK_CAUSAL_WINDOW = 2   /* ... and i - j < window (window = WSL + 1)   */
} iha_mask;

/* Element strides of a [B_outer, B_inner, seq, head, d] view; d is dense. */
typedef struct {
  int64_t b_outer;
  int64_t b_inner;
  int64_t seq;
  int64_t head;
} iha_strides;

/*
 * Premix forward ("Pseudo-Token Mixing", forward):
 *   y[b,n,h*P+p,f] = sum_{s<H} w[h,p,s] * x[b,n,s,f]
 * then, if rope != 0, each pseudo-head vector y[b,n,j,:] is rotated by the
 * rotate-half RoPE of position n: for i < d/2, angle = n * rope_base^(-2i/d),
 *   (y_i, y_{i+d/2}) <- (y_i cos - y_{i+d/2} sin, y_{i+d/2} cos + y_i sin).
 *   x  [B, N, H, d]    dtype dt (IHA_BF16 or IHA_F32), dense
 *   w  [H, P, H]       float32, dense
 *   y  [B, N, H*P, d]  dtype dt, dense, must not overlap x or w
 * Accumulation is fp32; bf16 outputs are rounded to nearest even.
 * Requires d % 8 == 0 (bf16) or d % 4 == 0 (f32), H <= 32, H*P <= 128;
 * rope needs d a power of two in [16, 128].
 */
iha_status iha_premix_fwd(const void* x, const float* w, void* y, int B, int N,
                          int H, int P, int d, iha_dtype dt, int rope,
                          float rope_base, void* stream);

/*
 * Premix forward of Q, K and V in one launch ("Pseudo-Token Mixing": one
 * premix per Q, K and V, each with its own weight; the pages fuse the
 * backward's six launches into two, and this fuses the forward's three into
 * one).  Tensor t in (q, k, v) computes exactly what iha_premix_fwd computes
 * for (x_t, w_t, y_t); RoPE (when rope != 0) is applied to q and k only.
 * All nine buffers follow iha_premix_fwd's layout and limits; no output may
 * overlap any input or another output.  Shapes outside the tensor-core
 * kernel run on the CUDA-core kernel: Q, K and V in one launch (with RoPE,
 * Q and K in one and V in a second), on the same stream.
 */
iha_status iha_premix_fwd_qkv(const void* xq, const void* xk, const void* xv,
                              const float* wq, const float* wk, const float* wv,
                              void* yq, void* yk, void* yv, int B, int N, int H, int P,
                              int d, iha_dtype dt, int rope, float rope_base, void* stream);

/*
 * Premix forward of Q, K and V of tokens at given positions, for tokens that
 * continue sequences (a decode step, a chunk of a prompt): exactly
 * iha_premix_fwd_qkv with rope != 0, except that token (b, n) rotates at
 * positions[b * N + n] instead of n.
 *   positions  int32 [B, N] (device), any order; |position| < 2^24 (beyond it
 *              the angles of the bf16 kernel lose accuracy)
 * All other buffers and limits as iha_premix_fwd_qkv.  Few bf16 tokens of d in
 * {64, 128}, 3 * B * N * ceil(H * P / 16) <= 768 (51 tokens of 20 -> 80 heads, 256
 * of 8 -> 16), run on a latency-bound kernel with fp32 products of the fp32
 * weight (last bits may differ from iha_premix_fwd_qkv's); more tokens and other
 * shapes on the same kernels as iha_premix_fwd_qkv, with the same bits.
 */
iha_status iha_premix_fwd_qkv_at(const void* xq, const void* xk, const void* xv,
                                 const float* wq, const float* wk, const float* wv,
                                 const int32_t* positions, void* yq, void* yk, void* yv,
                                 int B, int N, int H, int P, int d, iha_dtype dt,
                                 float rope_base, void* stream);

/*
 * Premix forward of Q, K and V with the interleaved pseudo-token layout of
 * the joint-softmax reading of Interleaved Head Attention ("IHA-CUDA", the
 * "interleaved" head layout and the softmax "joint" across pseudo-heads):
 *   y_t[b, n, p, h, f] = sum_s w_t[h, p, s] * x_t[b, n, s, f]  (+ RoPE at n)
 * i.e. the values of iha_premix_fwd_qkv with rows ordered p * H + h instead
 * of h * P + p.  Viewed as [B, N*P, H, d] (sequence stride H*d, head stride
 * d), it is an H-head sequence of N*P pseudo-tokens, pseudo-token n*P + p,
 * which mha_fwd attends over in place (causal on n*P + p).
 * bf16 only, d in {64, 128}, H <= 32, H*P <= 128; other limits as
 * iha_premix_fwd_qkv.
 */
iha_status iha_premix_fwd_qkv_interleaved(const void* xq, const void* xk, const void* xv,
                                          const float* wq, const float* wk, const float* wv,
                                          void* yq, void* yk, void* yv, int B, int N, int H,
                                          int P, int d, iha_dtype dt, int rope,
                                          float rope_base, void* stream);

/*
 * Rotary positions of query and key rows, for layers whose rotation is not the
 * premix's own: either layout of the pairs, part of a head, frequencies scaled for
 * long contexts, any positions.  Row (b, n, h) at position t = positions[b * N + n]:
 *   (y_a, y_b) = gain * (x_a cos - x_b sin, x_b cos + x_a sin),   angle = t * w_i,
 * for pairs i < rot / 2 of its first rot features: (a, b) = (i, i + rot / 2), or with
 * interleaved (2 i, 2 i + 1).  The other d - rot features are copied.
 * w_i = base^(-2 i / rot), changed by a factor f >= 1 as `scaling` says:
 *   IHA_ROPE_NONE    not at all
 *   IHA_ROPE_LINEAR  w_i / f
 *   IHA_ROPE_BASE    base * f^(rot / (rot - 2)) in the place of base
 *   IHA_ROPE_PARTS   w_i (g + (1 - g) / f), g = (trained w_i / 2 pi - slow) / (fast - slow)
 *                    within [0, 1]: pairs that turn more than `fast` times over the
 *                    trained length keep their frequency, below `slow` times it is w_i / f
 */
typedef enum {
  IHA_ROPE_NONE = 0,
  IHA_ROPE_LINEAR = 1,
  IHA_ROPE_BASE = 2,
  IHA_ROPE_PARTS = 3
} iha_rope_scaling;

typedef struct {
  /* set by the caller before iha_rope_init */
  int32_t rot;         /* rotated features of a head, even, 2 .. 256 */
  int32_t interleaved; /* 0 or 1 */
  int32_t scaling;     /* iha_rope_scaling */
  int32_t trained;     /* PARTS: positions of the trained length */
  double base;         /* > 1, usually 10000 */
  double factor;       /* f */
  double fast, slow;   /* PARTS: 0 <= slow < fast, usually 32 and 1 */
  double gain;         /* 0: 1, with PARTS 0.1 ln f + 1 */
  /* set by iha_rope_init */
  uint64_t turn[128];  /* 2^-64 turns of pair i per position, rounded */
  float mul;           /* the gain */
  int32_t unused;
} iha_rope;

/* Checks the caller's fields of a rope and fills in the others (host only). */
iha_status iha_rope_init(iha_rope* rope);

/*
 * The rotation of q and k in one launch, and of their gradients (which turns the
 * other way, with the same gain):
 *   q, yq      [B, N, Hq, d] views, dtype dt (bf16 or f32), element strides sq, syq
 *              (b_outer, seq, head; b_inner unused), >= 0, multiples of 16 bytes
 *   k, yk      [B, N, Hk, d] views likewise; both NULL with Hk = 0 for q alone
 *   positions  int32 [B, N] dense (device), any values; NULL: row (b, n) is at n
 *   rope       host memory, from iha_rope_init; copied before the call returns
 * yq may be q itself (same pointer and strides: in place), yk may be k; else no row of
 * an output may lie on a row of an input or of another output.
 * d a multiple of 16 bytes, rot <= d.  Angles modulo a turn are within 2^-31 turns at any
 * position, sines and cosines good to about 2^-23, products in fp32.
 */
iha_status iha_rope_fwd(const void* q, const void* k, const int32_t* positions, void* yq,
                        void* yk, const iha_rope* rope, int B, int N, int Hq, int Hk, int d,
                        iha_strides sq, iha_strides sk, iha_strides syq, iha_strides syk,
                        iha_dtype dt, void* stream);
iha_status iha_rope_bwd(const void* dyq, const void* dyk, const int32_t* positions, void* dq,
                        void* dk, const iha_rope* rope, int B, int N, int Hq, int Hk, int d,
                        iha_strides sdyq, iha_strides sdyk, iha_strides sdq, iha_strides sdk,
                        iha_dtype dt, void* stream);

/*
 * Premix input gradient ("Pseudo-Token Mixing", backward, dX = W^T dY):
 *   dx[b,n,s,f] = sum_{h,p} w[h,p,s] * g[b,n,h*P+p,f]
 * with g = dy, or g = R_n^T dy (inverse rotation) when rope != 0.
 *   dy [B, N, H*P, d]  dtype dt;  w [H, P, H] float32;  dx [B, N, H, d] dtype dt.
 * Same shape limits as iha_premix_fwd.
 */
iha_status iha_premix_bwd_dx(const void* dy, const float* w, void* dx, int B,
                             int N, int H, int P, int d, iha_dtype dt,
                             int rope, float rope_base, void* stream);

/*
 * Premix weight gradient ("Pseudo-Token Mixing", backward, dW = sum dY X^T):
 *   dw[h,p,s] = sum_{b,n,f} g[b,n,h*P+p,f] * x[b,n,s,f]   (g as in dX)
 *   dy [B, N, H*P, d] dtype dt;  x [B, N, H, d] dtype dt;
 *   dw [H, P, H] float32, OVERWRITTEN (zeroed on `stream` first).
 * Partial sums are reduced inside each block, then added with one float
 * atomic per element per block, so the last bits depend on block order.
 */
iha_status iha_premix_bwd_dw(const void* dy, const void* x, float* dw, int B,
                             int N, int H, int P, int d, iha_dtype dt,
                             int rope, float rope_base, void* stream);

/*
 * Premix backward, both gradients in one pass over dY ("Pseudo-Token Mixing",
 * backward): dx as iha_premix_bwd_dx and dw as iha_premix_bwd_dw, from one
 * read of dy (and x).  Algorithmic traffic per token: dY + X + dX instead of
 * 2 dY + X + dX for the two separate calls.
 *   dy [B, N, H*P, d], x [B, N, H, d], dx [B, N, H, d] (dtype dt);
 *   w [H, P, H] float32;  dw [H, P, H] float32, OVERWRITTEN.
 * Same shape limits as iha_premix_fwd; outputs must not overlap any input.
 */
iha_status iha_premix_bwd(const void* dy, const void* x, const float* w, void* dx,
                          float* dw, int B, int N, int H, int P, int d,
                          iha_dtype dt, int rope, float rope_base, void* stream);

/*
 * Premix backward of Q, K and V in one launch ("Pseudo-Token Mixing":
 * "Backward ... all three Q/K/V in a single launch each", six launches to
 * two).  Tensor t in (q, k, v) computes exactly what iha_premix_bwd computes
 * for (dy_t, x_t, w_t) into (dx_t, dw_t); RoPE (when rope != 0) applies to q
 * and k only.  Every buffer follows iha_premix_bwd's layout and limits; the
 * three dw are OVERWRITTEN (one small zeroing launch precedes the backward
 * launch on `stream`); no output may overlap any input or another output.
 * Shapes outside the tensor-core kernel run as three iha_premix_bwd calls.
 */
iha_status iha_premix_bwd_qkv(const void* dyq, const void* dyk, const void* dyv,
                              const void* xq, const void* xk, const void* xv,
                              const float* wq, const float* wk, const float* wv,
                              void* dxq, void* dxk, void* dxv,
                              float* dwq, float* dwk, float* dwv, int B, int N,
                              int H, int P, int d, iha_dtype dt, int rope,
                              float rope_base, void* stream);

/*
 * Multi-head softmax attention forward over Hh heads ("Kernel Design",
 * "FLOP Matching"; MaskUnitAttentionFast.forward):
 *   o[i] = sum_j softmax_j(scale * <q_i, k_j> | visible(i, j)) * v_j
 *   lse[i] = ln sum_{visible j} exp(scale * <q_i, k_j>)
 * Views: q, o are [B_outer, B_inner, Nq, Hh, d]; k, v are
 * [B_outer, B_inner, Nk, Hh, d]; element strides in sq, sk, sv, so.  With
 * B_inner = num mask units and seq stride = num_units * row, Hiera's
 * (T outer, units inner) layout is read in place.
 *   scale     <= 0 selects 1/sqrt(d)
 *   mask_mode IHA_MASK_NONE | IHA_MASK_CAUSAL | IHA_MASK_CAUSAL_WINDOW
 *             (causal masks require Nq == Nk)
 *   window    keys per query including the diagonal (W = WSL + 1), >= 1 for
 *             IHA_MASK_CAUSAL_WINDOW, ignored otherwise
 *   lse_out   nullable; float32 [B_outer, B_inner, Hh, Nq] dense
 * bf16: tensor-core kernel (tcgen05, TMEM accumulators, TMA tiles), fp32
 * softmax; needs 8 <= d <= 128, d % 8 == 0.  f32: CUDA-core kernel, fp32
 * throughout, d <= 128.
 */
iha_status mha_fwd(const void* q, const void* k, const void* v, void* o,
                   float* lse_out, int B_outer, int B_inner, int Hh, int Nq,
                   int Nk, int d, iha_strides sq, iha_strides sk,
                   iha_strides sv, iha_strides so, float scale,
                   iha_mask mask_mode, int window, iha_dtype dt, void* stream);

/*
 * Mask-unit attention with pooled queries (Hiera's q_pool; "hiera-optim
 * 0.1.0", hiera_optim/attention/mask_unit.py, MaskUnitAttentionFast.forward
 * with q_stride > 1): per (b_outer, b_inner, head) unit of T tokens, the
 * query rows are max-pooled over q_stride blocks of Tq = T / q_stride rows
 * (the block index is the slow axis),
 *   qp[t] = max_i q[i * Tq + t]          (elementwise, i < q_stride)
 * and attend, unmasked, over all T keys:
 *   o[t] = sum_j softmax_j(scale * <qp_t, k_j>) v_j,  lse[t] as mha_fwd.
 * The pooling happens inside the kernel, on the Q tile as it arrives; the
 * pooled queries are never written to memory.
 *   q, k, v   bf16 [B_outer, B_inner, T, Hh, d] views (strides sq, sk, sv)
 *   o         bf16 [B_outer, B_inner, Tq, Hh, d] view (strides so)
 *   lse_out   nullable; float32 [B_outer, B_inner, Hh, Tq] dense
 *   scale     <= 0 selects 1/sqrt(d)
 * Needs T <= 64, q_stride dividing T, d <= 128 and d % 8 == 0; alignment as
 * mha_fwd.  q_stride = 1 is mha_fwd's unmasked short-sequence attention.
 */
iha_status mha_fwd_qpool(const void* q, const void* k, const void* v, void* o,
                         float* lse_out, int B_outer, int B_inner, int Hh, int T,
                         int d, int q_stride, iha_strides sq, iha_strides sk,
                         iha_strides sv, iha_strides so, float scale,
                         iha_dtype dt, void* stream);

/*
 * Attention backward over Hh heads ("Repository Structure": preprocess,
 * backward, postprocess; "End-to-End Training Benchmark": the training step):
 * with P = softmax(scale Q K^T | mask) recomputed from lse and dO the
 * gradient of O = P V,
 *   D_i = sum_f dO_if O_if,   dS = P o (dO V^T - D)
 *   dq = scale dS K,   dk = scale dS^T Q,   dv = P^T dO.
 *   q, k, v, o, dout   bf16 [B, N, Hh, d] dense (o, lse: the forward's outputs)
 *   lse                float32 [B, Hh, N] (natural log, scale included)
 *   dq, dk, dv         bf16 [B, N, Hh, d] dense, written; must not overlap
 *                      each other, the inputs or the workspace
 *   workspace          device scratch of at least mha_bwd_workspace_bytes()
 *                      bytes, 256-byte aligned, owned by the caller: an fp32
 *                      dQ accumulator and per-row D and lse * log2(e); its
 *                      contents on entry do not matter and on return are
 *                      unspecified
 *   scale <= 0 selects 1/sqrt(d); mask_mode / window as mha_fwd (Nq = Nk = N).
 * Needs bf16, d % 16 == 0, d <= 128.  Three launches on `stream`; dq gathers
 * contributions with fp32 atomics, so its last bits depend on their order.
 */
size_t mha_bwd_workspace_bytes(int B, int Hh, int N, int d);
iha_status mha_bwd(const void* q, const void* k, const void* v, const void* o,
                   const void* dout, const float* lse, void* dq, void* dk, void* dv,
                   void* workspace, size_t workspace_bytes, int B, int Hh, int N,
                   int d, float scale, iha_mask mask_mode, int window,
                   iha_dtype dt, void* stream);

/*
 * Attention backward without any allocation.  The pages have no counterpart:
 * this entry point exists for callers that cannot hand the library a device
 * buffer and cannot call cudaMalloc themselves, for example a plugin inside a
 * host program whose own allocator owns all device memory, or a code path
 * that must not call cudaMalloc because it can synchronize the device.
 * Same arguments and results as mha_bwd, minus the workspace: the scratch
 * (fp32 dQ accumulator, per-row D and lse * log2(e)) lives in a 32 MiB array
 * built into the library, which every GPU that loads the library keeps for
 * the life of the process.
 *   - Problems whose scratch exceeds 32 MiB (mha_bwd_workspace_bytes > 32 MiB,
 *     e.g. B = 1, N = 4096, Hh = 8, d = 128 fits) are rejected with
 *     IHA_ERR_UNSUPPORTED before anything is launched; use mha_bwd.
 *   - The first call on a device looks up the array's device address (once
 *     per device, with that device current); make that first call before
 *     any stream capture on the device.
 *   - Every call shares the one array and it keeps the last call's contents;
 *     each call rewrites all of it that it reads, but calls that overlap on
 *     the GPU (other streams, other host threads) race on it: serialize them.
 */
iha_status mha_bwd_noalloc(const void* q, const void* k, const void* v,
                           const void* o, const void* dout, const float* lse,
                           void* dq, void* dk, void* dv, int B, int Hh, int N,
                           int d, float scale, iha_mask mask_mode, int window,
                           iha_dtype dt, void* stream);

/*
 * The 4-bit key-value cache.  A cached row (one token and head of K or of V,
 * d features) is d / 32 groups of 32 neighbouring features.  A value counts as
 * its bf16 rounding; a group has a bf16 scale s = bf16(max |x| / 7) and codes
 * c = round(x / s), ties to even, -7 <= c <= 7, and stands for s * c.  A group
 * whose maximum is below 2^-100 is held as zeros; one that holds a NaN or an
 * infinity reads back as NaN throughout.  36 bytes per 32 features of K and V
 * together (4.5 bits a value).
 *
 * The cache is n_pages pages of kv4_page_bytes() bytes, dense, 16-byte
 * aligned; a page holds `page` tokens (a multiple of 16) of all Hkv heads, K
 * and V.  A slot is a token's place: page id * page + offset in the page.  The
 * order of the bytes inside a page belongs to the library.  Pages need no
 * initial value.  d is 32, 64, 96 or 128; n_pages * page < 2^31.
 */
size_t kv4_page_bytes(int page, int Hkv, int d);  /* 0 for sizes it cannot hold */

/*
 * Quantise rows into the cache as they are written:
 *   cache[slots[b, n]] <- (k[b, n, :, :], v[b, n, :, :])
 *   k, v   [B_outer, B_inner, N, Hkv, d] views, dtype dt (bf16 or f32), element
 *          strides sk, sv (>= 0, multiples of 16 bytes; 0 repeats a row)
 *   slots  int32 [B_outer, B_inner, N] dense; -1 is padding, its row is not
 *          stored; any other value outside the cache is skipped and flagged
 *          (iha_device_error)
 * Slots that occur twice in one call race: the slot is left with a mixture.
 * Every byte of the cache outside the named slots keeps its value.
 */
iha_status kv4_store(const void* k, const void* v, const int32_t* slots, void* cache,
                     int B_outer, int B_inner, int N, int n_pages, int page, int Hkv, int d,
                     iha_strides sk, iha_strides sv, iha_dtype dt, void* stream);

/*
 * Read rows back: (k, v)[b, n, :, :] <- cache[slots[b, n]], s * c exactly in
 * f32 or rounded to bf16 (nearest even).  Slot -1, and a slot outside the
 * cache (also flagged), gives a row of zeros.  A slot may occur any number of
 * times.  Arguments as kv4_store; no row of k or v may lie on another row of
 * either (one row between others is fine: slices of one tensor).
 */
iha_status kv4_load(const void* cache, const int32_t* slots, void* k, void* v, int B_outer,
                    int B_inner, int N, int n_pages, int page, int Hkv, int d, iha_strides sk,
                    iha_strides sv, iha_dtype dt, void* stream);

/*
 * Softmax attention of Nq new tokens of each of B sequences over the 4-bit
 * cache: single-token decode (Nq = 1), several tokens at once (speculative
 * tokens, the P pseudo-tokens of the interleaved layout, short chunks).
 *   o[b, t, h] = sum_j softmax_j(scale <q[b, t, h], k_j>) v_j   over visible j,
 * k_j, v_j the values the cache stands for at key j of sequence b, head
 * h / (Hq / Hkv).  Sequence b has seq_lens[b] keys, the new tokens' own among
 * them; key j is in page block_table[b, j / page].  New token t sits at position
 * i = seq_lens[b] - Nq + t:
 *   IHA_MASK_NONE           every key of the sequence is visible
 *   IHA_MASK_CAUSAL         j <= i
 *   IHA_MASK_CAUSAL_WINDOW  j <= i and i - j < window
 * A row without visible keys (an empty sequence, i < 0) gives o = 0 and
 * lse = -inf.  What hidden keys hold, NaN too, has no influence.
 *   q, o         bf16 [B, Nq, Hq, d] views, element strides sq, so (b_outer,
 *                seq, head; b_inner unused), >= 0, multiples of 8; no row of o
 *                may lie on another
 *   cache        as kv4_store; block_table int32 [B, table_width] dense, only
 *                entries of pages with visible keys are read; seq_lens int32
 *                [B].  A page id outside the cache counts as hidden keys, a
 *                length outside [0, table_width * page] is clamped; both are
 *                flagged (iha_device_error).
 *   lse_out      nullable; float32 [B, Hq, Nq] dense, natural log, with scale
 *   workspace    device scratch of mha_fwd_kv4_workspace_bytes() bytes, 256-byte
 *                aligned, its first 4096 bytes ZERO-FILLED once before its first
 *                use (and again after device error 2; what the rest holds does
 *                not matter); every call leaves it ready for the
 *                next, of any shape that fits it.  Calls that may run at the
 *                same time (other streams, graphs replayed together) need a
 *                workspace each.
 *   scale <= 0 selects 1/sqrt(d); at most 1e30, and |q| * scale below 2^117 (beyond
 *   it a score's factor leaves fp32)
 * Accuracy: scores, sums and O are held in fp32.  A score is off by at most
 * scale 2^-13 sum over groups of (largest scale of K) (sum |q|), since codes enter
 * as c + 8; features of q below 2^-28 of its row's largest lose bits.  The products
 * p s with V's scales are rounded: up to 4 rows a key head (Nq * Hq / Hkv) to fp16
 * (2^-11 of a term, and the offset adds 2^-11 of sum p s), more rows to bf16 (2^-8 of
 * a term, as mha_fwd does).  o is rounded to bf16.
 * Hq a multiple of Hkv (at most 2048 times), Nq * Hq / Hkv <= 2^20, B and
 * table_width * page <= 2^30, d in {32, 64, 96, 128}, bf16.  No length is read on
 * the host, so a captured call replays with new seq_lens and block_table.  The
 * result does not depend on timing (no atomics on values).
 */
size_t mha_fwd_kv4_workspace_bytes(int B, int Nq, int Hq, int Hkv, int d);
iha_status mha_fwd_kv4(const void* q, const void* cache, const int32_t* block_table,
                       const int32_t* seq_lens, void* o, float* lse_out, void* workspace,
                       size_t workspace_bytes, int B, int Nq, int Hq, int Hkv, int d,
                       int n_pages, int page, int table_width, iha_strides sq, iha_strides so,
                       float scale, iha_mask mask_mode, int window, iha_dtype dt, void* stream);

/*
 * The 8-bit key-value cache.  16 consecutive positions of a sequence (a block) hold, for
 * each key-value head, K rows and V rows of d features as e4m3 codes c (8 bits: 4
 * of exponent, 3 of fraction) with one scale s = 2^e for the block's K and one for its
 * V: e is the smallest with every |x| <= 448 * 2^e, at least -100, and c = x / s rounded
 * to nearest even.  A value stands for s * c.  A row (one token and head, of K or
 * of V) that holds a NaN or an infinity stands for NaN throughout, and has no part in s.
 * 2 d + 1 bytes per token and head (a page is rounded up to 128 bytes).
 *
 * The cache is n_pages pages of kv8_page_bytes() bytes, dense, 16-byte aligned; a page
 * holds `page` tokens (a multiple of 16) of all Hkv heads, K and V.  Key j of sequence
 * b is in page block_table[b, j / page]; a slot is page id * page + offset.  The order
 * of the bytes inside a page belongs to the library.  Pages need no initial value.
 * d is 32, 64, 96 or 128; n_pages * page < 2^31.
 */
size_t kv8_page_bytes(int page, int Hkv, int d);  /* 0 for sizes it cannot hold */

/*
 * Add rows to the ends of sequences: sequence b has seq_lens[b] keys once they are
 * added, and row (b, n) of k and v is its key seq_lens[b] - N + n.  Of the N rows the
 * last counts[b] are added (all N if counts is NULL); rows of keys before the first
 * are padding.
 *   k, v         [B, N, Hkv, d] views, dtype dt (bf16 or f32), element strides sk, sv
 *                (b_outer, seq, head; b_inner unused), >= 0, multiples of 16 bytes
 *   block_table  int32 [B, table_width] dense, only entries of pages that get rows are read
 *   seq_lens     int32 [B], counts int32 [B] or NULL.  A length outside [0, table_width *
 *                page], a count outside [0, N] is clamped, a page id outside the cache is
 *                skipped; all are flagged (iha_device_error).
 * A block that has keys before its first new row keeps them: its scales become the
 * larger of what they were and what the new rows need, and where one grows the
 * codes that are there are rounded again (exact but for codes that become subnormal).
 * A scale never falls while its block goes on: where a length goes back (drafted tokens that
 * were rejected) and rows are added again, the block keeps the scale that the rejected rows
 * made necessary, and small values of its other rows stay as coarse as that made them.
 * (Such keys are those of earlier calls: in a page that was never written a sequence
 * starts at a multiple of 16.)
 * A block whose first row is new starts afresh, its rows behind the last key become
 * zeros.  Every other byte of the cache keeps its value.  Blocks that two sequences of
 * a call share race.
 */
iha_status kv8_append(const void* k, const void* v, const int32_t* block_table,
                      const int32_t* seq_lens, const int32_t* counts, void* cache, int B, int N,
                      int n_pages, int page, int table_width, int Hkv, int d, iha_strides sk,
                      iha_strides sv, iha_dtype dt, void* stream);

/*
 * Read rows back by their slots, s * c exactly in f32 or bf16 (infinite where it is 2^128:
 * values from 1.9375 * 2^127 on are rounded to that); arguments, padding and checks as
 * kv4_load.
 */
iha_status kv8_load(const void* cache, const int32_t* slots, void* k, void* v, int B_outer,
                    int B_inner, int N, int n_pages, int page, int Hkv, int d, iha_strides sk,
                    iha_strides sv, iha_dtype dt, void* stream);

/*
 * Softmax attention of Nq new tokens of each of B sequences over the 8-bit cache:
 * arguments, masks, lengths, limits and results as mha_fwd_kv4, and
 *   weights, weights_out   both NULL, or float32 [B, Hkv, table_width * page] dense: the
 *                attention weight that each key has gathered,
 *       weights_out[b, h, j] = weights[b, h, j] + sum over t and the query heads of h of
 *                              softmax_j(scale <q[b, t, .], k_j>),
 *                where key j is visible, else weights[b, h, j].  They may be the same
 *                array.  Needs Nq * Hq / Hkv <= 64; new keys usually start at 0
 *                (also where they take the places of rejected ones, whose weight stays).
 *                A call that gave up (device error 2) leaves weights_out unwritten.
 *   workspace    of mha_fwd_kv8_workspace_bytes() bytes, weight_keys = table_width * page
 *                for a call with weights, else 0; zeroed and shared like mha_fwd_kv4's
 *                (one workspace serves calls of both, one after the other)
 * Accuracy: scores, sums, weights and O are held in fp32, codes enter exactly, q with its
 * 8-bit mantissas (features below 2^-28 of a row's largest lose bits); p times V's scale
 * is rounded to fp16, 2^-11 of a term.  o is rounded to bf16.  The weights of a row add up
 * to 1 within about 2^-17, whatever the scores.  |q| * |k| * scale has to stay within fp32.  The result does not depend on timing.
 */
size_t mha_fwd_kv8_workspace_bytes(int B, int Nq, int Hq, int Hkv, int d, int weight_keys);
iha_status mha_fwd_kv8(const void* q, const void* cache, const int32_t* block_table,
                       const int32_t* seq_lens, void* o, float* lse_out, const float* weights,
                       float* weights_out, void* workspace, size_t workspace_bytes, int B, int Nq,
                       int Hq, int Hkv, int d, int n_pages, int page, int table_width,
                       iha_strides sq, iha_strides so, float scale, iha_mask mask_mode, int window,
                       iha_dtype dt, void* stream);

/*
 * Eviction: shorten sequences to the keys that matter, head by head.  Of a sequence of
 * n = seq_lens[b] > keep keys each head keeps its last `recent` and, of the others, the
 * keep - recent of the largest weight (of equal ones the first; NaN counts as -inf); a
 * sequence of up to keep keys is kept whole.  Kept rows are copied in the order of their
 * positions to positions 0, 1, ... of pages dest_table[b, .]; a block's scales there are the
 * largest that its rows come with, codes of other blocks are rounded again (exact but for
 * codes that become subnormal).  Rows behind the last key of a block become zeros.
 *   block_table  int32 [B, table_width], seq_lens int32 [B] (clamped and flagged as above)
 *   weights      float32 [B, Hkv, table_width * page] dense
 *   dest_table   int32 [B, dest_width]: pages that no sequence of the call reads and
 *                that differ from one another (not checked; sources may be shared)
 *   new_lens     int32 [B], written: min(n, keep)
 *   kept         int32 [B, Hkv, keep], written: positions of the kept keys, then -1
 *   weights_out  nullable; float32 [B, Hkv, dest_width * page], written: their weights
 *                (-0 perhaps as 0), then 0
 * 0 <= recent <= keep <= 2^30, dest_width * page >= min(keep, table_width * page).  Afterwards
 * keys sit at other distances than their tokens: attend with IHA_MASK_CAUSAL or
 * IHA_MASK_NONE.  A page id outside the cache leaves its rows zero or unwritten (flagged).
 */
iha_status kv8_evict(void* cache, const int32_t* block_table, const int32_t* seq_lens,
                     const float* weights, const int32_t* dest_table, int32_t* new_lens,
                     int32_t* kept, float* weights_out, int B, int n_pages, int page,
                     int table_width, int dest_width, int Hkv, int d, int keep, int recent,
                     void* stream);

/*
 * Mask-unit gather (README item 2, x[mask] -> gather):
 *   out[b,k,t,:] = x[b, tok(keep[b,k], t), :]
 * where the grid is row-major [grid_h, grid_w], mask units are mu_h x mu_w
 * (unit u = (u / (grid_w/mu_w), u % (grid_w/mu_w))), t = ty*mu_w + tx, and
 *   tok(u, t) = (uy*mu_h + ty) * grid_w + ux*mu_w + tx.
 *   x    [B, grid_h*grid_w, C] elements of elem_bytes bytes, dense
 *   keep [B, n_keep] int32 unit ids in [0, units); out-of-range ids are
 *        skipped on the GPU and flagged in iha_device_error()
 *   out  [B, n_keep, mu_h*mu_w, C]
 * Bit-exact byte copy.  Requires grid_h % mu_h == 0, grid_w % mu_w == 0.
 */
iha_status mu_gather(const void* x, const int32_t* keep, void* out, int B,
                     int grid_h, int grid_w, int mu_h, int mu_w, int n_keep,
                     int C, int elem_bytes, void* stream);

/*
 * Mask-unit scatter (README item 2, x_dec[mask] = ... -> scatter), in place:
 *   x[b, tok(keep[b,k], t), :] = src[b,k,t,:]; other tokens untouched.
 * Same shapes and rules as mu_gather; duplicate ids within a sample race.
 */
iha_status mu_scatter(const void* src, const int32_t* keep, void* x, int B,
                      int grid_h, int grid_w, int mu_h, int mu_w, int n_keep,
                      int C, int elem_bytes, void* stream);

/*
 * Hiera stage-1 attention step in one pass: gather, mask-unit attention and
 * scatter ("hiera-optim 0.1.0": README item 2 and MaskUnitAttentionFast.forward;
 * the qkv and proj layers around the attention are not on this path, so
 * Q = K = V = the unit's tokens).  For every kept unit (b, keep[b,k]):
 *   canvas[b, tok(u, t), :] = sum_t' softmax_t'(scale x_t . x_t') x_t'
 * with x_t = x[b, tok(u, t), :], t, t' over the unit's mu_h*mu_w tokens, and
 * tok() as for mu_gather; every other canvas token is left untouched.  It
 * equals mu_gather -> mha_fwd (mask none) -> mu_scatter without the
 * gathered units ever being written to memory.
 *   x      [B, grid_h*grid_w, C] bf16, dense, 16-byte aligned
 *   keep   [B, n_keep] int32 unit ids (out-of-range ids: unit skipped,
 *          iha_device_error() flagged)
 *   canvas [B, grid_h*grid_w, C] bf16, must not overlap x or keep
 * Requires mu_h*mu_w <= 64, C % 8 == 0, C <= 128, grid_h % mu_h == 0,
 * grid_w % mu_w == 0, n_keep <= units; scale <= 0 means C^-1/2.
 */
iha_status mu_attention_fused(const void* x, const int32_t* keep, void* canvas, int B,
                              int grid_h, int grid_w, int mu_h, int mu_w, int n_keep,
                              int C, float scale, iha_dtype dt, void* stream);

/*
 * Test hook for the failure path; never needed in normal use.  Arms the next
 * bf16 mha_fwd, mha_fwd_kv4 or mha_fwd_kv8 launch made on the calling host thread (one shot)
 * so that CTA 0 withholds the load of its first V tile (the caches' attentions: the
 * completion of its first blocks' copy) and every wait of that launch
 * gives up after limit_us microseconds (1 .. 1e6) instead of the normal 4 s.
 * The launch then takes its abort path: the waiting role raises the block's
 * abort flag, the others unwind, copies in flight land, the MMAs drain,
 * tensor memory is released, and the kernel returns with device error 2
 * (iha_device_error); rows that CTA 0 had a part in are left unwritten, and so is all of
 * mha_fwd_kv8's weights_out.  The GPU context stays usable and the next launch runs
 * normally (caches: once its workspace is zeroed again).
 * IHA_ERR_INVALID_ARG for a limit out of range.
 */
iha_status iha_test_fail_next_wait(int limit_us);

/* Static description of a status code. */
const char* iha_status_string(iha_status status);

/* Detail of the last error returned on the calling host thread ("" if none). */
const char* iha_last_error(void);

/*
 * Device error word of the current device: 0 if no kernel has flagged an
 * error, else a bitwise OR of codes (1 = out-of-range keep index, 2 = a
 * bounded internal wait gave up, 4 = a kernel found its dynamic shared memory
 * not 1024-byte aligned and did nothing, 8 = a slot, page id, length or count
 * outside the 4-bit or 8-bit cache).  Synchronises the device; clears the word if clear != 0.
 * Returns -1 if the word cannot be read.
 */
int iha_device_error(int clear);

#ifdef __cplusplus
}
#endif

#endif /* IHA_H_ */
