/*
 * lard_attn.h -- C ABI of liblard_attn: attention operators that stand beside
 * the relation-KL kernels of lard.h, for NVIDIA B200 (sm_100a).
 *
 *   Cross attention: softmax attention of n query rows over the m key rows of
 *   another sequence (an encoder's states), forward and backward; with n = 1
 *   it is the decoding step.
 *   Prefix attention: B sequences that share one long prefix (many questions
 *   about one document); the prefix is read once per key head for the whole
 *   batch, each sequence adds the rows of its own behind it.
 *
 * They keep what the relation-KL kernels keep (lard.h): one log-sum-exp per
 * row, no n x m map.  With Z = tau Q K^T over the keys j that row i may see,
 *   LSE_i = log sum_j exp Z_ij,  P = exp(Z - LSE),  O = P V,
 * and, for an upstream gradient dO,
 *   delta_i = sum_c dO_ic O_ic,  dP = dO V^T,  dZ = P (dP - delta),
 *   dQ = tau dZ K,  dK = tau dZ^T Q,  dV = P^T dO.
 * A row that sees no key has O = 0, LSE = -infinity and no part in any gradient.
 *
 * Conventions for every entry point:
 *   - Tensors are lard_attn_view: element (b, h, i, c) of [B, H, rows, d] lies at
 *     ptr + b * batch + h * head + i * row + c, strides in elements.  Both
 *     [B, H, rows, d] and [B, rows, H, d] tensors, and slices of wider ones,
 *     are views.  ptr is 16-byte aligned and the strides are multiples of 16
 *     bytes, 0 <= stride < 2^40 bytes.  An input's batch or head stride may be 0 (one
 *     block shared by all); an output's elements may not overlap one another.
 *   - Grouped heads: Hq is a multiple of Hkv, query head h reads key head
 *     h / (Hq / Hkv).
 *   - Inputs and outputs are bf16 (LARD_DTYPE_BF16) or fp32 (LARD_DTYPE_FP32),
 *     one type per call; d is 64 or 128.  LSE is fp32, contiguous [B, Hq, n].
 *     Products, softmax statistics and sums are held in fp32; for bf16 the
 *     probabilities (and dZ) are rounded to bf16 where they enter a product, and
 *     delta is formed from the rounded out (see rest); every output is rounded once.
 *   - Lengths (k_len, s_len) are int32 in device memory, so that a captured
 *     graph can be replayed with other lengths; a length outside [0, rows] counts
 *     as the nearer bound.  Key and value rows at or past their sequence's length are not used:
 *     they may hold anything, infinities and NaN included.
 *   - The caller owns every buffer.  The workspace is device memory, 16-byte
 *     aligned, of at least the bytes that the operator's _workspace_bytes gives for the same
 *     sizes; its contents have no meaning before or after the call.  Calls whose work can
 *     overlap on the GPU (two streams, two graphs) need a workspace each.  It may be NULL
 *     where 0 bytes are needed.
 *   - No output may overlap an input, the workspace or another output.  Interleaved
 *     views are recognised where their strides are the same (dK and dV as
 *     the two halves of one [B, m, 2, H, d] buffer); other views are
 *     compared by the address range that they span.
 *   - Errors, streams, devices and bounded waits are as in lard.h; the fault word
 *     of these kernels is read with lard_attn_device_status.
 *   - 1 <= n, m, P, S <= 2^31 - 256 (P or S may be 0 for prefix attention, not
 *     both), Hq / Hkv * n <= 2^31 - 256, B * Hq < 2^30.  Prefix attention takes the
 *     queries of all sequences together: B * Hq / Hkv * n <= 2^31 - 256.
 *   - A launch has at most 2^31 - 1 blocks (a block has the rows, or keys, of one key head
 *     of one sequence: in bf16 256 rows in the forward pass, 128 rows or keys in the
 *     backward pass, in fp32 64; fewer where there are no more), and a forward call
 *     that splits its keys, or has both shared and own keys, joins at most 2^31 - 1
 *     rows (B * Hq * n).  A call that would need more is refused with LARD_ERR_INVALID_ARG.
 */
#ifndef LARD_ATTN_H
#define LARD_ATTN_H

#include "lard.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct lard_attn_view {
    void* ptr;
    long long batch, head, row; /* strides in elements */
} lard_attn_view;

/*
 * Cross attention.
 *   q      in  [B, Hq, n, d].
 *   k, v   in  [B, Hkv, m, d].
 *   k_len  in  [B] or NULL (all m rows): key rows of each sequence.
 *   out    [B, Hq, n, d]: written by the forward pass, read by the backward pass.
 *   rest   [B, Hq, n, d] or ptr NULL; bf16 only (not used for fp32): what rounding
 *          left of out, O - out, itself rounded.  Written by the forward
 *          pass, read by the backward pass, which then forms delta from out + rest.
 *          Without it delta has the error of out's rounding, which adds about
 *          a tenth to the error of dq and dk (2.6e-3 of their norm in place of 2.4e-3).
 *   lse    [B, Hq, n]: written by the forward pass, read by the backward pass.
 *   dout   in  [B, Hq, n, d]: upstream gradient of out (backward pass).
 *   dq     out [B, Hq, n, d], dk, dv out [B, Hkv, m, d] (backward pass): the
 *          gradients, summed over the query heads that share a key head; rows
 *          at or past k_len are written as zeros.
 * Fields that a pass does not use are ignored.
 */
typedef struct lard_cross_attn {
    lard_dtype dtype;
    int B, Hq, Hkv, n, m, d;
    float tau; /* logit scale, finite and > 0 */
    lard_attn_view q, k, v;
    const int* k_len;
    lard_attn_view out;
    float* lse;
    lard_attn_view dout, dq, dk, dv;
    lard_attn_view rest;
} lard_cross_attn;

/* Bytes of workspace of each pass; 0 also for sizes that the call would refuse. */
LARD_API size_t lard_cross_attn_fwd_workspace_bytes(const lard_cross_attn* a);
LARD_API size_t lard_cross_attn_bwd_workspace_bytes(const lard_cross_attn* a);

/* Writes out, lse and, if given, rest.  Deterministic. */
LARD_API lard_status lard_cross_attn_fwd(const lard_cross_attn* a, void* workspace, size_t workspace_bytes,
                                         cudaStream_t stream);

/* Writes dq, dk and dv, given what lard_cross_attn_fwd wrote for the same inputs.  Deterministic. */
LARD_API lard_status lard_cross_attn_bwd(const lard_cross_attn* a, void* workspace, size_t workspace_bytes,
                                         cudaStream_t stream);

/*
 * Prefix attention: the n newest rows of each of B sequences attend to P rows
 * that all sequences share and to their own rows behind those.
 *   q       in  [B, Hq, n, d]: queries of the n newest rows.
 *   kp, vp  in  [Hkv, P, d] (the views' batch stride is not used); ignored if P = 0.
 *   ks, vs  in  [B, Hkv, S, d]: room for S rows of each sequence's own, the
 *               n newest among them; ignored (s_len too) if S = 0.
 *   s_len   in  [B] or NULL (all S rows): rows of its own that each sequence has.
 *               Query i sees every shared row and its sequence's own rows
 *               j <= s_len - n + i (none where that is negative).
 *   out     out [B, Hq, n, d];  lse out [B, Hq, n].
 * A non-finite value in an own row may reach every new row of that sequence.
 * Deterministic.  There is no backward pass (a serving operator).
 */
typedef struct lard_prefix_attn_args {
    lard_dtype dtype;
    int B, Hq, Hkv, n, P, S, d;
    float tau;
    lard_attn_view q, kp, vp, ks, vs;
    const int* s_len;
    lard_attn_view out;
    float* lse;
} lard_prefix_attn_args;

LARD_API size_t lard_prefix_attn_workspace_bytes(const lard_prefix_attn_args* a);
LARD_API lard_status lard_prefix_attn(const lard_prefix_attn_args* a, void* workspace, size_t workspace_bytes,
                                      cudaStream_t stream);

/* lard_device_status (lard.h) for the kernels of this library.  Bits: 0x1-0x4 a role of the
 * forward kernel, 0x10-0x80 a role of the backward kernel, 0x100 an exit wait. */
LARD_API lard_status lard_attn_device_status(cudaStream_t stream, unsigned int* fault_bits);

#ifdef __cplusplus
}
#endif

#endif /* LARD_ATTN_H */
