/*
 * nvfp4_ffn.h - dense feed-forward layers beside the NVFP4 and FP8 ones of nvfp4.h, in the same library:
 * the 16-bit gated block with its gradients, products of 8-bit integers, and the clipping of gradients.
 * Pointers, streams, statuses and dev_status are those of nvfp4.h; every call takes its sizes from its own comment.
 */
#ifndef NVFP4_FFN_H_
#define NVFP4_FFN_H_

#include "nvfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Gated feed-forward block on 16-bit tensors: both projections, the activation and the product
 *   g = x Wg^T,  u = x Wu^T,  h = act(g) u
 * in one kernel, summed in fp32; act(g) = g sigma(p(g)) of the fp32 sums, p = g (NVFP4_SILU) or
 * 2 sqrt(2/pi) (g + 0.044715 g^3) (NVFP4_GELU_TANH: gelu in its tanh form). h is rounded once.
 *   x          device [M, K], bf16 or fp16 (type NVFP4_BF16 / NVFP4_F16), rows ldx elements apart
 *   w_gate, w_up  device [I, K], of the same type, rows ld_gate and ld_up apart (the halves of one
 *              [2 I, K] tensor, for instance)
 *   h          [M, I] written, rows ldh apart
 *   gate, up   fp32 [M, I] contiguous, 32-byte aligned, written: g and u as they are summed, for the backward call;
 *              or both NULL
 *   workspace  nvfp4_gated_ffn_workspace_bytes(M, I, K) bytes, 16-byte aligned (NULL where that is 0)
 * I, K and the row strides are positive multiples of 8, pointers 16-byte aligned, I and K at most 2^24. h, gate, up and the
 * workspace share no byte with each other or with an operand: NVFP4_ERR_INVALID_ARG (columns of one buffer beside each
 * other are fine). A NaN or an infinity stays in its token's row. dev_status as for nvfp4_gemm.
 */
enum { NVFP4_SILU = 0, NVFP4_GELU_TANH = 1 };
size_t nvfp4_gated_ffn_workspace_bytes(int64_t M, int64_t I, int64_t K);
int nvfp4_gated_ffn(const uint16_t* x, int64_t ldx, const uint16_t* w_gate, int64_t ld_gate, const uint16_t* w_up,
                    int64_t ld_up, int32_t type, int32_t activation, uint16_t* h, int64_t ldh, float* gate, float* up,
                    int64_t M, int64_t I, int64_t K, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                    void* stream);

/*
 * Its gradients, from the forward call's gate and up and the gradient dh of h:
 *   dg = dh u act'(g),  du = dh act(g);  dx = dg Wg + du Wu,  dWg = dg^T x,  dWu = du^T x
 * dg and du are rounded to the type (the tensor cores read them), the sums are fp32, the results are
 * rounded once. With fp16 a dg or du beyond 65,504 is infinite, and with it what it is summed into, and one below 2^-25 is
 * zero: dh is scaled as for any fp16 backward pass.
 *   gate, up   device fp32 [M, I] contiguous;  dh [M, I], rows lddh apart
 *   dx         [M, K] contiguous, written, or NULL: not wanted (w_gate and w_up may then be NULL)
 *   dw_gate, dw_up  [I, K] contiguous, written, or NULL each (x may be NULL when both are). M == 0 writes zeros.
 *   workspace  nvfp4_gated_ffn_backward_workspace_bytes(M, I, K) bytes, 256-byte aligned
 * No result may share memory with another, with the workspace or with an operand, nor the workspace with an operand:
 * NVFP4_ERR_INVALID_ARG. (Between rows that lie apart there may be other tensors.)
 * The weights' gradients sum over all M rows: a NaN in a row of x, gate, up or dh reaches all that it
 * meets, so padding rows must hold finite values (and dh zeros).
 */
size_t nvfp4_gated_ffn_backward_workspace_bytes(int64_t M, int64_t I, int64_t K);
int nvfp4_gated_ffn_backward(const uint16_t* x, int64_t ldx, const uint16_t* w_gate, int64_t ld_gate, const uint16_t* w_up,
                             int64_t ld_up, const float* gate, const float* up, const uint16_t* dh, int64_t lddh,
                             int32_t type, int32_t activation, uint16_t* dx, uint16_t* dw_gate, uint16_t* dw_up, int64_t M,
                             int64_t I, int64_t K, void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream);

/*
 * 8-bit integers with a scale for each row (token or output channel): value = code * scale.
 *   s = amax_row (1/127) (1 for a row of zeros),  code = rn(x (127 (1/amax_row))), ties to even, -127..127,
 * every step, 1/127 and 1/amax_row too, one IEEE fp32 operation (rows with amax below 2^-100 are first multiplied by 2^100). A row that holds
 * an infinity or NaN gets codes 0 and scale NaN: what is made of it is NaN.
 *   x     device [M, K], bf16 or fp16 (type), rows ldx elements apart (a multiple of 8), 16-byte aligned
 *   q, s  int8 [M, K], 16-byte aligned, and fp32 [M], written. K % 16 == 0 (K == 0: scales of 1). They share no memory
 *         with each other or with x: NVFP4_ERR_INVALID_ARG.
 */
int nvfp4_int8_quantize(const uint16_t* x, int64_t ldx, int32_t type, int64_t M, int64_t K, int8_t* q, float* s, void* stream);

/*
 * y[m, n] = sa[m] sb[n] sum_k a[m, k] b[n, k]: the sum is exact, converted once to fp32, times sa, times sb (each
 * one fp32 operation), and rounded once to y's type.
 *   a, sa   int8 codes [M, K] and fp32 scales [M] (tokens);  b, sb  codes [N, K] and scales [N] (channels);
 *           any codes, -128 included
 *   y       [M, N] row-major, bf16, fp16 or fp32 (y_type), 16-byte aligned (a, b and the workspace too)
 *   workspace  nvfp4_int8_gemm_workspace_bytes(M, N, K) bytes (NULL where that is 0)
 * K % 16 == 0, 16 <= K <= 131,056 (the sums fit 32 bits); any M >= 0, N >= 1. y and the workspace share no memory with
 * each other or with an operand: NVFP4_ERR_INVALID_ARG. dev_status as for nvfp4_gemm (calls of up to 8 tokens wait for
 * nothing and never write it).
 */
size_t nvfp4_int8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K);
int nvfp4_int8_gemm(const int8_t* a, const float* sa, const int8_t* b, const float* sb, void* y, int32_t y_type, int64_t M,
                    int64_t N, int64_t K, void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream);

/*
 * Norm over a list of gradients, and clipping to a largest norm:
 *   norm = sqrt(sum of all squares),  out_i = grads_i min(1, max_norm / (norm + 1e-6))
 * (one fp32 factor, or where it is below 2^-126 a power of two times one; a NaN or infinite norm gives the factor that this
 * formula gives; a finite norm that fp32 does not hold is written as infinity, its factor is that of the fp64 value).
 * Squares are added in fp32 over at most 64 values of a thread, everything else in fp64; where such a sum leaves fp32's
 * range its values are added in fp64 again. The order of the sums depends on the list's sizes and types alone, not on
 * addresses: results repeat bit for bit.
 *   grads, out, numel, types  HOST arrays of `count` device pointers, element counts and types (NVFP4_BF16,
 *              NVFP4_F16, NVFP4_F32), read before the call returns. out NULL: in place. Pointers need
 *              their elements' alignment only. Empty gradients may have null pointers.
 *   max_norm   >= 0; infinity: nothing is scaled, whatever the norm (in place: only the norm is computed; else copied)
 *   norm       device fp32 [1], written (0 for an empty list)
 *   workspace  nvfp4_grad_clip_workspace_bytes(count) bytes, 16-byte aligned
 * Results must not share memory with each other or with another gradient (the same tensor twice, for
 * instance), nor the norm or the workspace with any of them or each other: NVFP4_ERR_INVALID_ARG.
 */
size_t nvfp4_grad_clip_workspace_bytes(int32_t count);
int nvfp4_grad_clip(const void* const* grads, void* const* out, const int64_t* numel, const int32_t* types, int32_t count,
                    float max_norm, float* norm, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* NVFP4_FFN_H_ */
