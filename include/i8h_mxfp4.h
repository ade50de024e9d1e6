/*
 * i8h_mxfp4 — the routed experts in MXFP4: quantiser, grouped gate_up and
 * grouped down projection on gfx950's FP4 matrix cores. Part of libi8h.so;
 * i8h.h's conventions hold for every call (device pointers, the caller's
 * buffers, host-side validation before any launch, T == 0 a no-op).
 *
 * MXFP4 is the 4-bit format of the OCP Microscaling Formats (MX) specification
 * v1.0: a block of 32 consecutive values of K shares one E8M0 scale, byte s
 * standing for 2^(s - 127) (255: NaN), and each value is E2M1: a sign and one
 * of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (codes 0..7, the sign in bit 3). Two codes go
 * to a byte, the value of lower index in the low nibble. A matrix [R, K] is
 * codes [R, K/2] and scales [R, K/32], both uint8, rows contiguous.
 *
 * The products take both operands in MXFP4 (v_mfma_scale_f32_*_f8f6f4), and
 * sum in float32: products of two E2M1 values and their scales are exact
 * multiples of 2^-149 (what lies below is lost), and the matrix unit keeps
 * float32's full significand when it adds them, subnormals included. Sums past
 * float32's largest value are infinite. A NaN scale makes every output NaN
 * whose row or column holds it.
 */
#ifndef I8H_MXFP4_H
#define I8H_MXFP4_H

#include "i8h.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of floating-point arrays: float32, or bf16 bit patterns. */
enum { I8H_F32 = 0, I8H_BF16 = 1 };

/* Quantiser: x [T, K] (x_type: I8H_F32 or I8H_BF16, 16-B aligned, K % 32 ==
 * 0) to codes [T, K/2] (16-B aligned) and scales [T, K/32]. Per block, with
 * a = max |x|:
 *   s = max(floor(log2 a) - 2, -127) + 127      (0 where a == 0)
 *   code = E2M1(x * 2^(127 - s))                (nearest, ties to the even
 *          code, magnitudes above 6 become 6, the sign of zero is kept)
 * which is the conversion that the MX specification gives for E2M1. A block
 * with an infinity or NaN gets s = 255 and codes 0. T*K above 2^35 - 2048:
 * I8H_EUNSUPPORTED (for both calls). */
int mxfp4_quantize(const void* x, int x_type, int T, int K, uint8_t* codes, uint8_t* scales, void* stream);

/* The values that codes and scales stand for: out [T, K] (out_type, 16-B
 * aligned). Exact, but for magnitudes above the type's largest, which become
 * infinities (s = 253 or 254 only); NaN in blocks with s = 255. */
int mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int T, int K, void* out, int out_type,
                     void* stream);

/* Grouped gate_up with MXFP4 weights: x (bf16 [T, K], 16-B aligned, not
 * rotated or rotated as the weights were) is quantised as mxfp4_quantize
 * does, then for the pair in expert-sorted row r (expert e, token t)
 *   gu[r, n] = sum_b 2^(sw[e,n,b] + sx[t,b] - 254) sum_{k in b} qw[e,n,k] qx[t,k]
 * with the epilogue, row order and outputs of moe_gateup_i8h_grouped.
 *
 * codes [E, N, K/2] 16-B aligned, scales [E, N, K/32] 4-B aligned; K % 128 ==
 * 0; N positive and even (odd: I8H_EINVAL) and a multiple of 64, N*K < 2^32 and T*(K + 256) <
 * 2^32 (else I8H_EUNSUPPORTED). gate_up float32 [T*topk, N] or NULL; act [T*topk, N/2]
 * of act_type (bf16: each value rounded to nearest even from the float32
 * one) or NULL; both 16-B aligned. workspace: at least
 * moe_gateup_mxfp4_workspace_size(T, K, E, topk) bytes, 256-B aligned
 * (may be NULL when that size is 0: with few rows an expert the call is one
 * launch that needs none); what it holds after the call is unspecified. */
size_t moe_gateup_mxfp4_workspace_size(int T, int K, int E, int topk);
int moe_gateup_mxfp4_grouped(const uint16_t* x, int T, int K, const uint8_t* codes, const uint8_t* scales,
                             int E, int N, int topk, const int32_t* expert_off, const int32_t* sorted_pairs,
                             float* gate_up, void* act, int act_type, void* workspace,
                             size_t workspace_bytes, void* stream);

/* Grouped down projection with MXFP4 weights and the weighted combine, the
 * MXFP4 form of moe_down_bf16_combine: the expert-sorted act rows [P, I]
 * (act_type, 16-B aligned, I % 32 == 0) are quantised as mxfp4_quantize does,
 *   y[r, h]   = sum_b 2^(sw[e,h,b] + sa[r,b] - 254) sum_{i in b} qw[e,h,i] qa[r,i]
 *   out[t, h] = sum_j topk_w[t, j] * y[pair_pos[t*topk + j], h]   (slot order)
 * codes [E, H, I/2] 16-B aligned, scales [E, H, I/32] 4-B aligned; H % 32 ==
 * 0 (H % 8 != 0: I8H_EINVAL, else I8H_EUNSUPPORTED), H < 2^25, H*I <
 * 2^32 and T*topk*(I + 256) < 2^32 (else I8H_EUNSUPPORTED). out float32 [T, H],
 * 16-B aligned. topk_ids, topk_w, expert_off, pair_pos: as moe_route_permute
 * writes them. workspace: at least moe_down_mxfp4_workspace_size(T, I, E,
 * H, topk) bytes, 256-B aligned (may be NULL when that size is 0,
 * as for gate_up), contents unspecified afterwards. */
size_t moe_down_mxfp4_workspace_size(int T, int I, int E, int H, int topk);
int moe_down_mxfp4_combine(const void* act, int act_type, int T, int I, const uint8_t* codes,
                           const uint8_t* scales, int E, int H, int topk, const int32_t* topk_ids,
                           const float* topk_w, const int32_t* expert_off, const int32_t* pair_pos,
                           float* out, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* I8H_MXFP4_H */
