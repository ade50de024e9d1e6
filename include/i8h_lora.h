/*
 * i8h_lora — low-rank adapters of many requests beside a shared projection:
 * each row of the batch names the adapter that adds to its output. Part of
 * libi8h.so; i8h.h's conventions hold (device pointers, the caller's buffers,
 * host-side validation before any launch, T == 0 a no-op).
 *
 * Adapter l holds A_l [R, K] and B_l [N, R] in bf16 and a scale. With l =
 * adapter[t]:
 *   delta[t, n] = sum_r B_l[n, r] * (scale[l] * sum_k A_l[r, k] * x[t, k])
 * and delta[t] = 0 where l lies outside [0, L), for instance -1: those rows
 * have no adapter, and whatever the other rows' adapters hold does not reach
 * them. Adapters of smaller rank are padded with zeros to R. Products are
 * exact, sums float32; the inner sums enter the second product as float32
 * values (as three bf16 parts), not rounded. Results are the same, bit for
 * bit, in every run. An infinity in B gives one, or NaN where it meets an
 * inner sum of 0 or an infinity of the other sign (a subnormal inner sum may
 * count as 0 there).
 */
#ifndef I8H_LORA_H
#define I8H_LORA_H

#include "i8h_mxfp4.h"

#ifdef __cplusplus
extern "C" {
#endif

#define I8H_LORA_MAX_RANK 256

/* Device scratch of both calls, in bytes: the inner sums, T x R float32, in up
 * to 8 slices of K. lora_add takes none for few rows of low rank (T <= 256,
 * R <= 64, T * R <= 4096): its own size is 0 there, else the same. Sizes never
 * fall as T or R grow: scratch for the largest batch serves smaller ones. */
size_t lora_workspace_size(int T, int R);
size_t lora_add_workspace_size(int T, int R);

/* out[t] = base[t] + delta[t]: adapters beside any projection, base being its
 * output. base and out [T, N] of base_type (I8H_F32 or I8H_BF16: the float32
 * sum is rounded once, to nearest even), rows ldb and ldo elements apart,
 * aligned to the element; out may be base (with ldo == ldb), other overlap of
 * out with an input is refused (column slices of one matrix may lie side by
 * side). Rows without an adapter are copied bit for bit.
 * x [T, K] bf16, rows ldx apart (ldx % 8 == 0), 16-B aligned; lora_a
 * [L, R, K], lora_b [L, N, R] bf16, 16-B aligned; adapter [T] int32;
 * lora_scale [L] float32. K % 8 == 0, R % 8 == 0, L >= 1, any N >= 1 (else
 * I8H_EINVAL); R <= I8H_LORA_MAX_RANK, N and K <= 2^22, T <= 2^26, T * N <=
 * 2^35, row distances <= 2^24 (else I8H_EUNSUPPORTED).
 * workspace: at least lora_add_workspace_size(T, R) bytes, 256-B aligned,
 * contents on entry ignored (may be NULL when that size is 0). */
int lora_add(const void* base, int base_type, int64_t ldb, const uint16_t* x, int64_t ldx, int T, int K, int N,
             const uint16_t* lora_a, const uint16_t* lora_b, int L, int R, const int32_t* adapter,
             const float* lora_scale, void* out, int64_t ldo, void* workspace, size_t workspace_bytes,
             void* stream);

/* y[t] = linear_i8f16's product + delta[t]: the dense int8 linear with f16
 * scales and its adapters in one product. x, codes, scales, y as for
 * linear_i8f16 (K % 128 == 0, N % 16 == 0), the adapters and limits as above
 * (up to 32 tokens of low rank, linear_i8f16 and lora_add in place on its
 * output are the faster calls);
 * T * K < 2^31 (else I8H_EUNSUPPORTED). y overlaps no input. workspace: at
 * least lora_workspace_size(T, R) bytes. */
int linear_i8f16_lora(const uint16_t* x, int T, int K, const int8_t* codes, const uint16_t* scales, int N,
                      const uint16_t* lora_a, const uint16_t* lora_b, int L, int R, const int32_t* adapter,
                      const float* lora_scale, float* y, void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* I8H_LORA_H */
