// C ABI of the MXFP4 experts (i8h_mxfp4.h) and the verification of drafted
// tokens (i8h_draft.h): host-side validation and launch. Every check runs
// before any HIP call, so an invalid call has no effect.

#include <hip/hip_runtime.h>

#include "../../include/i8h_draft.h"
#include "../../include/i8h_mxfp4.h"
#include "launch.hpp"

namespace {

using i8h::kMaxExperts;
using i8h::kMaxTopk;

constexpr int kDraftMaxD = 1023;
constexpr int kDraftMaxB = 65535;   // a sequence per grid row

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int from_hip(hipError_t e) { return e == hipSuccess ? I8H_OK : I8H_EHIP; }
inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline bool is_type(int t) { return t == I8H_F32 || t == I8H_BF16; }

// the products address the quantised rows with 32-bit offsets (144 bytes a stage of 256)
inline bool rows_fit(int64_t rows, int K) { return rows * ((int64_t)K + i8h::kMxStage) < ((int64_t)1 << 32); }

// a thread per 8 values: a launch holds fewer than 2^32 threads, in workgroups of 256
inline bool quant_fits(int64_t rows, int K) { return rows * (K / 8) <= ((int64_t)1 << 32) - 256; }

}  // namespace

extern "C" {

int mxfp4_quantize(const void* x, int x_type, int T, int K, uint8_t* codes, uint8_t* scales, void* stream) {
  if (!is_type(x_type) || T < 0 || K <= 0 || (K % 32) != 0) return I8H_EINVAL;
  if (!quant_fits(T, K)) return I8H_EUNSUPPORTED;
  if (T == 0) return I8H_OK;
  if (!x || !codes || !scales || !aligned(x, 16) || !aligned(codes, 16)) return I8H_EINVAL;
  return from_hip(i8h::launch_mxfp4_quantize(x, x_type == I8H_BF16, (int64_t)T * K, codes, scales,
                                             as_stream(stream)));
}

int mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int T, int K, void* out, int out_type,
                     void* stream) {
  if (!is_type(out_type) || T < 0 || K <= 0 || (K % 32) != 0) return I8H_EINVAL;
  if (!quant_fits(T, K)) return I8H_EUNSUPPORTED;
  if (T == 0) return I8H_OK;
  if (!codes || !scales || !out || !aligned(codes, 16) || !aligned(out, 16)) return I8H_EINVAL;
  return from_hip(i8h::launch_mxfp4_dequantize(codes, scales, (int64_t)T * K, out, out_type == I8H_BF16,
                                               as_stream(stream)));
}

size_t moe_gateup_mxfp4_workspace_size(int T, int K, int E, int topk) {
  if (T <= 0 || K <= 0 || (K % 128) != 0 || E <= 0 || topk <= 0 || i8h::mx_few_gateup(T, K, topk)) return 0;
  return i8h::MxWorkspace(T, K, (int64_t)T * topk, E).total;
}

int moe_gateup_mxfp4_grouped(const uint16_t* x, int T, int K, const uint8_t* codes, const uint8_t* scales, int E,
                             int N, int topk, const int32_t* expert_off, const int32_t* sorted_pairs,
                             float* gate_up, void* act, int act_type, void* workspace, size_t workspace_bytes,
                             void* stream) {
  if (!is_type(act_type) || T < 0 || K <= 0 || (K % 128) != 0 || E <= 0 || N <= 0 || topk <= 0) return I8H_EINVAL;
  if (E > kMaxExperts || topk > kMaxTopk || topk > E) return I8H_EUNSUPPORTED;
  if ((N % 2) != 0) return I8H_EINVAL;          // gate and up halves
  if ((N % 64) != 0 || (int64_t)N * K >= (int64_t)1 << 32) return I8H_EUNSUPPORTED;   // 32-bit offsets in an expert
  if ((int64_t)T * topk >= (int64_t)1 << 31) return I8H_EUNSUPPORTED;
  if (!rows_fit(T, K) || !i8h::mx_launch_fits(K, (int64_t)T * topk, E, N)) return I8H_EUNSUPPORTED;
  if (T == 0) return I8H_OK;
  if (!x || !codes || !scales || !expert_off || !sorted_pairs) return I8H_EINVAL;
  if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(expert_off, 4) ||
      !aligned(sorted_pairs, 4))
    return I8H_EINVAL;
  if ((gate_up && !aligned(gate_up, 16)) || (act && !aligned(act, 16))) return I8H_EINVAL;
  const size_t need = moe_gateup_mxfp4_workspace_size(T, K, E, topk);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return I8H_EINVAL;
  if (!gate_up && !act) return I8H_OK;          // nothing requested
  if (i8h::mx_few_gateup(T, K, topk))
    return from_hip(i8h::launch_gateup_mxfp4_few(x, T, K, codes, scales, E, N, topk, expert_off, sorted_pairs, gate_up,
                                                 act, act_type == I8H_BF16, as_stream(stream)));
  return from_hip(i8h::launch_gateup_mxfp4(x, T, K, codes, scales, E, N, topk, expert_off, sorted_pairs, gate_up, act,
                                           act_type == I8H_BF16, static_cast<uint8_t*>(workspace),
                                           as_stream(stream)));
}

size_t moe_down_mxfp4_workspace_size(int T, int I, int E, int H, int topk) {
  if (T <= 0 || I <= 0 || (I % 32) != 0 || E <= 0 || H <= 0 || topk <= 0 || i8h::mx_few_down(T, I, topk)) return 0;
  const int64_t P = (int64_t)T * topk;
  return i8h::MxWorkspace(P, I, P, E).total + round_up((size_t)P * H * sizeof(float), 256);
}

int moe_down_mxfp4_combine(const void* act, int act_type, int T, int I, const uint8_t* codes, const uint8_t* scales,
                           int E, int H, int topk, const int32_t* topk_ids, const float* topk_w,
                           const int32_t* expert_off, const int32_t* pair_pos, float* out, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (!is_type(act_type) || T < 0 || I <= 0 || (I % 32) != 0 || H <= 0 || (H % 8) != 0 || E <= 0 || topk <= 0)
    return I8H_EINVAL;
  if (E > kMaxExperts || topk > kMaxTopk || topk > E) return I8H_EUNSUPPORTED;
  // 32-bit offsets in an expert, and in 32 rows of y
  if ((H % 32) != 0 || (int64_t)H * I >= (int64_t)1 << 32 || H >= 1 << 25) return I8H_EUNSUPPORTED;
  const int64_t P = (int64_t)T * topk;
  if (P >= (int64_t)1 << 31) return I8H_EUNSUPPORTED;
  if (!rows_fit(P, I) || !i8h::mx_launch_fits(I, P, E, H)) return I8H_EUNSUPPORTED;
  if (T == 0) return I8H_OK;
  if (!act || !codes || !scales || !topk_ids || !topk_w || !expert_off || !pair_pos || !out) return I8H_EINVAL;
  if (!aligned(act, 16) || !aligned(codes, 16) || !aligned(scales, 4) || !aligned(out, 16)) return I8H_EINVAL;
  if (!aligned(topk_ids, 4) || !aligned(topk_w, 4) || !aligned(expert_off, 4) || !aligned(pair_pos, 4))
    return I8H_EINVAL;
  const size_t need = moe_down_mxfp4_workspace_size(T, I, E, H, topk);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return I8H_EINVAL;
  if (i8h::mx_few_down(T, I, topk))
    return from_hip(i8h::launch_down_mxfp4_few(act, act_type == I8H_BF16, T, I, codes, scales, H, topk, topk_ids,
                                               topk_w, pair_pos, out, as_stream(stream)));
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* y = reinterpret_cast<float*>(ws + i8h::MxWorkspace(P, I, P, E).total);
  return from_hip(i8h::launch_down_mxfp4(act, act_type == I8H_BF16, T, I, codes, scales, E, H, topk, topk_w, expert_off,
                                         pair_pos, ws, y, out, as_stream(stream)));
}

size_t draft_verify_workspace_size(int B, int V) {
  if (B <= 0 || V <= 0) return 0;
  return round_up(i8h::draft_workspace_bytes(B, V), 256);
}

int draft_verify(const void* target_probs, const void* draft_probs, int prob_type, const int32_t* drafted,
                 const int32_t* draft_len, const float* u, const float* u_next, int B, int D, int V, int32_t* tokens,
                 int32_t* accepted, void* workspace, size_t workspace_bytes, void* stream) {
  if (!is_type(prob_type) || B < 0 || D < 0 || V <= 0) return I8H_EINVAL;
  if (D > kDraftMaxD || B > kDraftMaxB) return I8H_EUNSUPPORTED;
  if (B == 0) return I8H_OK;
  if (!target_probs || !u_next || !tokens || !accepted || (D > 0 && (!drafted || !u))) return I8H_EINVAL;
  const size_t el = prob_type == I8H_F32 ? 4 : 2;
  if (!aligned(target_probs, el) || !aligned(draft_probs, el) || !aligned(drafted, 4) || !aligned(draft_len, 4) ||
      !aligned(u, 4) || !aligned(u_next, 4) || !aligned(tokens, 4) || !aligned(accepted, 4))
    return I8H_EINVAL;
  if (!workspace || workspace_bytes < draft_verify_workspace_size(B, V) || !aligned(workspace, 256))
    return I8H_EINVAL;
  return from_hip(i8h::launch_draft_verify(target_probs, draft_probs, prob_type == I8H_BF16, drafted, draft_len, u,
                                           u_next, B, D, V, workspace, tokens, accepted,
                                           as_stream(stream)));
}

}  // extern "C"
