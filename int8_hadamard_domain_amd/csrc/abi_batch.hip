// C ABI of the choice of experts by scores (i8h_scored.h) and the low-rank
// adapters (i8h_lora.h): host-side validation and launch. Every check runs
// before any HIP call, so an invalid call has no effect.

#include <hip/hip_runtime.h>

#include "../../include/i8h_lora.h"
#include "../../include/i8h_scored.h"
#include "launch.hpp"

namespace {

using i8h::kMaxExperts;
using i8h::kMaxTopk;

constexpr int kLoraMaxN = 1 << 22;      // grid rows of 64 columns and more
constexpr int kLoraMaxK = 1 << 22;      // rows of a tile are addressed with 32-bit offsets
constexpr int64_t kLoraMaxLd = 1 << 24;
constexpr int kLoraMaxT = 1 << 26;
// A launch holds fewer than 2^32 threads: workgroups of 256 take 32 x 256 of the output, of 512 (the linear) 128 x 128,
// and ragged edges make them fewer than four times as many.
constexpr int64_t kLoraMaxOutput = (int64_t)1 << 35;

inline bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int from_hip(hipError_t e) { return e == hipSuccess ? I8H_OK : I8H_EHIP; }
inline hipStream_t as_stream(void* s) { return reinterpret_cast<hipStream_t>(s); }
inline size_t round_up(size_t v, size_t a) { return (v + a - 1) / a * a; }
inline bool is_type(int t) { return t == I8H_F32 || t == I8H_BF16; }
inline size_t type_size(int t) { return t == I8H_F32 ? 4 : 2; }

// rows x cols elements, rows ld elements apart
struct Span {
  uintptr_t from, to, width, step;        // bytes: the whole, of a row, from row to row
  Span(const void* p, int64_t rows, int64_t cols, int64_t ld, size_t size) {
    from = reinterpret_cast<uintptr_t>(p);
    to = from + size * (uintptr_t)((rows - 1) * ld + cols);
    width = size * (uintptr_t)cols;
    step = size * (uintptr_t)ld;
  }
  bool meets(const Span& o) const {
    if (from >= o.to || o.from >= to) return false;
    if (step != o.step) return true;
    // rows the same distance apart: column slices of one matrix do not meet where their columns do not
    const uintptr_t d = o.from >= from ? (o.from - from) % step : (step - (from - o.from) % step) % step;
    return d < width || step - d < o.width;
  }
};

// whether the output meets what the kernels still read while they write it
bool meets_lora(const Span& o, const uint16_t* x, int64_t T, int64_t K, int64_t ldx, int64_t N, const uint16_t* a,
                const uint16_t* b, int64_t L, int64_t R, const int32_t* adapter, const float* scale,
                const void* workspace, size_t workspace_bytes) {
  return o.meets(Span(x, T, K, ldx, 2)) || o.meets(Span(a, L, R * K, R * K, 2)) ||
         o.meets(Span(b, L, N * R, N * R, 2)) || o.meets(Span(adapter, 1, T, T, 4)) ||
         o.meets(Span(scale, 1, L, L, 4)) || (workspace_bytes > 0 && o.meets(Span(workspace, 1, workspace_bytes, 1, 1)));
}

int check_lora(const uint16_t* x, int T, const uint16_t* a, const uint16_t* b, const int32_t* adapter, const float* scale,
               const void* workspace, size_t workspace_bytes, size_t need) {
  if (T == 0) return I8H_OK;
  if (!x || !a || !b || !adapter || !scale) return I8H_EINVAL;
  if (!aligned(x, 16) || !aligned(a, 16) || !aligned(b, 16) || !aligned(adapter, 4) || !aligned(scale, 4))
    return I8H_EINVAL;
  if (need > 0 && (!workspace || !aligned(workspace, 256) || workspace_bytes < need)) return I8H_EINVAL;
  return I8H_OK;
}

}  // namespace

extern "C" {

size_t moe_route_scored_workspace_size(int T, int E, int topk) {
  if (T <= 0 || E <= 0 || topk <= 0 || E > kMaxExperts || topk > kMaxTopk) return 0;
  return round_up(i8h::scored_workspace_bytes(T, E, topk), 256);
}

int moe_route_scored_permute(const void* logits, int logits_type, int T, int E, int topk, int score,
                             const float* bias, int groups, int topk_groups, int group_top, int renormalize,
                             float scale, int32_t* topk_ids, float* topk_w, int32_t* expert_off,
                             int32_t* sorted_pairs, int32_t* pair_pos, void* workspace, size_t workspace_bytes,
                             void* stream) {
  if (!is_type(logits_type) || T < 0 || E <= 0 || topk <= 0) return I8H_EINVAL;
  if (score != I8H_SCORE_SOFTMAX && score != I8H_SCORE_SIGMOID) return I8H_EINVAL;
  if (groups <= 0 || (E % groups) != 0 || topk_groups <= 0 || topk_groups > groups) return I8H_EINVAL;
  if (group_top < 1 || group_top > 2 || (groups > 1 && group_top > E / groups)) return I8H_EINVAL;
  if (topk > (int64_t)topk_groups * (E / groups)) return I8H_EINVAL;
  if (E > kMaxExperts || topk > kMaxTopk || groups > I8H_MAX_GROUPS) return I8H_EUNSUPPORTED;
  if ((int64_t)T * topk >= (int64_t)1 << 31) return I8H_EUNSUPPORTED;
  if (!i8h::scored_fits(T, E, topk)) return I8H_EUNSUPPORTED;
  if (T == 0) return I8H_OK;
  if (!logits || !topk_ids || !topk_w || !expert_off || !sorted_pairs || !pair_pos) return I8H_EINVAL;
  if (!aligned(logits, type_size(logits_type)) || !aligned(bias, 4) || !aligned(topk_ids, 4) ||
      !aligned(topk_w, 4) || !aligned(expert_off, 4) || !aligned(sorted_pairs, 4) || !aligned(pair_pos, 4))
    return I8H_EINVAL;
  const size_t need = moe_route_scored_workspace_size(T, E, topk);
  if (need > 0 && (!workspace || workspace_bytes < need || !aligned(workspace, 256))) return I8H_EINVAL;
  return from_hip(i8h::launch_route_scored(logits, logits_type == I8H_BF16, T, E, topk, score == I8H_SCORE_SIGMOID,
                                           bias, groups, topk_groups, group_top, renormalize != 0, scale, topk_ids,
                                           topk_w, expert_off, sorted_pairs, pair_pos, workspace,
                                           as_stream(stream)));
}

size_t lora_workspace_size(int T, int R) {
  if (T <= 0 || R <= 0) return 0;
  return round_up((size_t)i8h::lora_sums(T) * R * sizeof(float), 256);
}

size_t lora_add_workspace_size(int T, int R) { return i8h::lora_few(T, R) ? 0 : lora_workspace_size(T, R); }

int lora_add(const void* base, int base_type, int64_t ldb, const uint16_t* x, int64_t ldx, int T, int K, int N,
             const uint16_t* lora_a, const uint16_t* lora_b, int L, int R, const int32_t* adapter,
             const float* lora_scale, void* out, int64_t ldo, void* workspace, size_t workspace_bytes,
             void* stream) {
  if (!is_type(base_type) || T < 0 || K <= 0 || (K % 8) != 0 || N <= 0 || L <= 0 || R <= 0 || (R % 8) != 0)
    return I8H_EINVAL;
  if (ldb < N || ldo < N || ldx < K || (ldx % 8) != 0) return I8H_EINVAL;
  if (R > I8H_LORA_MAX_RANK || N > kLoraMaxN || T > kLoraMaxT || K > kLoraMaxK) return I8H_EUNSUPPORTED;
  if ((int64_t)T * N > kLoraMaxOutput) return I8H_EUNSUPPORTED;
  if (ldb > kLoraMaxLd || ldo > kLoraMaxLd || ldx > kLoraMaxLd) return I8H_EUNSUPPORTED;
  const size_t need = lora_add_workspace_size(T, R);
  const int rc = check_lora(x, T, lora_a, lora_b, adapter, lora_scale, workspace, workspace_bytes, need);
  if (rc != I8H_OK || T == 0) return rc;
  const size_t el = type_size(base_type);
  if (!base || !out || !aligned(base, el) || !aligned(out, el)) return I8H_EINVAL;
  const Span o(out, T, N, ldo, el);
  if (base == out ? ldb != ldo : o.meets(Span(base, T, N, ldb, el))) return I8H_EINVAL;
  if (meets_lora(o, x, T, K, ldx, N, lora_a, lora_b, L, R, adapter, lora_scale, workspace, need))
    return I8H_EINVAL;
  hipStream_t st = as_stream(stream);
  if (i8h::lora_few(T, R))
    return from_hip(i8h::launch_lora_few(base, base_type == I8H_BF16, ldb, x, ldx, T, K, N, lora_a, lora_b, L, R,
                                         adapter, lora_scale, out, ldo, st));
  float* h = static_cast<float*>(workspace);
  int slices = 1;
  if (i8h::launch_lora_shrink(x, ldx, T, K, lora_a, L, R, adapter, lora_scale, h, &slices, st) != hipSuccess)
    return I8H_EHIP;
  return from_hip(i8h::launch_lora_add(base, base_type == I8H_BF16, ldb, T, N, lora_b, L, R, adapter, h, slices, out,
                                       ldo, st));
}

int linear_i8f16_lora(const uint16_t* x, int T, int K, const int8_t* codes, const uint16_t* scales, int N,
                      const uint16_t* lora_a, const uint16_t* lora_b, int L, int R, const int32_t* adapter,
                      const float* lora_scale, float* y, void* workspace, size_t workspace_bytes, void* stream) {
  if (T < 0 || K <= 0 || (K % 128) != 0 || N <= 0 || (N % 16) != 0 || L <= 0 || R <= 0 || (R % 8) != 0)
    return I8H_EINVAL;
  if (R > I8H_LORA_MAX_RANK || N > kLoraMaxN || K > kLoraMaxK || (int64_t)T * K >= (int64_t)1 << 31) return I8H_EUNSUPPORTED;
  if (T > kLoraMaxT || (int64_t)T * N > kLoraMaxOutput) return I8H_EUNSUPPORTED;
  const size_t need = lora_workspace_size(T, R);
  const int rc = check_lora(x, T, lora_a, lora_b, adapter, lora_scale, workspace, workspace_bytes, need);
  if (rc != I8H_OK || T == 0) return rc;
  if (!codes || !scales || !y || !aligned(codes, 16) || !aligned(scales, 2) || !aligned(y, 4)) return I8H_EINVAL;
  const Span o(y, T, N, N, 4);
  if (o.meets(Span(codes, N, K, K, 1)) || o.meets(Span(scales, N, K / 128, K / 128, 2)) ||
      meets_lora(o, x, T, K, K, N, lora_a, lora_b, L, R, adapter, lora_scale, workspace, need))
    return I8H_EINVAL;
  hipStream_t st = as_stream(stream);
  float* h = static_cast<float*>(workspace);
  int slices = 1;
  if (i8h::launch_lora_shrink(x, K, T, K, lora_a, L, R, adapter, lora_scale, h, &slices, st) != hipSuccess) return I8H_EHIP;
  return from_hip(i8h::launch_linear_i8f16_lora(x, T, K, codes, scales, N, lora_b, L, R, adapter, h, slices, y, st));
}

}  // extern "C"
