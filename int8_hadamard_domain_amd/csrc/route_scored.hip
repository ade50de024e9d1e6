// Experts by scores: softmax or sigmoid over all experts, a bias for balance,
// groups, top-k, weights with or without renormalisation; then the stable
// permutation of moe_route_permute.
//
// Kernels
//   k_scored_rows     per chunk of tokens (at most 256 pairs): a wave per
//                     token chooses its experts; the chunk's histogram
//   k_route_scatter   (route.hip) totals, scan and stable ranks of a chunk
//
// The order of the choice values s + bias is that of float64: two experts
// whose float32 values round alike must not change places.

#include "common.hpp"
#include "launch.hpp"
#include "topk.hpp"

namespace i8h {

namespace {

constexpr int kScWaves = 4;                  // waves of a workgroup, a token each at a time
constexpr int kScThreads = kWave * kScWaves;

struct ScoredRule {
  const float* bias;       // [E] or NULL
  int E, k, groups, keep, top;
  bool sigmoid, renorm;
  float scale;
};

// Order-preserving map of a float64 to an unsigned key; NaN to 0, below every number.
__device__ __forceinline__ uint64_t order_key64(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);   // -0 + 0 = +0
  const uint64_t k = (b >> 63) ? ~b : (b | 0x8000000000000000ull);
  return v == v ? k : 0ull;
}

__device__ __forceinline__ uint64_t wave_max64(uint64_t v) {
#define I8H_STEP(M)                                                                                        \
  {                                                                                                        \
    const uint64_t o = (uint64_t)(uint32_t)xor_lane_i<M>((int)(uint32_t)v) |                               \
                       (uint64_t)(uint32_t)xor_lane_i<M>((int)(uint32_t)(v >> 32)) << 32;                  \
    v = o > v ? o : v;                                                                                     \
  }
  I8H_STEP(1) I8H_STEP(2) I8H_STEP(4) I8H_STEP(8) I8H_STEP(16) I8H_STEP(32)
#undef I8H_STEP
  return v;
}

__device__ __forceinline__ double wave_sum64(double v) {
#define I8H_STEP(M)                                                                                        \
  {                                                                                                        \
    const uint64_t b = __builtin_bit_cast(uint64_t, v);                                                    \
    const uint64_t o = (uint64_t)(uint32_t)xor_lane_i<M>((int)(uint32_t)b) |                               \
                       (uint64_t)(uint32_t)xor_lane_i<M>((int)(uint32_t)(b >> 32)) << 32;                  \
    v += __builtin_bit_cast(double, o);                                                                    \
  }
  I8H_STEP(1) I8H_STEP(2) I8H_STEP(4) I8H_STEP(8) I8H_STEP(16) I8H_STEP(32)
#undef I8H_STEP
  return v;
}

// One token by one wave, all in float64. Lane l holds the logits of experts
// VPL l .. VPL l + VPL - 1. Lane j < k returns the j-th choice and its weight.
// `lds` is the wave's own: E doubles.
template <int VPL>
__device__ __forceinline__ void scored_token(const float (&v)[VPL], const ScoredRule& R, int lane, double* lds,
                                             int& id, float& weight) {
  const int E = R.E;
  // scores
  double s[VPL];
  if (R.sigmoid) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) s[i] = 1.0 / (1.0 + exp(-(double)v[i]));
  } else {
    uint32_t m = 0;                            // key of the largest logit that is a number
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (VPL * lane + i < E) m = max(m, order_key(v[i]));
    const uint64_t top = wave_max64((uint64_t)m);
    const float mx = key_logit((uint32_t)top);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      s[i] = v[i] == -INFINITY || VPL * lane + i >= E ? 0.0 : exp((double)v[i] - (double)mx);
      sum += s[i];
    }
    sum = wave_sum64(sum);
#pragma unroll
    for (int i = 0; i < VPL; ++i) s[i] = sum == 0.0 ? 0.0 : s[i] / sum;   // only -inf: no scores
  }
  // choice keys, and the groups that stay
  uint64_t key[VPL];
  uint32_t open = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = VPL * lane + i;
    if (e < E) open |= 1u << i;
    key[i] = R.bias == nullptr ? (uint64_t)order_key(v[i]) : order_key64(s[i] + (double)R.bias[e < E ? e : 0]);
  }
  if (R.keep < R.groups) {
    const int size = E / R.groups;
    const bool by_key = R.bias == nullptr && R.top == 1;   // the largest logit's group is the one of largest score
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = VPL * lane + i;
      if (e < E)
        lds[e] = by_key ? __builtin_bit_cast(double, key[i]) : R.bias == nullptr ? s[i] : s[i] + (double)R.bias[e];
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    uint64_t worth = 0;
    if (lane < R.groups) {
      uint64_t a = 0, b = 0;                   // keys of the two largest
      for (int i = 0; i < size; ++i) {
        const double x = lds[lane * size + i];
        const uint64_t kx = by_key ? __builtin_bit_cast(uint64_t, x) : order_key64(x);
        if (kx > a) {
          b = a;
          a = kx;
        } else if (kx > b) {
          b = kx;
        }
      }
      worth = a;
      if (R.top == 2) {
        const auto value = [](uint64_t k) {
          return k == 0 ? __builtin_nan("") : __builtin_bit_cast(double, (k >> 63) ? k & 0x7fffffffffffffffull : ~k);
        };
        worth = order_key64(value(a) + value(b));
      }
    }
    int rank = 0;
    for (int g = 0; g < R.groups; ++g) {
      const uint64_t o = (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)worth, g) |
                         (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(worth >> 32), g) << 32;
      rank += o > worth || (o == worth && g < lane) ? 1 : 0;
    }
    const uint64_t stays = __ballot(lane < R.groups && rank < R.keep);
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const int e = VPL * lane + i;
      if (e < E && !((stays >> (e / size)) & 1)) open &= ~(1u << i);
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
  // the k largest keys, the lowest index first among equals
  int my_id = 0;
  for (int j = 0; j < R.k; ++j) {
    uint64_t m = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if ((open >> i) & 1u) m = key[i] > m ? key[i] : m;
    m = wave_max64(m);
    int first = VPL;
#pragma unroll
    for (int i = VPL - 1; i >= 0; --i)
      if (((open >> i) & 1u) && key[i] == m) first = i;
    const int owner = __ffsll((unsigned long long)__ballot(first < VPL)) - 1;
    const int at = __builtin_amdgcn_readlane(first, owner);
    if (lane == owner) open &= ~(1u << at);
    if (lane == j) my_id = VPL * owner + at;
  }
  // weights: the chosen scores by way of LDS
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (VPL * lane + i < E) lds[VPL * lane + i] = s[i];
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  double w = lane < R.k ? lds[my_id] : 0.0;
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  if (R.renorm) {
    const double total = wave_sum64(w);
    w = total == 0.0 ? 0.0 : w / total;
  }
  id = lane < R.k ? my_id : -1;
  weight = (float)(w * (double)R.scale);
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t v) { return bf16_to_f32(v); }

template <int VPL, typename X>
__device__ __forceinline__ void load_row(const X* __restrict__ row, int E, int lane, float (&v)[VPL]) {
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    const int e = VPL * lane + i;
    v[i] = e < E ? to_f32(row[e]) : -INFINITY;
  }
}

template <int VPL, typename X>
__global__ void __launch_bounds__(kScThreads)
k_scored_rows(const X* __restrict__ logits, int T, ScoredRule R, int tpc, int32_t* __restrict__ ids,
              float* __restrict__ w, int32_t* __restrict__ hist) {
  __shared__ int cnt[kWave * VPL];
  __shared__ double lds[kScWaves][kWave * VPL];
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  for (int e = threadIdx.x; e < R.E; e += blockDim.x) cnt[e] = 0;
  __syncthreads();
  const int t0 = blockIdx.x * tpc, t1 = min(T, t0 + tpc);
  for (int t = t0 + wave; t < t1; t += kScWaves) {
    float v[VPL];
    load_row<VPL>(logits + (size_t)t * R.E, R.E, lane, v);
    int id;
    float wt;
    scored_token<VPL>(v, R, lane, lds[wave], id, wt);
    if (lane < R.k) {
      ids[(size_t)t * R.k + lane] = id;
      w[(size_t)t * R.k + lane] = wt;
      atomicAdd(&cnt[id], 1);   // counts only: order does not matter
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < R.E; e += blockDim.x) hist[(size_t)blockIdx.x * R.E + e] = cnt[e];
}

template <typename X>
hipError_t launch(const void* logits, int T, const ScoredRule& R, int32_t* ids, float* w, int32_t* expert_off,
                  int32_t* sorted_pairs, int32_t* pair_pos, int32_t* hist, hipStream_t st) {
  const int nc = (int)route_chunks(T, R.k), tpc = route_chunk_tokens(T, R.k);
  const X* l = static_cast<const X*>(logits);
  if (R.E <= 64) k_scored_rows<1, X><<<nc, kScThreads, 0, st>>>(l, T, R, tpc, ids, w, hist);
  else if (R.E <= 128) k_scored_rows<2, X><<<nc, kScThreads, 0, st>>>(l, T, R, tpc, ids, w, hist);
  else if (R.E <= 256) k_scored_rows<4, X><<<nc, kScThreads, 0, st>>>(l, T, R, tpc, ids, w, hist);
  else if (R.E <= 512) k_scored_rows<8, X><<<nc, kScThreads, 0, st>>>(l, T, R, tpc, ids, w, hist);
  else k_scored_rows<16, X><<<nc, kScThreads, 0, st>>>(l, T, R, tpc, ids, w, hist);
  return launch_route_scatter(ids, T, R.E, R.k, hist, expert_off, sorted_pairs, pair_pos, st);
}

}  // namespace

size_t scored_workspace_bytes(int T, int E, int k) { return (size_t)route_chunks(T, k) * E * sizeof(int32_t); }

hipError_t launch_route_scored(const void* logits, bool bf16, int T, int E, int k, bool sigmoid, const float* bias,
                               int groups, int keep, int top, bool renorm, float scale, int32_t* ids, float* w,
                               int32_t* expert_off, int32_t* sorted_pairs, int32_t* pair_pos, void* ws,
                               hipStream_t st) {
  const ScoredRule R = {bias, E, k, groups, keep, top, sigmoid, renorm, scale};
  int32_t* hist = static_cast<int32_t*>(ws);
  if (bf16) return launch<uint16_t>(logits, T, R, ids, w, expert_off, sorted_pairs, pair_pos, hist, st);
  return launch<float>(logits, T, R, ids, w, expert_off, sorted_pairs, pair_pos, hist, st);
}

}  // namespace i8h
