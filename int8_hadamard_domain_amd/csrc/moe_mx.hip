// Grouped MXFP4 products of the routed experts: gate_up with its GELU
// epilogue, and the down projection with the weighted combine.
//
// Both operands are MXFP4 (activations quantised per token, or per act row,
// just before): for sorted row r of expert e
//   c[r, n] = sum_b 2^(sw[e,n,b] + sx[r,b] - 254) sum_{k in b} qw[e,n,k] qx[r,k]
// v_mfma_scale_f32_32x32x64_f8f6f4 takes the codes as they lie in memory and
// the block scales beside them, so there is no decode and no fold: a product
// step is the instruction alone. Its float32 sums keep the full significand
// (products far below the largest of an instruction are kept, unlike the E4M3
// forms), so the result is as exact as a float32 sum.
//
// The weights are the A operand (32 rows: for gate_up 16 gate rows and the
// matching 16 up rows, so both halves of an output meet in one lane), the
// activation rows the B operand (32 columns). A wave owns 32 weight rows and
// walks the expert's activation rows 32 at a time, operands straight from
// global memory.

#include "launch.hpp"
#include "mxfp4.hpp"

namespace i8h {

namespace {

constexpr int kMgThreads = 256;   // 4 waves, a 32-row weight tile each
constexpr int kMgWaves = kMgThreads / kWave;

struct MxArgs {
  const uint8_t* xq;   // activation codes, rows of K/2 bytes
  const uint8_t* xs;   // activation scales, rows of K/32
  const uint8_t* wq;   // [E, R, K/2]
  const uint8_t* ws;   // [E, R, K/32]
  int E, R, K, topk;
  const int32_t* expert_off;
  const int32_t* sorted_pairs;   // gate_up: activation row of sorted row r is sorted_pairs[r] / topk
};

// one 64-deep step's operand of a row: blocks 2 j + half (zero past the row's last block)
__device__ __forceinline__ u32x4 mx_codes(const uint8_t* row, int b, int nb) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (b < nb) v = *reinterpret_cast<const u32x4*>(row + 16 * b);
  return v;
}
__device__ __forceinline__ uint32_t mx_scale(const uint8_t* row, int b, int nb) { return b < nb ? row[b] : 127u; }

// GU: gate_up with epilogue (out0 = gate_up or NULL, out1 = act or NULL);
// otherwise out0 = y [P, R]
template <bool GU, typename AT>
__global__ void __launch_bounds__(kMgThreads)
k_mx_grouped(const MxArgs a, float* __restrict__ out0, AT* __restrict__ out1) {
  const int e = blockIdx.y;
  const int r0 = a.expert_off[e], m_e = a.expert_off[e + 1] - r0;
  if (m_e <= 0) return;
  const int lane = threadIdx.x % kWave, half = lane / 32, col = lane % 32;
  const int tile = blockIdx.x * kMgWaves + threadIdx.x / kWave;
  const int I = a.R / 2, nb = a.K / kMxBlock;
  if (tile * 32 >= a.R) return;
  // weight row of this lane
  int n;
  if constexpr (GU) n = col < 16 ? tile * 16 + col : I + tile * 16 + col - 16;
  else n = tile * 32 + col;
  const uint8_t* wq = a.wq + ((size_t)e * a.R + n) * (a.K / 2);
  const uint8_t* ws = a.ws + ((size_t)e * a.R + n) * nb;
  for (int m = 0; m < m_e; m += 32) {
    const int r = r0 + min(m + col, m_e - 1);
    const int xr = GU ? a.sorted_pairs[r] / a.topk : r;
    const uint8_t* xq = a.xq + (size_t)xr * (a.K / 2);
    const uint8_t* xs = a.xs + (size_t)xr * nb;
    f32x16 acc = {};
    for (int b = half; b < nb + half; b += 2)
      acc = mx_mfma32<0, 0>(mx_codes(wq, b, nb), mx_codes(xq, b, nb), acc, mx_scale(ws, b, nb), mx_scale(xs, b, nb));
    if (m + col >= m_e) continue;
    if constexpr (GU) {
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        // gate rows 8 q + 4 half .. +3 of the tile in registers 4 q .. +3, their up rows in 8 + 4 q .. +3
        const int i = tile * 16 + 8 * q + 4 * half;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float g = acc[4 * q + j], u = acc[8 + 4 * q + j];
          if (out0) {
            out0[(size_t)r * a.R + i + j] = g;
            out0[(size_t)r * a.R + I + i + j] = u;
          }
          if (out1) put_act(out1, (size_t)r * I + i + j, gelu_tanh(g) * u);
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        out0[(size_t)r * a.R + tile * 32 + 8 * (j / 4) + 4 * half + j % 4] = acc[j];
    }
  }
}

// out[t, h .. h + 3] = sum_j w[t, j] y[pos[t k + j], h .. h + 3], slot order
__global__ void __launch_bounds__(kMgThreads)
k_mx_combine(const float* __restrict__ y, int H, int k, const float* __restrict__ tw, const int32_t* __restrict__ pos,
             float* __restrict__ out) {
  const int64_t t = blockIdx.x;
  const int h = 4 * (blockIdx.y * kMgThreads + threadIdx.x);
  if (h >= H) return;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < k; ++j) {
    const float wj = tw[t * k + j];
    const f32x4 v = *reinterpret_cast<const f32x4*>(y + (size_t)pos[t * k + j] * H + h);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = fmaf(wj, v[i], o[i]);
  }
  *reinterpret_cast<f32x4*>(out + t * H + h) = o;
}

}  // namespace

hipError_t launch_gateup_mxfp4(const uint8_t* xq, const uint8_t* xs, int K, const uint8_t* codes,
                               const uint8_t* scales, int E, int N, int k, const int32_t* expert_off,
                               const int32_t* sorted_pairs, float* gu, void* act, bool act_bf16, hipStream_t st) {
  const MxArgs a = {xq, xs, codes, scales, E, N, K, k, expert_off, sorted_pairs};
  const dim3 grid(cdiv(N / 32, kMgWaves), E);
  if (act_bf16)
    k_mx_grouped<true><<<grid, kMgThreads, 0, st>>>(a, gu, static_cast<uint16_t*>(act));
  else
    k_mx_grouped<true><<<grid, kMgThreads, 0, st>>>(a, gu, static_cast<float*>(act));
  return hipGetLastError();
}

hipError_t launch_down_mxfp4(const uint8_t* aq, const uint8_t* as, int T, int I, const uint8_t* codes,
                             const uint8_t* scales, int E, int H, int k, const float* tw, const int32_t* expert_off,
                             const int32_t* pos, float* y, float* out, hipStream_t st) {
  const MxArgs a = {aq, as, codes, scales, E, H, I, k, expert_off, nullptr};
  const dim3 grid(cdiv(H / 32, kMgWaves), E);
  k_mx_grouped<false><<<grid, kMgThreads, 0, st>>>(a, y, static_cast<float*>(nullptr));
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  k_mx_combine<<<dim3(T, cdiv(H / 4, kMgThreads)), kMgThreads, 0, st>>>(y, H, k, tw, pos, out);
  return hipGetLastError();
}

}  // namespace i8h
