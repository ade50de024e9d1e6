// Low-rank adapters of many requests beside a shared projection.
//   h[t, r]   = scale[l] * sum_k A[l][r, k] x[t, k],  l = adapter[t]
//   out[t, n] = base[t, n] + sum_r B[l][n, r] h[t, r]
//
// Kernels
//   k_lora_shrink  h: a workgroup owns 16 rows of the batch and goes through
//                  the adapters they name; its eight waves split K
//   k_lora_add     out: a wave owns 16 rows x 64 columns
//
// Both run on v_mfma_f32_16x16x32_bf16 with a row of the batch per matrix row
// (or column), so what an adapter holds reaches no row but its own: values of
// rows that name another adapter are computed and dropped. h is float32; the
// second product takes it as the sum of three bf16 values (8 significand bits
// each, the split is exact), so nothing is rounded between the products.

#include "common.hpp"
#include "launch.hpp"
#include "lora.hpp"

namespace i8h {

namespace {

constexpr int kShWaves = 8;                    // waves of the shrink kernel, each a share of K
constexpr int kShThreads = kWave * kShWaves;
constexpr int kAddWaves = 4;
constexpr int kAddThreads = kWave * kAddWaves;
constexpr int kAddTiles = 4;                   // 16-column tiles a wave
constexpr int kAddCols = kAddWaves * kAddTiles * 16;

__device__ __forceinline__ bf16x8 load8(const uint16_t* p, bool live) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (live) v = *reinterpret_cast<const u32x4*>(p);
  return __builtin_bit_cast(bf16x8, v);
}

// NG: 16-wide groups of R a workgroup computes
template <int NG>
__global__ void __launch_bounds__(kShThreads)
k_lora_shrink(const uint16_t* __restrict__ x, int64_t ldx, int T, int K, const uint16_t* __restrict__ a, int L, int R,
              const int32_t* __restrict__ adapter, const float* __restrict__ scale, float* __restrict__ h) {
  __shared__ f32x4 part[kShWaves][NG][kWave];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane % 16, kq = lane / 16;
  const int64_t t0 = (int64_t)blockIdx.x * 16;
  const int r0 = blockIdx.z * 16 * NG;
  const bool row = t0 + c < T;
  const int ad = lora_row_adapter(adapter, t0, T, L, c);
  const uint16_t* xrow = x + (t0 + c) * ldx;
  uint32_t left = lora_rows(ad >= 0);
  int skip = blockIdx.y;
  while (left != 0) {
    const int l = __builtin_amdgcn_readlane(ad, __ffs(left) - 1);
    const uint32_t mine = lora_rows(ad == l);
    left &= ~mine;
    if (skip-- > 0) continue;
    skip = gridDim.y - 1;
    const uint16_t* al = a + (size_t)l * R * K;
    f32x4 acc[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) acc[g] = {0.f, 0.f, 0.f, 0.f};
    for (int64_t k0 = 128 * wave; k0 < K; k0 += 128 * kShWaves) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t k = k0 + 32 * kq + 8 * i;
        const bf16x8 xv = load8(xrow + k, row && k < K);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          const int r = r0 + 16 * g + c;
          const bf16x8 av = load8(al + (size_t)r * K + k, r < R && k < K);
          acc[g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, av, acc[g], 0, 0, 0);
        }
      }
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) part[wave][g][lane] = acc[g];
    __syncthreads();
    if (wave < NG) {
      f32x4 s = part[0][wave][lane];
#pragma unroll
      for (int w = 1; w < kShWaves; ++w) {
        const f32x4 o = part[w][wave][lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += o[i];
      }
      const int r = r0 + 16 * wave + c;
      const float f = scale[l];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r < R && ((mine >> (4 * kq + i)) & 1)) h[(t0 + 4 * kq + i) * R + r] = f * s[i];
    }
    __syncthreads();
  }
}

template <bool BF16>
__global__ void __launch_bounds__(kAddThreads)
k_lora_add(const void* base, int64_t ldb, int T, int N, const uint16_t* __restrict__ b, int L, int R,
           const int32_t* __restrict__ adapter, const float* __restrict__ h, void* out, int64_t ldo, bool vec) {
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane % 16, kq = lane / 16;
  const int64_t t0 = (int64_t)blockIdx.x * 16;
  const int n0 = blockIdx.y * kAddCols + wave * kAddTiles * 16;
  if (n0 >= N) return;
  const int ad = lora_row_adapter(adapter, t0, T, L, c);
  f32x4 acc[kAddTiles];
#pragma unroll
  for (int j = 0; j < kAddTiles; ++j) acc[j] = {0.f, 0.f, 0.f, 0.f};
  lora_expand<kAddTiles>(b, N, R, h, t0, T, n0, ad, lane, acc);
  if (t0 + c >= T) return;
  // the lane's row t0 + c, columns n0 + 16 j + 4 kq ..
#pragma unroll
  for (int j = 0; j < kAddTiles; ++j) {
    const int n = n0 + 16 * j + 4 * kq;
    if constexpr (BF16) {
      const uint16_t* s = static_cast<const uint16_t*>(base) + (t0 + c) * ldb + n;
      uint16_t* d = static_cast<uint16_t*>(out) + (t0 + c) * ldo + n;
      if (vec && n + 3 < N) {
        const u32x2 v = *reinterpret_cast<const u32x2*>(s);
        u32x2 o = {pack_bf16x2(bf16_lo(v[0]) + acc[j][0], bf16_hi(v[0]) + acc[j][1]),
                   pack_bf16x2(bf16_lo(v[1]) + acc[j][2], bf16_hi(v[1]) + acc[j][3])};
        *reinterpret_cast<u32x2*>(d) = ad >= 0 ? o : v;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < N) d[i] = ad >= 0 ? __builtin_bit_cast(uint16_t, (__bf16)(bf16_to_f32(s[i]) + acc[j][i])) : s[i];
      }
    } else {
      const float* s = static_cast<const float*>(base) + (t0 + c) * ldb + n;
      float* d = static_cast<float*>(out) + (t0 + c) * ldo + n;
      if (vec && n + 3 < N) {
        const f32x4 v = *reinterpret_cast<const f32x4*>(s);
        f32x4 o;
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = ad >= 0 ? v[i] + acc[j][i] : v[i];
        *reinterpret_cast<f32x4*>(d) = o;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < N) d[i] = ad >= 0 ? s[i] + acc[j][i] : s[i];
      }
    }
  }
}

}  // namespace

hipError_t launch_lora_shrink(const uint16_t* x, int64_t ldx, int T, int K, const uint16_t* a, int L, int R,
                              const int32_t* adapter, const float* scale, float* h, hipStream_t st) {
  // a workgroup per 16 rows and adapter among them while rows are few, else one that goes through its rows' adapters
  const int y = T <= 1024 ? min(min(T, 16), L) : 1;
  if (R <= 16)
    k_lora_shrink<1><<<dim3(cdiv(T, 16), y, 1), kShThreads, 0, st>>>(x, ldx, T, K, a, L, R, adapter, scale, h);
  else if (R <= 32)
    k_lora_shrink<2><<<dim3(cdiv(T, 16), y, 1), kShThreads, 0, st>>>(x, ldx, T, K, a, L, R, adapter, scale, h);
  else
    k_lora_shrink<4><<<dim3(cdiv(T, 16), y, cdiv(R, 64)), kShThreads, 0, st>>>(x, ldx, T, K, a, L, R, adapter, scale,
                                                                              h);
  return hipGetLastError();
}

hipError_t launch_lora_add(const void* base, bool bf16, int64_t ldb, int T, int N, const uint16_t* b, int L, int R,
                           const int32_t* adapter, const float* h, void* out, int64_t ldo, hipStream_t st) {
  const uintptr_t unit = bf16 ? 8 : 16;   // four elements
  const bool vec = reinterpret_cast<uintptr_t>(base) % unit == 0 && reinterpret_cast<uintptr_t>(out) % unit == 0 &&
                   ldb % 4 == 0 && ldo % 4 == 0;
  const dim3 grid(cdiv(T, 16), cdiv(N, kAddCols));
  if (bf16) k_lora_add<true><<<grid, kAddThreads, 0, st>>>(base, ldb, T, N, b, L, R, adapter, h, out, ldo, vec);
  else k_lora_add<false><<<grid, kAddThreads, 0, st>>>(base, ldb, T, N, b, L, R, adapter, h, out, ldo, vec);
  return hipGetLastError();
}

}  // namespace i8h
