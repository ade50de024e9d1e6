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
#include "xlane.hpp"

namespace i8h {

namespace {

constexpr int kShWaves = 8;                    // waves of the shrink kernel, each a share of K
constexpr int kShThreads = kWave * kShWaves;
constexpr int kFewWaves = 8;
constexpr int kFewThreads = kWave * kFewWaves;
constexpr int kAddWaves = 4;
constexpr int kAddThreads = kWave * kAddWaves;
constexpr int kAddTiles = 4;                   // 16-column tiles a wave
constexpr int kAddCols = kAddWaves * kAddTiles * 16;

__device__ __forceinline__ bf16x8 load8(const uint16_t* p, bool live) {
  u32x4 v = {0u, 0u, 0u, 0u};
  if (live) v = *reinterpret_cast<const u32x4*>(p);
  return __builtin_bit_cast(bf16x8, v);
}

// NG: 16-wide groups of R a workgroup computes; KI: 32-wide pieces of K a
// wave's step. A load takes 64 contiguous bytes of a row (four lanes); the
// next step's are issued before this one's products. Lanes whose row names
// another adapter load the first row that names this one, and lanes past R the
// last row of A: their sums are dropped.
template <int NG, int KI>
__global__ void __launch_bounds__(kShThreads)
k_lora_shrink(const uint16_t* __restrict__ x, int64_t ldx, int T, int K, const uint16_t* __restrict__ a, int L, int R,
              const int32_t* __restrict__ adapter, const float* __restrict__ scale, float* __restrict__ h) {
  __shared__ f32x4 part[kShWaves][NG][kWave];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int c = lane % 16, kq = lane / 16;
  const int64_t t0 = (int64_t)blockIdx.x * 16;
  const int r0 = blockIdx.z * 16 * NG;
  const int ad = lora_row_adapter(adapter, t0, T, L, c);
  uint32_t left = lora_rows(ad >= 0);
  int skip = blockIdx.y;
  while (left != 0) {
    const int first = __ffs(left) - 1;
    const int l = __builtin_amdgcn_readlane(ad, first);
    const uint32_t mine = lora_rows(ad == l);
    left &= ~mine;
    if (skip-- > 0) continue;
    skip = gridDim.y - 1;
    constexpr int kStep = 32 * KI;
    const int steps = (K + kStep - 1) / kStep;
    const uint16_t* xp = x + (t0 + (ad == l ? c : first)) * ldx + 8 * kq;
    const uint16_t* ap[NG];
#pragma unroll
    for (int g = 0; g < NG; ++g) ap[g] = a + ((size_t)l * R + min(r0 + 16 * g + c, R - 1)) * K + 8 * kq;
    f32x4 acc[NG];
    bf16x8 xv[2][KI], av[2][NG][KI];
#pragma unroll
    for (int g = 0; g < NG; ++g) acc[g] = {0.f, 0.f, 0.f, 0.f};
    const auto load = [&](int to, int step) {
      const int k0 = kStep * step;
      if (k0 + kStep <= K) {
#pragma unroll
        for (int i = 0; i < KI; ++i) {
          xv[to][i] = load8(xp + k0 + 32 * i, true);
#pragma unroll
          for (int g = 0; g < NG; ++g) av[to][g][i] = load8(ap[g] + k0 + 32 * i, true);
        }
      } else {
#pragma unroll
        for (int i = 0; i < KI; ++i) {
          const bool in = k0 + 32 * i + 8 * kq < K;
          xv[to][i] = load8(xp + k0 + 32 * i, in);
#pragma unroll
          for (int g = 0; g < NG; ++g) av[to][g][i] = load8(ap[g] + k0 + 32 * i, in);
        }
      }
    };
    const auto multiply = [&](int from) {
#pragma unroll
      for (int i = 0; i < KI; ++i)
#pragma unroll
        for (int g = 0; g < NG; ++g)
          acc[g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv[from][i], av[from][g][i], acc[g], 0, 0, 0);
    };
    int s = wave;
    if (s < steps) load(0, s);
    while (s < steps) {
      if (s + kShWaves < steps) load(1, s + kShWaves);
      multiply(0);
      s += kShWaves;
      if (s >= steps) break;
      if (s + kShWaves < steps) load(0, s + kShWaves);
      multiply(1);
      s += kShWaves;
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) part[wave][g][lane] = acc[g];
    __syncthreads();
    if (wave < NG) {
      f32x4 sum = part[0][wave][lane];
#pragma unroll
      for (int w = 1; w < kShWaves; ++w) {
        const f32x4 o = part[w][wave][lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] += o[i];
      }
      const int r = r0 + 16 * wave + c;
      const float f = scale[l];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r < R && ((mine >> (4 * kq + i)) & 1)) h[(t0 + 4 * kq + i) * R + r] = f * sum[i];
    }
    __syncthreads();
  }
}

__device__ __forceinline__ void fma8(float& s, const u32x4& p, const u32x4& q) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(bf16_lo(p[i]), bf16_lo(q[i]), s);
    s = fmaf(bf16_hi(p[i]), bf16_hi(q[i]), s);
  }
}

// Few rows, one launch: a workgroup owns a row and 512 columns. Its waves
// compute the row's R inner sums, a wave per sum (whole lines of A, 8 values a
// lane and load; each workgroup of a row does it again, from L2), then a
// thread per column multiplies them with its row of B, which is on its way
// from the start. PIECES: 16-byte pieces of B a thread keeps (R <= 8 PIECES).
template <bool BF16, int PIECES>
__global__ void __launch_bounds__(kFewThreads)
k_lora_few(const void* base, int64_t ldb, const uint16_t* __restrict__ x, int64_t ldx, int K, int N,
           const uint16_t* __restrict__ a, const uint16_t* __restrict__ b, int L, int R,
           const int32_t* __restrict__ adapter, const float* __restrict__ scale, void* out, int64_t ldo) {
  __shared__ float hs[8 * PIECES];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t t = blockIdx.y;
  const int n = blockIdx.x * kFewThreads + threadIdx.x;
  const int l = adapter[t];
  const bool has = (uint32_t)l < (uint32_t)L;
  uint32_t bits = 0;                           // base's element
  if (n < N) {
    if constexpr (BF16) bits = static_cast<const uint16_t*>(base)[t * ldb + n];
    else bits = static_cast<const uint32_t*>(base)[t * ldb + n];
  }
  if (has) {
    u32x4 bv[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      bv[i] = {0u, 0u, 0u, 0u};
      if (n < N && 8 * i < R) bv[i] = *reinterpret_cast<const u32x4*>(b + ((size_t)l * N + n) * R + 8 * i);
    }
    const uint16_t* xr = x + t * ldx;
    for (int r = wave; r < R; r += 2 * kFewWaves) {
      // two sums at a time: r and r + kFewWaves
      const bool two = r + kFewWaves < R;
      const uint16_t* a0 = a + ((size_t)l * R + r) * K;
      const uint16_t* a1 = two ? a0 + (size_t)kFewWaves * K : a0;
      float s0 = 0.0f, s1 = 0.0f;
#pragma unroll 4
      for (int64_t k = 8 * lane; k < K; k += 8 * kWave) {
        const u32x4 xv = *reinterpret_cast<const u32x4*>(xr + k);
        fma8(s0, *reinterpret_cast<const u32x4*>(a0 + k), xv);
        fma8(s1, *reinterpret_cast<const u32x4*>(a1 + k), xv);
      }
      s0 = wave_sum(s0);
      s1 = wave_sum(s1);
      if (lane == 0) {
        hs[r] = scale[l] * s0;
        if (two) hs[r + kFewWaves] = scale[l] * s1;
      }
    }
    __syncthreads();
    float d = 0.0f;
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      if (8 * i < R) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          d = fmaf(bf16_lo(bv[i][q]), hs[8 * i + 2 * q], d);
          d = fmaf(bf16_hi(bv[i][q]), hs[8 * i + 2 * q + 1], d);
        }
      }
    }
    if constexpr (BF16) bits = __builtin_bit_cast(uint16_t, (__bf16)(bf16_to_f32((uint16_t)bits) + d));
    else bits = __float_as_uint(__uint_as_float(bits) + d);
  }
  if (n < N) {
    if constexpr (BF16) static_cast<uint16_t*>(out)[t * ldo + n] = (uint16_t)bits;
    else static_cast<uint32_t*>(out)[t * ldo + n] = bits;
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
  // the lane's row t0 + c, columns n0 + 16 j + 4 kq ..: base is on its way before the products
  const bool row = t0 + c < T;
  const int n1 = n0 + 4 * kq;
  f32x4 v[kAddTiles];
  u32x2 w[kAddTiles];
#pragma unroll
  for (int j = 0; j < kAddTiles; ++j) {
    const int n = n1 + 16 * j;
    v[j] = {0.f, 0.f, 0.f, 0.f};
    w[j] = {0u, 0u};
    if (!row) continue;
    if constexpr (BF16) {
      const uint16_t* s = static_cast<const uint16_t*>(base) + (t0 + c) * ldb + n;
      if (vec && n + 3 < N) {
        w[j] = *reinterpret_cast<const u32x2*>(s);
      } else {
        uint32_t e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = n + i < N ? s[i] : 0u;
        w[j] = {e[0] | e[1] << 16, e[2] | e[3] << 16};
      }
    } else {
      const float* s = static_cast<const float*>(base) + (t0 + c) * ldb + n;
      if (vec && n + 3 < N) {
        v[j] = *reinterpret_cast<const f32x4*>(s);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = n + i < N ? s[i] : 0.0f;
      }
    }
  }
  f32x4 acc[kAddTiles];
#pragma unroll
  for (int j = 0; j < kAddTiles; ++j) acc[j] = {0.f, 0.f, 0.f, 0.f};
  lora_expand<kAddTiles>(b, N, R, h, t0, T, n0, ad, lane, acc);
  if (!row) return;
#pragma unroll
  for (int j = 0; j < kAddTiles; ++j) {
    const int n = n1 + 16 * j;
    if constexpr (BF16) {
      uint16_t* d = static_cast<uint16_t*>(out) + (t0 + c) * ldo + n;
      if (ad >= 0)
        w[j] = {pack_bf16x2(bf16_lo(w[j][0]) + acc[j][0], bf16_hi(w[j][0]) + acc[j][1]),
                pack_bf16x2(bf16_lo(w[j][1]) + acc[j][2], bf16_hi(w[j][1]) + acc[j][3])};
      if (vec && n + 3 < N) {
        *reinterpret_cast<u32x2*>(d) = w[j];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < N) d[i] = (uint16_t)(w[j][i / 2] >> (16 * (i % 2)));
      }
    } else {
      float* d = static_cast<float*>(out) + (t0 + c) * ldo + n;
      if (ad >= 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] += acc[j][i];
      }
      if (vec && n + 3 < N) {
        *reinterpret_cast<f32x4*>(d) = v[j];
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < N) d[i] = v[j][i];
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
    k_lora_shrink<1, 4><<<dim3(cdiv(T, 16), y, 1), kShThreads, 0, st>>>(x, ldx, T, K, a, L, R, adapter, scale, h);
  else if (R <= 32)
    k_lora_shrink<2, 4><<<dim3(cdiv(T, 16), y, 1), kShThreads, 0, st>>>(x, ldx, T, K, a, L, R, adapter, scale, h);
  else
    k_lora_shrink<4, 2><<<dim3(cdiv(T, 16), y, cdiv(R, 64)), kShThreads, 0, st>>>(x, ldx, T, K, a, L, R, adapter, scale,
                                                                              h);
  return hipGetLastError();
}

bool lora_few(int T, int R) { return T <= 64 && R <= 64; }

hipError_t launch_lora_few(const void* base, bool bf16, int64_t ldb, const uint16_t* x, int64_t ldx, int T, int K,
                           int N, const uint16_t* a, const uint16_t* b, int L, int R, const int32_t* adapter,
                           const float* scale, void* out, int64_t ldo, hipStream_t st) {
  const dim3 grid(cdiv(N, kFewThreads), T);
#define I8H_FEW(TYPE, PIECES)                                                                                 \
  k_lora_few<TYPE, PIECES><<<grid, kFewThreads, 0, st>>>(base, ldb, x, ldx, K, N, a, b, L, R, adapter, scale, out, ldo)
  if (bf16) {
    if (R <= 16) I8H_FEW(true, 2);
    else if (R <= 32) I8H_FEW(true, 4);
    else I8H_FEW(true, 8);
  } else {
    if (R <= 16) I8H_FEW(false, 2);
    else if (R <= 32) I8H_FEW(false, 4);
    else I8H_FEW(false, 8);
  }
#undef I8H_FEW
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
