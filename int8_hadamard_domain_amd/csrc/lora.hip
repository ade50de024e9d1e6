// Low-rank adapters of many requests beside a shared projection.
//   h[t, r]   = scale[l] * sum_k A[l][r, k] x[t, k],  l = adapter[t]
//   out[t, n] = base[t, n] + sum_r B[l][n, r] h[t, r]
//
// Kernels
//   k_lora_few     few rows: both products in one launch, on the vector ALU
//   k_lora_shrink  h, in slices of K
//   k_lora_add     out
//
// The latter two run on v_mfma_f32_16x16x32_bf16 with a row of the batch per
// matrix row (or column), so what an adapter holds reaches no row but its own:
// values of rows that name another adapter are computed and dropped. h is
// float32; the second product takes it as the sum of three bf16 values (8
// significand bits each, the split is exact), so nothing is rounded between
// the products.

#include <algorithm>

#include "common.hpp"
#include "launch.hpp"
#include "lora.hpp"
#include "xlane.hpp"

namespace i8h {

namespace {

constexpr int kShWaves = 4;                    // the shrink kernel: rows and K of a stage
constexpr int kShThreads = kWave * kShWaves;
constexpr int kShRows = 64;
constexpr int kShK = 256;
constexpr int kFewWaves = 8;
constexpr int kFewThreads = kWave * kFewWaves;
constexpr int kAddThreads = 256;               // the add kernel: rows and columns of a step
constexpr int kAddRows = 32;
constexpr int kAddCols = 256;

// h of 64 rows, 16 NG columns of R and a slice of K, for the adapters that the
// rows name (every gridDim.z / rgroups-th of them, from its own on). Stages of
// 256 of K go through LDS, whole lines a row, the next one's loads in flight
// behind this one's products; a wave takes a quarter of a stage's K for all 64
// rows, so that it reads each operand once, and the four waves' sums meet in
// LDS. 16-byte piece p of a row lies at p ^ (row % 16): the fragment reads of
// 16 rows take all banks. Rows that name another adapter keep what LDS held,
// and lanes past R the last row of A: their sums are dropped.
template <int NG>
__global__ void __launch_bounds__(kShThreads)
k_lora_shrink(const uint16_t* __restrict__ x, int64_t ldx, int T, int K, const uint16_t* __restrict__ a, int L, int R,
              const int32_t* __restrict__ adapter, const float* __restrict__ scale, int rgroups,
              float* __restrict__ h) {
  constexpr int kPieces = kShK / 8;                          // of a row and stage
  constexpr int kXL = kShRows * kPieces / kShThreads;        // loads a thread and stage
  constexpr int kAL = 16 * NG * kPieces / kShThreads;
  constexpr int kStageBytes = (kShRows + 16 * NG) * kShK * 2, kSumBytes = kShWaves * 4 * NG * kWave * 16;
  __shared__ __align__(16) uint8_t sm[kStageBytes > kSumBytes ? kStageBytes : kSumBytes];
  u32x4* xs = reinterpret_cast<u32x4*>(sm);                  // [row][piece]
  u32x4* as = xs + kShRows * kPieces;
  f32x4* sums = reinterpret_cast<f32x4*>(sm);                // [wave][tile][lane]
  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c = lane % 16, kq = lane / 16;
  const int64_t t0 = (int64_t)blockIdx.x * kShRows;
  const int r0 = (blockIdx.z % rgroups) * 16 * NG, every = gridDim.z / rgroups;
  const int all = (K + kShK - 1) / kShK, slices = gridDim.y;
  const int s0 = (int)((int64_t)all * blockIdx.y / slices), s1 = (int)((int64_t)all * (blockIdx.y + 1) / slices);
  const int piece = tid % kPieces, row0 = tid / kPieces;     // a thread's rows: row0 + kShThreads / kPieces * j
  constexpr int kRowStep = kShThreads / kPieces;
  int ad = t0 + lane < T ? adapter[t0 + lane] : -1;          // lane: a row of the tile
  ad = (uint32_t)ad < (uint32_t)L ? ad : -1;
  uint64_t left = __ballot(ad >= 0);
  int skip = blockIdx.z / rgroups;
  while (left != 0) {
    const int l = __builtin_amdgcn_readlane(ad, __ffsll((unsigned long long)left) - 1);
    const uint64_t mine = __ballot(ad == l);
    left &= ~mine;
    if (skip-- > 0) continue;
    skip = every - 1;
    const uint16_t* xp = x + (t0 + row0) * ldx + 8 * piece;
    const uint16_t* ap = a + (size_t)l * R * K + 8 * piece;
    u32x4 xr[kXL], ar[kAL];
    const auto load = [&](int s) {
      const bool in = kShK * s + 8 * piece < K;
#pragma unroll
      for (int j = 0; j < kXL; ++j) {
        xr[j] = {0u, 0u, 0u, 0u};
        if (in && ((mine >> (row0 + kRowStep * j)) & 1))
          xr[j] = *reinterpret_cast<const u32x4*>(xp + (int64_t)kRowStep * j * ldx + kShK * s);
      }
#pragma unroll
      for (int j = 0; j < kAL; ++j) {
        const int r = min(r0 + row0 + kRowStep * j, R - 1);
        ar[j] = {0u, 0u, 0u, 0u};
        if (in) ar[j] = *reinterpret_cast<const u32x4*>(ap + (size_t)r * K + kShK * s);
      }
    };
    f32x4 acc[4][NG];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int g = 0; g < NG; ++g) acc[i][g] = {0.f, 0.f, 0.f, 0.f};
    load(s0);
    for (int s = s0; s < s1; ++s) {
#pragma unroll
      for (int j = 0; j < kXL; ++j) {
        const int r = row0 + kRowStep * j;
        xs[r * kPieces + (piece ^ (r % 16))] = xr[j];
      }
#pragma unroll
      for (int j = 0; j < kAL; ++j) {
        const int r = row0 + kRowStep * j;
        as[r * kPieces + (piece ^ (r % 16))] = ar[j];
      }
      __syncthreads();
      if (s + 1 < s1) load(s + 1);
#pragma unroll
      for (int q = 0; q < kPieces / 4 / kShWaves; ++q) {
        const int p = 4 * (kPieces / 4 / kShWaves * wave + q) + kq;
        bf16x8 av[NG];
#pragma unroll
        for (int g = 0; g < NG; ++g) av[g] = __builtin_bit_cast(bf16x8, as[(16 * g + c) * kPieces + (p ^ c)]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bf16x8 xv = __builtin_bit_cast(bf16x8, xs[(16 * i + c) * kPieces + (p ^ c)]);
#pragma unroll
          for (int g = 0; g < NG; ++g) acc[i][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv, av[g], acc[i][g], 0, 0, 0);
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int g = 0; g < NG; ++g) sums[(wave * 4 * NG + i * NG + g) * kWave + lane] = acc[i][g];
    __syncthreads();
    // wave w adds up the tiles of rows 16 w .. 16 w + 15
    const float f = scale[l];
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      f32x4 sum = sums[(wave * NG + g) * kWave + lane];
#pragma unroll
      for (int w = 1; w < kShWaves; ++w) {
        const f32x4 o = sums[(w * 4 * NG + wave * NG + g) * kWave + lane];
#pragma unroll
        for (int i = 0; i < 4; ++i) sum[i] += o[i];
      }
      const int r = r0 + 16 * g + c;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 16 * wave + 4 * kq + i;
        if (r < R && ((mine >> row) & 1)) h[((int64_t)blockIdx.y * T + t0 + row) * R + r] = f * sum[i];
      }
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

// Four elements of a row of base or out, in float32 or as packed bf16.
template <bool BF16>
struct Quad {
  f32x4 f;
  u32x2 b;
  __device__ __forceinline__ void load(const void* p, int64_t at, int n, int N, bool vec) {
    if constexpr (BF16) {
      const uint16_t* s = static_cast<const uint16_t*>(p) + at;
      if (vec && n + 3 < N) {
        b = *reinterpret_cast<const u32x2*>(s);
      } else {
        uint32_t e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = n + i < N ? s[i] : 0u;
        b = {e[0] | e[1] << 16, e[2] | e[3] << 16};
      }
    } else {
      const float* s = static_cast<const float*>(p) + at;
      if (vec && n + 3 < N) {
        f = *reinterpret_cast<const f32x4*>(s);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = n + i < N ? s[i] : 0.0f;
      }
    }
  }
  __device__ __forceinline__ void add(const f32x4& d) {
    if constexpr (BF16) {
      b = {pack_bf16x2(bf16_lo(b[0]) + d[0], bf16_hi(b[0]) + d[1]),
           pack_bf16x2(bf16_lo(b[1]) + d[2], bf16_hi(b[1]) + d[3])};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) f[i] += d[i];
    }
  }
  __device__ __forceinline__ void store(void* p, int64_t at, int n, int N, bool vec) const {
    if constexpr (BF16) {
      uint16_t* d = static_cast<uint16_t*>(p) + at;
      if (vec && n + 3 < N) {
        *reinterpret_cast<u32x2*>(d) = b;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < N) d[i] = (uint16_t)(b[i / 2] >> (16 * (i % 2)));
      }
    } else {
      float* d = static_cast<float*>(p) + at;
      if (vec && n + 3 < N) {
        *reinterpret_cast<f32x4*>(d) = f;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < N) d[i] = f[i];
      }
    }
  }
};

// out of 32 rows and `steps` times 256 columns: the slices of h are added up
// once a workgroup and lie in LDS in three bf16 parts; a wave goes through its
// 64 columns of each step with the next step's base on its way.
template <bool BF16>
__global__ void __launch_bounds__(kAddThreads)
k_lora_add(const void* base, int64_t ldb, int T, int N, const uint16_t* __restrict__ b, int L, int R,
           const int32_t* __restrict__ adapter, const float* __restrict__ h, int slices, int steps, void* out,
           int64_t ldo, bool vec) {
  extern __shared__ __align__(16) uint8_t sm[];
  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c = lane % 16, kq = lane / 16;
  const int64_t t0 = (int64_t)blockIdx.x * kAddRows;
  int ad[2];
  ad[0] = lora_row_adapter(adapter, t0, T, L, c);
  ad[1] = lora_row_adapter(adapter, t0, T, L, 16 + c);
  int n0 = blockIdx.y * steps * kAddCols + 64 * wave;
  Quad<BF16> now[2][4], next[2][4];
  const auto load = [&](Quad<BF16> (&q)[2][4], int n1) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (t0 + 16 * m + c < T)
          q[m][j].load(base, (t0 + 16 * m + c) * ldb + n1 + 16 * j + 4 * kq, n1 + 16 * j + 4 * kq, N, vec);
  };
  load(next, n0);
  const int ld = lora_split_stride(R);
  lora_split_rows<kAddRows, kAddThreads>(h, slices, T, R, adapter, L, t0, sm, ld, tid);
  __syncthreads();
  const uint32_t rows[2] = {lora_rows(ad[0] >= 0), lora_rows(ad[1] >= 0)};
  for (int s = 0; s < steps && n0 < N; ++s, n0 += kAddCols) {
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) now[m][j] = next[m][j];
    if (s + 1 < steps && n0 + kAddCols < N) load(next, n0 + kAddCols);
    uint32_t left[2] = {rows[0], rows[1]};
    while ((left[0] | left[1]) != 0) {
      const int l = left[0] != 0 ? __builtin_amdgcn_readlane(ad[0], __ffs(left[0]) - 1)
                                 : __builtin_amdgcn_readlane(ad[1], __ffs(left[1]) - 1);
      left[0] &= ~lora_rows(ad[0] == l);
      left[1] &= ~lora_rows(ad[1] == l);
      f32x4 d[2][4];
      lora_products<2, 4>(b + (size_t)l * N * R, N, R, sm, ld, n0, lane, d);
      // the rows of other adapters keep what they have, whatever this one holds
#pragma unroll
      for (int m = 0; m < 2; ++m)
        if (ad[m] == l) {
#pragma unroll
          for (int j = 0; j < 4; ++j) now[m][j].add(d[m][j]);
        }
    }
#pragma unroll
    for (int m = 0; m < 2; ++m)
      if (t0 + 16 * m + c < T) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          now[m][j].store(out, (t0 + 16 * m + c) * ldo + n0 + 16 * j + 4 * kq, n0 + 16 * j + 4 * kq, N, vec);
      }
  }
}

}  // namespace

int lora_slices(int T) { return std::max(1, std::min(8, 256 / ((T - 1) / kShRows + 1))); }

hipError_t launch_lora_shrink(const uint16_t* x, int64_t ldx, int T, int K, const uint16_t* a, int L, int R,
                              const int32_t* adapter, const float* scale, float* h, int* slices, hipStream_t st) {
  *slices = std::min(lora_slices(T), cdiv(K, kShK));
  // while rows are few, workgroups of their own for up to 16 of a tile's adapters
  const int spread = T <= 1024 ? std::min({16, T, L}) : 1;
  const int rgroups = R <= 64 ? 1 : cdiv(R, 64);
  const dim3 grid(cdiv(T, kShRows), *slices, rgroups * spread);
#define I8H_SHRINK(NG) \
  k_lora_shrink<NG><<<grid, kShThreads, 0, st>>>(x, ldx, T, K, a, L, R, adapter, scale, rgroups, h)
  if (R <= 16) I8H_SHRINK(1);
  else if (R <= 32) I8H_SHRINK(2);
  else I8H_SHRINK(4);
#undef I8H_SHRINK
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
                           const int32_t* adapter, const float* h, int slices, void* out, int64_t ldo,
                           hipStream_t st) {
  const uintptr_t unit = bf16 ? 8 : 16;   // four elements
  const bool vec = reinterpret_cast<uintptr_t>(base) % unit == 0 && reinterpret_cast<uintptr_t>(out) % unit == 0 &&
                   ldb % 4 == 0 && ldo % 4 == 0;
  const int tiles = cdiv(T, kAddRows), cols = cdiv(N, kAddCols);
  const int steps = (int)std::max<int64_t>(1, std::min<int64_t>(4, (int64_t)tiles * cols / 512));
  const dim3 grid(tiles, cdiv(cols, steps));
  const size_t lds = (size_t)3 * kAddRows * lora_split_stride(R);
  if (bf16)
    k_lora_add<true><<<grid, kAddThreads, lds, st>>>(base, ldb, T, N, b, L, R, adapter, h, slices, steps, out, ldo,
                                                     vec);
  else
    k_lora_add<false><<<grid, kAddThreads, lds, st>>>(base, ldb, T, N, b, L, R, adapter, h, slices, steps, out, ldo,
                                                      vec);
  return hipGetLastError();
}

}  // namespace i8h
