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
#include <type_traits>

#include "common.hpp"
#include "launch.hpp"
#include "lora.hpp"
#include "xlane.hpp"

namespace i8h {

namespace {

constexpr int kShWaves = 4;                    // the shrink kernel: rows and K of a stage
constexpr int kShThreads = kWave * kShWaves;
constexpr int kShRows = 64;
constexpr int kShK = 128;
constexpr int kFewWaves = 16;
constexpr int kFewThreads = kWave * kFewWaves;
constexpr int kAddThreads = 256;               // the add kernel: rows and columns of a step
constexpr int kAddCols = 256;
constexpr int kAddBRow = 80;                   // bytes of LDS of a row of B, 32 of R: 64 and 16 of padding

// Workgroups are dealt to the XCDs in turn: the i-th of n (a multiple of their
// number) takes place i % kXcds * n / kXcds + i / kXcds, so that each XCD's L2
// sees neighbouring ones.
constexpr int kXcds = 8;
__device__ __forceinline__ int xcd_run(int i, int n) { return i % kXcds * (n / kXcds) + i / kXcds; }

// 16 bytes at a uniform address and a lane's byte offset (32 bits: the entry
// points bound row distances and K).
__device__ __forceinline__ u32x4 load16(const void* p, uint32_t off) {
  return *reinterpret_cast<const u32x4*>(static_cast<const uint8_t*>(p) + off);
}

// h of 64 rows, 16 NG columns of R and a slice of K, for the adapters that the
// rows name (each `every`-th of them, from its own on). Stages of
// 128 of K go through LDS, whole lines a row, the next two's loads in flight
// behind this one's products; a wave takes a quarter of a stage's K for all 64
// rows, so that it reads each operand once, and the four waves' sums meet in
// LDS. 16-byte piece p of a row lies at p ^ (row % 16): the fragment reads of
// 16 rows take all banks. Rows that name another adapter are zero,
// and lanes past R hold the last row of A: their sums are dropped. The tiles start
// at different stages: rows lie a power of two apart more often than not, and
// all tiles at the same piece of K would ask the same L2 channels. The next
// adapter's first loads are issued before this one's sums are added up.
// 11.3 us for 2048 rows of K = 4096 and rank 64, five requests: 1.7 TB/s; 13.7 us
// for 8191 rows of K = 2048 and rank 32. Bound by the chain adapter, first loads,
// four or eight stages, sums in LDS: the loads of two stages in flight are all
// that the registers hold.
template <int NG>
__global__ void __launch_bounds__(kShThreads, 2)
k_lora_shrink(const uint16_t* __restrict__ x, int64_t ldx, int T, int K, const uint16_t* __restrict__ a, int L, int R,
              const int32_t* __restrict__ adapter, const float* __restrict__ scale, int slices, int rgroups, int every,
              int wgs, float* __restrict__ h) {
  constexpr int kPieces = kShK / 8;                          // of a row and stage
  constexpr int kXL = kShRows * kPieces / kShThreads;        // loads a thread and stage
  constexpr int kAL = 16 * NG * kPieces / kShThreads;
  constexpr int kStageBytes = (kShRows + 16 * NG) * kShK * 2, kSumBytes = kShWaves * 2 * NG * kWave * 16;
  __shared__ __align__(16) uint8_t sm[kStageBytes > kSumBytes ? kStageBytes : kSumBytes];
  u32x4* xs = reinterpret_cast<u32x4*>(sm);                  // [row][piece]
  u32x4* as = xs + kShRows * kPieces;
  f32x4* sums = reinterpret_cast<f32x4*>(sm);                // [wave][tile][lane]
  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c = lane % 16, kq = lane / 16;
  // the workgroup's tile, slice, group of R and first adapter
  int wg = xcd_run(blockIdx.x, gridDim.x);
  if (wg >= wgs) return;
  const int slice = wg % slices;
  wg /= slices;
  const int r0 = wg % rgroups * 16 * NG;
  wg /= rgroups;
  int skip = wg % every;
  const int tile = wg / every;
  const int64_t t0 = (int64_t)tile * kShRows;
  const int all = (K + kShK - 1) / kShK;
  const int s0 = (int)((int64_t)all * slice / slices), stages = (int)((int64_t)all * (slice + 1) / slices) - s0;
  const int turn = tile % stages;
  const int piece = tid % kPieces, row0 = tid / kPieces;     // a thread's rows: row0 + kShThreads / kPieces * j
  constexpr int kRowStep = kShThreads / kPieces;
  const uint16_t* xt = x + t0 * ldx;
  int ad = t0 + lane < T ? adapter[t0 + lane] : -1;          // lane: a row of the tile
  ad = (uint32_t)ad < (uint32_t)L ? ad : -1;
  uint64_t left = __ballot(ad >= 0), mine = 0;
  int l = -1;
  // the next of the workgroup's adapters, and its rows
  const auto next = [&]() {
    l = -1;
    while (left != 0 && l < 0) {
      const int at = __builtin_amdgcn_readlane(ad, __ffsll((unsigned long long)left) - 1);
      const uint64_t of = __ballot(ad == at);
      left &= ~of;
      if (skip-- > 0) continue;
      skip = every - 1;
      l = at;
      mine = of;
    }
  };
  u32x4 xr[2][kXL], ar[2][kAL];
  const auto load = [&](int to, int i) {
    const int s = s0 + (i + turn < stages ? i + turn : i + turn - stages);
    const bool in = kShK * s + 8 * piece < K;
    const uint16_t* al = a + (size_t)l * R * K;
#pragma unroll
    for (int j = 0; j < kXL; ++j) {
      xr[to][j] = {0u, 0u, 0u, 0u};
      if (in && ((mine >> (row0 + kRowStep * j)) & 1))
        xr[to][j] = load16(xt + kShK * s, 2u * ((uint32_t)(row0 + kRowStep * j) * (uint32_t)ldx + 8u * piece));
    }
#pragma unroll
    for (int j = 0; j < kAL; ++j) {
      const int r = min(r0 + row0 + kRowStep * j, R - 1);
      ar[to][j] = {0u, 0u, 0u, 0u};
      if (in) ar[to][j] = load16(al + kShK * s, 2u * ((uint32_t)r * (uint32_t)K + 8u * piece));
    }
  };
  f32x4 acc[4][NG];
  const auto stage = [&](int from, int s) {
#pragma unroll
    for (int j = 0; j < kXL; ++j) {
      const int r = row0 + kRowStep * j;
      xs[r * kPieces + (piece ^ (r % 16))] = xr[from][j];
    }
#pragma unroll
    for (int j = 0; j < kAL; ++j) {
      const int r = row0 + kRowStep * j;
      as[r * kPieces + (piece ^ (r % 16))] = ar[from][j];
    }
    __syncthreads();
    if (s + 2 < stages) load(from, s + 2);
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
  };
  next();
  float f = 0.0f;
  if (l >= 0) {
    f = scale[l];
    load(0, 0);
    if (stages > 1) load(1, 1);
  }
  while (l >= 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int g = 0; g < NG; ++g) acc[i][g] = {0.f, 0.f, 0.f, 0.f};
    for (int s = 0; s < stages; s += 2) {
      stage(0, s);
      if (s + 1 < stages) stage(1, s + 1);
    }
    // the next adapter's first loads are on their way while this one's sums are added up
    const uint64_t done = mine;
    const float by = f;
    next();
    if (l >= 0) {
      f = scale[l];
      load(0, 0);
      if (stages > 1) load(1, 1);
    }
    // the waves' sums, 32 rows at a time
#pragma unroll
    for (int half = 0; half < 2; ++half) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int g = 0; g < NG; ++g) sums[((wave * 2 + i) * NG + g) * kWave + lane] = acc[2 * half + i][g];
      __syncthreads();
      for (int tile = wave; tile < 2 * NG; tile += kShWaves) {
        f32x4 sum = sums[tile * kWave + lane];
#pragma unroll
        for (int w = 1; w < kShWaves; ++w) {
          const f32x4 o = sums[(w * 2 * NG + tile) * kWave + lane];
#pragma unroll
          for (int i = 0; i < 4; ++i) sum[i] += o[i];
        }
        const int r = r0 + 16 * (tile % NG) + c;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 16 * (2 * half + tile / NG) + 4 * kq + i;
          if (r < R && ((done >> row) & 1)) h[((int64_t)slice * T + t0 + row) * R + r] = by * sum[i];
        }
      }
      __syncthreads();
    }
  }
}

__device__ __forceinline__ void fma8(float& s, const u32x4& p, const u32x4& q) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(bf16_lo(p[i]), bf16_lo(q[i]), s);
    s = fmaf(bf16_hi(p[i]), bf16_hi(q[i]), s);
  }
}

// Few rows, one launch: a workgroup owns a row and 1024 columns. Its waves
// compute the row's R inner sums, SUMS of them at a time each (whole lines of A,
// 8 values a lane and load; each workgroup of a row does it again, from L2). A
// wave's 64 columns of B lie one behind the other in memory and are on their way
// from the start, 64 pieces of 16 bytes a load; a piece's part of the product goes
// to its column by way of LDS. (A column a lane takes the load path 64 accesses an
// instruction: 64 rows of 64 requests, 2048 x 4096 bf16, rank 64 18.4 against 15.7
// us, 16 rows 15.7 against 12.6. Up to rank 16 that is little, and LDS a detour:
// one row 3.3 against 3.7 us.) 16 waves: with 8 of twice the sums one row of rank
// 16 takes 3.1 us, 64 rows 6.4 in place of 5.5, of rank 64 25 in place of 18. One
// row is a launch and two loads that depend on each other; more read A once a row
// and 1024 columns from L2. PIECES: 16-byte pieces of B a lane keeps (R <= 8 PIECES).
template <bool BF16, int PIECES, int SUMS>
__global__ void __launch_bounds__(kFewThreads)
k_lora_few(const void* base, int64_t ldb, const uint16_t* __restrict__ x, int64_t ldx, int K, int N,
           const uint16_t* __restrict__ a, const uint16_t* __restrict__ b, int L, int R,
           const int32_t* __restrict__ adapter, const float* __restrict__ scale, void* out, int64_t ldo) {
  constexpr bool kTurn = PIECES > 2;
  constexpr int kParts = kTurn ? kWave * PIECES * 9 / 8 : 1;       // a float of padding after each eight
  __shared__ __align__(16) float hs[8 * PIECES];
  __shared__ float parts[kFewWaves][kParts];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t t = blockIdx.y;
  const int n0 = blockIdx.x * kFewThreads + kWave * wave, n = n0 + lane;
  const int l = adapter[t];
  const bool has = (uint32_t)l < (uint32_t)L;
  uint32_t bits = 0;                           // base's element
  if (n < N) {
    if constexpr (BF16) bits = static_cast<const uint16_t*>(base)[t * ldb + n];
    else bits = static_cast<const uint32_t*>(base)[t * ldb + n];
  }
  if (has) {
    const int per = R / 8;                     // pieces a column
    const int pieces = max(0, min(kWave, N - n0)) * per;
    const u32x4* bl = reinterpret_cast<const u32x4*>(b + ((size_t)l * N + min(n0, N)) * R);
    u32x4 bv[PIECES];
#pragma unroll
    for (int i = 0; i < PIECES; ++i) {
      const int at = kTurn ? kWave * i + lane : per * lane + i;
      bv[i] = {0u, 0u, 0u, 0u};
      if (at < pieces && (kTurn || i < per)) bv[i] = bl[at];
    }
    const uint16_t* xr = x + t * ldx;
    for (int r = wave; r < R; r += SUMS * kFewWaves) {
      // r, r + kFewWaves, .. (past R: the first again, dropped)
      const uint16_t* ar[SUMS];
      float sum[SUMS];
#pragma unroll
      for (int i = 0; i < SUMS; ++i) {
        ar[i] = a + ((size_t)l * R + (r + i * kFewWaves < R ? r + i * kFewWaves : r)) * K;
        sum[i] = 0.0f;
      }
#pragma unroll (SUMS == 1 ? 4 : 2)
      for (int64_t k = 8 * lane; k < K; k += 8 * kWave) {
        const u32x4 xv = *reinterpret_cast<const u32x4*>(xr + k);
#pragma unroll
        for (int i = 0; i < SUMS; ++i) fma8(sum[i], *reinterpret_cast<const u32x4*>(ar[i] + k), xv);
      }
#pragma unroll
      for (int i = 0; i < SUMS; ++i) {
        const float v = wave_sum(sum[i]);
        if (lane == 0 && r + i * kFewWaves < R) hs[r + i * kFewWaves] = scale[l] * v;
      }
    }
    __syncthreads();
    // the products of a piece of B with its part of h
    const auto product = [&](int i, int piece) {
      const f32x4 h0 = *reinterpret_cast<const f32x4*>(hs + 8 * piece);
      const f32x4 h1 = *reinterpret_cast<const f32x4*>(hs + 8 * piece + 4);
      float p = bf16_lo(bv[i][0]) * h0[0];
      p = fmaf(bf16_hi(bv[i][0]), h0[1], p);
      p = fmaf(bf16_lo(bv[i][1]), h0[2], p);
      p = fmaf(bf16_hi(bv[i][1]), h0[3], p);
      p = fmaf(bf16_lo(bv[i][2]), h1[0], p);
      p = fmaf(bf16_hi(bv[i][2]), h1[1], p);
      p = fmaf(bf16_lo(bv[i][3]), h1[2], p);
      return fmaf(bf16_hi(bv[i][3]), h1[3], p);
    };
    float d = 0.0f;
    if constexpr (kTurn) {
      float* mine = parts[wave];
      int piece = lane % per;
      const int step = kWave % per;
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        if (i < per) {
          const int at = kWave * i + lane;
          mine[at + at / 8] = product(i, piece);
          piece = piece + step < per ? piece + step : piece + step - per;
        }
      }
      lora_wave_order();
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const int at = lane * per + i;
        if (i < per) d += mine[at + at / 8];
      }
    } else {
#pragma unroll
      for (int i = 0; i < PIECES; ++i)
        if (i < per) d += product(i, i);
    }
    if constexpr (BF16) bits = __builtin_bit_cast(uint16_t, (__bf16)(bf16_to_f32((uint16_t)bits) + d));
    else bits = __float_as_uint(__uint_as_float(bits) + d);
  }
  if (n < N) {
    if constexpr (BF16) static_cast<uint16_t*>(out)[t * ldo + n] = (uint16_t)bits;
    else static_cast<uint32_t*>(out)[t * ldo + n] = bits;
  }
}

// 16 bytes of a row of base or out, four float32 values or eight bf16. FULL: all there and aligned.
template <bool BF16>
struct Piece {
  static constexpr int kE = BF16 ? 8 : 4;
  u32x4 v;
  template <bool FULL>
  __device__ __forceinline__ void load(const void* p, uint32_t at, int n, int N) {
    if constexpr (FULL) {
      v = load16(p, (16 / kE) * at);
    } else if constexpr (BF16) {
      const uint16_t* s = static_cast<const uint16_t*>(p) + at;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = (n + 2 * i < N ? (uint32_t)s[2 * i] : 0u) | (n + 2 * i + 1 < N ? (uint32_t)s[2 * i + 1] << 16 : 0u);
    } else {
      const uint32_t* s = static_cast<const uint32_t*>(p) + at;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = n + i < N ? s[i] : 0u;
    }
  }
  __device__ __forceinline__ void add(const float* d) {
    const f32x4 d0 = *reinterpret_cast<const f32x4*>(d);
    if constexpr (BF16) {
      const f32x4 d1 = *reinterpret_cast<const f32x4*>(d + 4);
      v = {pack_bf16x2(bf16_lo(v[0]) + d0[0], bf16_hi(v[0]) + d0[1]),
           pack_bf16x2(bf16_lo(v[1]) + d0[2], bf16_hi(v[1]) + d0[3]),
           pack_bf16x2(bf16_lo(v[2]) + d1[0], bf16_hi(v[2]) + d1[1]),
           pack_bf16x2(bf16_lo(v[3]) + d1[2], bf16_hi(v[3]) + d1[3])};
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + d0[i]);
    }
  }
  template <bool FULL>
  __device__ __forceinline__ void store(void* p, uint32_t at, int n, int N) const {
    if constexpr (FULL) {
      *reinterpret_cast<u32x4*>(static_cast<uint8_t*>(p) + (16 / kE) * at) = v;
    } else if constexpr (BF16) {
      uint16_t* d = static_cast<uint16_t*>(p) + at;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (n + i < N) d[i] = (uint16_t)(v[i / 2] >> (16 * (i % 2)));
    } else {
      uint32_t* d = static_cast<uint32_t*>(p) + at;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < N) d[i] = v[i];
    }
  }
};

// out of 16 MT rows and 256 columns, 64 a wave. h is added up over its slices
// once a workgroup and lies in LDS in three bf16 parts. Neighbouring lanes are
// served together only where they take neighbouring bytes, and the matrix
// layouts deal a row to lanes 16 apart; so base and out are loaded and stored
// with 128 bytes of a row on neighbouring lanes, B 64 bytes of a row on four,
// and a wave's own LDS turns B's rows and the products into the other order
// (64 us without, 55 with, of 8191 x 4096 float32 rows: 278 MB at 5.0 TB/s, where
// a copy of 268 MB takes 51 us; 2048 x 2048 bf16 rows of rank 64 9.2 us, 1.8 TB/s,
// bound by the chain of h, B and the products in each workgroup). Four workgroups a
// CU: left alone the compiler takes 129 registers for 16 bf16 rows, and those 2048
// rows with the shrink 22.8 in place of 20.4 us; 32 bf16 rows take 168.
template <bool BF16, int MT>
__global__ void __launch_bounds__(kAddThreads, BF16 && MT == 2 ? 3 : 4)
k_lora_add(const void* base, int64_t ldb, int T, int N, const uint16_t* __restrict__ b, int L, int R,
           const int32_t* __restrict__ adapter, const float* __restrict__ h, int slices, int colgroups, int wgs,
           void* out, int64_t ldo, bool vec) {
  using P = Piece<BF16>;
  constexpr int kNT = BF16 ? 2 : 1, kPasses = 2 / kNT, kCols = 32 * kNT;             // columns a pass: 128 bytes a row
  constexpr int kLpr = kCols / P::kE, kRpc = kWave / kLpr, kRows = 16 * MT;   // lanes a row, rows a load
  constexpr int kChunks = kRows / kRpc;
  extern __shared__ __align__(16) uint8_t sm[];
  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int c = lane % 16, kq = lane / 16;
  const int wg = xcd_run(blockIdx.x, gridDim.x);
  if (wg >= wgs) return;
  const int64_t t0 = (int64_t)(wg / colgroups) * kRows;
  int ad[MT];
  uint32_t rows[MT];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    ad[m] = lora_row_adapter(adapter, t0, T, L, 16 * m + c);
    rows[m] = lora_rows(ad[m] >= 0);
  }
  const int n0 = wg % colgroups * kAddCols + 64 * wave;
  const void* from = static_cast<const uint8_t*>(base) + t0 * ldb * (BF16 ? 2 : 4);
  void* to = static_cast<uint8_t*>(out) + t0 * ldo * (BF16 ? 2 : 4);
  const int ld = lora_split_stride(R);
  uint8_t* own = sm + 3 * kRows * ld + wave * (kCols * kAddBRow);
  // FULL: all of the workgroup's rows and columns are there, and vectors are aligned
  const auto run = [&](auto full) {
    constexpr bool FULL = decltype(full)::value;
    const int row = lane / kLpr, n1 = n0 + P::kE * (lane % kLpr);      // chunk i of pass g: row + kRpc i, n1 + kCols g
    P q[kPasses][kChunks];
#pragma unroll
    for (int g = 0; g < kPasses; ++g)
#pragma unroll
      for (int i = 0; i < kChunks; ++i)
        if (FULL || t0 + row + kRpc * i < T)
          q[g][i].template load<FULL>(from, (uint32_t)(row + kRpc * i) * (uint32_t)ldb + n1 + kCols * g, n1 + kCols * g, N);
    lora_split_rows<kRows, kAddThreads>(h, slices, T, R, 0, R, adapter, L, t0, sm, ld, tid);
    __syncthreads();
#pragma unroll
    for (int g = 0; g < kPasses; ++g) {
      const int ng = n0 + kCols * g, n = n1 + kCols * g;
      f32x4 sum[MT][2 * kNT];
      uint32_t left[MT];
      // 32 of R of the pass's rows of B, a step ahead of their use: an adapter's first while the one before multiplies
      u32x4 w[2 * kNT];
      const auto fetch = [&](int l, int r0) {
        const uint16_t* bl = b + ((size_t)l * N + ng) * R;
#pragma unroll
        for (int i = 0; i < 2 * kNT; ++i) {
          const int nb = 16 * i + lane / 4, r = 8 * (lane % 4);
          w[i] = {0u, 0u, 0u, 0u};
          if ((FULL || ng + nb < N) && r0 + r < R) w[i] = load16(bl + r0, 2u * ((uint32_t)nb * (uint32_t)R + r));
        }
      };
      const auto first = [&]() {
        int l = -1;
#pragma unroll
        for (int m = 0; m < MT; ++m)
          if (l < 0 && left[m] != 0) l = __builtin_amdgcn_readlane(ad[m], __ffs(left[m]) - 1);
        return l;
      };
      const auto products = [&](auto finite) {
#pragma unroll
        for (int m = 0; m < MT; ++m) {
          left[m] = rows[m];
#pragma unroll
          for (int j = 0; j < 2 * kNT; ++j) sum[m][j] = {0.f, 0.f, 0.f, 0.f};
        }
        int ahead = first();
        if (ahead >= 0) fetch(ahead, 0);
        while (ahead >= 0) {
          const int l = ahead;
#pragma unroll
          for (int m = 0; m < MT; ++m) left[m] &= ~lora_rows(ad[m] == l);
          f32x4 d[MT][2 * kNT];
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 2 * kNT; ++j) d[m][j] = {0.f, 0.f, 0.f, 0.f};
          ahead = first();
          for (int r0 = 0; r0 < R; r0 += 32) {
            lora_wave_order();
#pragma unroll
            for (int i = 0; i < 2 * kNT; ++i)
              *reinterpret_cast<u32x4*>(own + (16 * i + lane / 4) * kAddBRow + 16 * (lane % 4)) = w[i];
            lora_wave_order();
            bf16x8 bv[2 * kNT];
#pragma unroll
            for (int j = 0; j < 2 * kNT; ++j)
              bv[j] = *reinterpret_cast<const bf16x8*>(own + (16 * j + c) * kAddBRow + 16 * kq);
            if (r0 + 32 < R) fetch(l, r0 + 32);
            else if (ahead >= 0) fetch(ahead, 0);
            lora_multiply<MT, kNT, decltype(finite)::value>(bv, R, r0, sm, ld, lane, d);
          }
          // the rows of other adapters keep what they have, whatever this one holds
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 2 * kNT; ++j)
#pragma unroll
              for (int i = 0; i < 4; ++i) sum[m][j][i] = ad[m] == l ? d[m][j][i] : sum[m][j][i];
        }
      };
      products(std::false_type{});
      float all = 0.0f;
#pragma unroll
      for (int m = 0; m < MT; ++m) all += lora_total(sum[m]);
      if (__builtin_expect(__ballot(all != all) != 0, 0)) products(std::true_type{});
      // 16 rows at a time through the wave's LDS
      constexpr int kTurn = kCols + 4;         // floats from row to row
      float* turn = reinterpret_cast<float*>(own);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        if (rows[m] != 0) {
          lora_wave_order();
#pragma unroll
          for (int j = 0; j < 2 * kNT; ++j) *reinterpret_cast<f32x4*>(turn + kTurn * c + 16 * j + 4 * kq) = sum[m][j];
          lora_wave_order();
        }
#pragma unroll
        for (int i = m * kChunks / MT; i < (m + 1) * kChunks / MT; ++i) {
          const int r = row + kRpc * i;
          if ((rows[m] >> (r % 16)) & 1) q[g][i].add(turn + kTurn * (r % 16) + P::kE * (lane % kLpr));
          if (FULL || t0 + r < T) q[g][i].template store<FULL>(to, (uint32_t)r * (uint32_t)ldo + n, n, N);
        }
      }
    }
  };
  if (vec && t0 + kRows <= T && wg % colgroups * kAddCols + kAddCols <= N) run(std::true_type{});
  else run(std::false_type{});
}

}  // namespace

// As many slices as make 512 workgroups of the tiles.
constexpr int kShFill = 512;
static int lora_slices(int T) { return std::max(1, std::min(kLoraSlices, kShFill / ((T - 1) / kShRows + 1))); }

// Never less for more rows: slices times rows go up and down with T (4096 rows are 8 slices, 4097 are 7), at most to
// kShFill tiles.
int64_t lora_sums(int T) { return std::min((int64_t)kLoraSlices * T, std::max((int64_t)kShFill * kShRows, (int64_t)T)); }

hipError_t launch_lora_shrink(const uint16_t* x, int64_t ldx, int T, int K, const uint16_t* a, int L, int R,
                              const int32_t* adapter, const float* scale, float* h, int* slices, hipStream_t st) {
  *slices = std::min(lora_slices(T), cdiv(K, kShK));
  // While rows are few, workgroups of their own for several of a tile's adapters. Measured, us with 1, 2, 4 and 16 of
  // them: 1024 rows of 64 requests (rank 32, and the linear with it) -, -, 40.8, 42.7; 2048 rows of five requests (rank 64,
  // and the add) 24.4, 21.3, 22.4, -; 4096 rows of five 32.9, -, 35.3, -.
  const int spread = std::min({T <= 512 ? 8 : T <= 1024 ? 4 : T <= 2048 ? 2 : 1, T, L});
  const int rgroups = R <= 64 ? 1 : cdiv(R, 64);
  const int wgs = cdiv(T, kShRows) * *slices * rgroups * spread, grid = cdiv(wgs, kXcds) * kXcds;
#define I8H_SHRINK(NG)                                                                                            \
  k_lora_shrink<NG><<<grid, kShThreads, 0, st>>>(x, ldx, T, K, a, L, R, adapter, scale, *slices, rgroups, spread, \
                                                 wgs, h)
  if (R <= 16) I8H_SHRINK(1);
  else if (R <= 32) I8H_SHRINK(2);
  else I8H_SHRINK(4);
#undef I8H_SHRINK
  return hipGetLastError();
}

// Few rows of low rank take one launch on the vector unit, which reads A and B once a row: what it costs grows with T R,
// and it does not mind that every row has another adapter; the two kernels work once for each adapter of a tile. Measured
// (2048 x 4096 bf16, 48 adapters), us here and there with as many requests as rows, then with 4 (128 rows: 8) requests:
//    64 rows, rank 16    5.4  24.4     3.8   9.0      and past the border:
//    64 rows, rank 64   15.6  35.0    12.3  11.8      128 rows, rank 64   28.4  36.7    22.3  13.3
//   128 rows, rank 16    8.4  25.2     6.4   9.3      256 rows, rank 32   24.7  28.5    19.2   9.8
//   256 rows, rank 16   13.8  25.7     8.7   8.8      512 rows, rank 8    18.3  29.7    18.5  10.4
bool lora_few(int T, int R) { return T <= 256 && R <= 64 && T * R <= 4096; }

hipError_t launch_lora_few(const void* base, bool bf16, int64_t ldb, const uint16_t* x, int64_t ldx, int T, int K,
                           int N, const uint16_t* a, const uint16_t* b, int L, int R, const int32_t* adapter,
                           const float* scale, void* out, int64_t ldo, hipStream_t st) {
#define I8H_FEW(TYPE, PIECES, SUMS)                                                                                     \
  k_lora_few<TYPE, PIECES, SUMS><<<dim3(cdiv(N, kFewThreads), T), kFewThreads, 0, st>>>(base, ldb, x, ldx, K, N, a, b, L, \
                                                                                        R, adapter, scale, out, ldo)
  if (bf16) {
    if (R <= 16) I8H_FEW(true, 2, 1);
    else if (R <= 32) I8H_FEW(true, 4, 2);
    else I8H_FEW(true, 8, 4);
  } else {
    if (R <= 16) I8H_FEW(false, 2, 1);
    else if (R <= 32) I8H_FEW(false, 4, 2);
    else I8H_FEW(false, 8, 4);
  }
#undef I8H_FEW
  return hipGetLastError();
}

hipError_t launch_lora_add(const void* base, bool bf16, int64_t ldb, int T, int N, const uint16_t* b, int L, int R,
                           const int32_t* adapter, const float* h, int slices, void* out, int64_t ldo,
                           hipStream_t st) {
  const int unit = bf16 ? 8 : 4;          // elements of 16 bytes
  const bool vec = reinterpret_cast<uintptr_t>(base) % 16 == 0 && reinterpret_cast<uintptr_t>(out) % 16 == 0 &&
                   ldb % unit == 0 && ldo % unit == 0;
  const int colgroups = cdiv(N, kAddCols);
  const auto run = [&](auto type, auto mt) {
    constexpr int kRows = 16 * decltype(mt)::value;
    const int wgs = cdiv(T, kRows) * colgroups, grid = cdiv(wgs, kXcds) * kXcds;
    const size_t lds = (size_t)3 * kRows * lora_split_stride(R) + kAddThreads / kWave * (bf16 ? 64 : 32) * kAddBRow;
    k_lora_add<decltype(type)::value, decltype(mt)::value>
        <<<grid, kAddThreads, lds, st>>>(base, ldb, T, N, b, L, R, adapter, h, slices, colgroups, wgs, out, ldo, vec);
  };
  const std::integral_constant<int, 1> one;
  const std::integral_constant<int, 2> two;
  // 16 rows a workgroup while that many make few workgroups: a tile then has half the adapters, one after the other. us
  // with 16 and 32 rows (2048 x 4096 bf16, rank 16, and the shrink): 512 rows of 512 requests 29.3, 40.3, of 4 requests
  // 9.8, 10.6; 2048 rows of 64 requests 22.5, 24.1, of 4 17.7, 18.6; 8191 rows of 64 requests 61.0, 58.5.
  const bool few = (int64_t)cdiv(T, 32) * colgroups <= 1024;
  if (bf16 && few) run(std::true_type{}, one);
  else if (bf16) run(std::true_type{}, two);
  else if (few) run(std::false_type{}, one);
  else run(std::false_type{}, two);
  return hipGetLastError();
}

}  // namespace i8h
