// The dense int8 linear with f16 scales (linear.hip) for batches whose rows
// name low-rank adapters:
//   y[t, n] = sum_g s[n, g] * sum_{k in g} q[n, k] * x[t, k] + sum_r B[l][n, r] h[t, r],  l = adapter[t]
// h comes from the shrink kernel (lora.hip), in slices of K.
//
// A workgroup of eight waves owns 16 MT tokens x 16 NT WN columns. WK waves
// share a wave's columns and split the K groups; the others stand side by side
// along N. A stage is WK groups of K: the tokens' rows go through LDS, whole
// lines a row, BUFS - 1 stages' copies in flight behind this one's products (one
// barrier a stage); each wave streams its codes into registers (64 contiguous
// bytes a row), as far ahead, and decodes them to bf16 (exact) once for all its
// tokens. Per group a wave runs v_mfma_f32_16x16x32_bf16 from zero accumulators
// and folds the sums into its float32 result with the column's scale. The K
// positions of an operand are dealt so that a lane's codes are whole 16-byte
// loads: of the 64 positions 64 j .. of a group's half, lane quarter q holds
// 16 q .. 16 q + 15, and MFMA 2 j + u takes 8 u .. 8 u + 7 of them, of both
// operands alike.
//
// At the end the WK waves' results meet in LDS, each wave taking its share of
// the token tiles, and the adapters' products are added from there: h in three
// bf16 parts (their sum is the float32 value), the rows of other adapters
// dropped after the product.
//
// Measured (4096 x 2048, medians, without the shrink): 16 tokens of rank 16 6.8
// us, 128 tokens 14.0 (both bound by the chain first loads, stages, join,
// adapters), 1024 tokens of rank 32 35.2 us: 498 TFLOP/s. Of its 65,000 cycles
// 8,000 go by before the first products (every CU asks for its first 96 KB at
// once), 11,000 in the join and the adapters; each of the eight stages takes
// 5,500, of which the matrix units need 2,050: the tokens' copies go at 31 bytes
// a clock and CU, as long as the products, and codes of 16 bytes a row at 15.
// Tried at that size and not kept: copies dealt between the products (42.2
// against 40.9 us with the shrink), codes loaded 64 bytes a quad of lanes and
// exchanged between lanes and registers (43.4), the next stage's decoding between
// this one's products with both of these (40.3, and 69.8 against 69.9 at 2048
// tokens), codes through LDS as well (55), two workgroups of four waves a CU (47).
// Up to 32 tokens of low rank the plain linear and lora_add in place on its output
// take less, in a graph and us, this and those with rank 16: 1 token 11.0, 8.5; 16
// tokens 11.4, 9.3; 32 tokens 13.7, 11.3; 64 tokens 14.8, 18.5; 128 tokens 18.6,
// 34.7. Of rank 64: 16 tokens 13.0, 14.0; 64 tokens 16.5, 26.8.

#include <algorithm>
#include <type_traits>

#include "common.hpp"
#include "launch.hpp"
#include "lora.hpp"

namespace i8h {

namespace {

constexpr int kLlRank = 128;                 // of R that the epilogue holds in LDS at a time
constexpr int kLlXcds = 8;

__device__ __forceinline__ bf16x8 ll_decode(uint32_t lo, uint32_t hi) {
  u32x4 p;
  p[0] = pack_bf16x2(sbyte<0>(lo), sbyte<1>(lo));
  p[1] = pack_bf16x2(sbyte<2>(lo), sbyte<3>(lo));
  p[2] = pack_bf16x2(sbyte<0>(hi), sbyte<1>(hi));
  p[3] = pack_bf16x2(sbyte<2>(hi), sbyte<3>(hi));
  return __builtin_bit_cast(bf16x8, p);
}

typedef __attribute__((address_space(3))) void ll_lds_t;

// one 16-byte copy per lane, global (uniform base + 32-bit lane offset) -> LDS
// (M0 = the wave's LDS base; lane l's bytes land at base + 16 l); the kernel
// waits with vmcnt. M0 is a register the compiler reserves: it sets it right
// before its own instructions that read it, and naming it clobbered orders the
// statement against those; the compiler's warning that it does not preserve
// reserved registers is what is wanted here.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ void ll_copy16(uint32_t off, const void* base, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds)
               : "memory", "m0");
}
#pragma clang diagnostic pop
// s_waitcnt vmcnt(n) with expcnt and lgkmcnt unconstrained (gfx9 field layout)
constexpr int ll_vmcnt(int n) { return (n & 15) | (n >> 4) << 14 | (0x7 << 4) | (0xF << 8); }

template <int MT, int NT, int WN, int WAVES, int BUFS>
struct LlShape {
  static constexpr int kThreads = kWave * WAVES, kWk = WAVES / WN;
  static constexpr int kRows = 16 * MT, kCols = 16 * NT * WN;
  static constexpr int kPieces = 16 * kWk;                              // 16-byte pieces of a row and stage
  static constexpr int kLoads = kRows * kPieces / kThreads;           // a thread and stage
  static constexpr int kStage = kPieces == 32 ? kRows / 2 * 1040 : kRows * (16 * kPieces + 16);   // bytes
  static constexpr int kJoin = WAVES * MT * NT * kWave * 16;         // the waves' results
};

// Where 16-byte piece p of row r of a stage lies in LDS. A copy instruction
// fills 64 pieces in a row, and its lanes must take whole 64-byte blocks of the
// source in order (permuted inside a block they are four accesses, not one: 46
// against 38 us at 1024 x 4096 x 2048), so the layout is plain but for 16 bytes
// of padding after each kilobyte or longer row and, with two rows a copy, the
// halves of 128 bytes swapped in odd rows. The fragment reads, 16 rows times
// four even (or odd) pieces, then take each bank slot the same number of times.
template <int PIECES>
__device__ __forceinline__ int ll_place(int r, int p) {
  if constexpr (PIECES == 32) return (r / 2) * 1040 + (r % 2) * 512 + 16 * (p ^ (r % 2 * 8));
  else return r * (16 * PIECES + 16) + 16 * p;
}

template <int MT, int NT, int WN, int WAVES, int BUFS>
__global__ void __launch_bounds__(kWave * WAVES)
k_linear_lora(const uint16_t* __restrict__ x, int T, int K, const int8_t* __restrict__ codes,
              const uint16_t* __restrict__ scales, int N, const uint16_t* __restrict__ b, int L, int R,
              const int32_t* __restrict__ adapter, const float* __restrict__ h, int slices, int ttiles, int wgs,
              float* __restrict__ y) {
  using S = LlShape<MT, NT, WN, WAVES, BUFS>;
  constexpr int WK = S::kWk;
  extern __shared__ __align__(16) uint8_t sm[];
  const int tid = threadIdx.x, lane = tid % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int wn = wave % WN, wk = wave / WN;
  const int c = lane % 16, kq = lane / 16;
  // the token tiles of a column tile follow one another on one XCD: its L2 reads the codes once
  const int wg = blockIdx.x % kLlXcds * (gridDim.x / kLlXcds) + blockIdx.x / kLlXcds;
  if (wg >= wgs) return;
  const int t0 = wg % ttiles * S::kRows, n0 = wg / ttiles * S::kCols + 16 * NT * wn;
  int ad[MT < WK ? 1 : MT / WK];               // of the tiles that the wave keeps in the end
#pragma unroll
  for (int o = 0; o < (MT < WK ? 1 : MT / WK); ++o)
    ad[o] = lora_row_adapter(adapter, t0 + 16 * (wk + o * WK), T, L, c);
  const int G = K / kGroup, stages = (G + WK - 1) / WK;
  // Workgroups start at different stages: rows lie a power of two apart more often than not, and all of them at the
  // same piece of K would ask the same L2 channels.
  const int turn = wg % stages;

  // rows past T, columns past N and pieces past K stand for the last ones: nothing of theirs is stored
  const uint32_t lds = (uint32_t)(uintptr_t)(ll_lds_t*)sm;
  const auto load_x = [&](int s, int buf) {
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) {
      const int at = S::kThreads * i + kWave * wave;              // the wave's first piece of this copy
      const int row = (at + lane) / S::kPieces;
      const int p = S::kPieces == 32 ? (lane % 32) ^ (lane / 32 * 8) : at % S::kPieces + lane;
      const int k = min((s * S::kPieces + p) * 8, K - 8);
      ll_copy16(2u * ((uint32_t)min(t0 + row, T - 1) * (uint32_t)K + (uint32_t)k), x,
                lds + buf * S::kStage + ll_place<S::kPieces>(at / S::kPieces, at % S::kPieces));
    }
  };
  // the wave's columns: a uniform base and a lane's 32-bit offset (the entry point bounds K)
  const int nb = min(n0, N - 16);
  const int8_t* cbase = codes + (size_t)nb * K;
  const uint16_t* sbase = scales + (size_t)nb * G;
  uint32_t coff[NT], soff[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    const uint32_t n = min(n0 + 16 * j + c, N - 1) - nb;
    coff[j] = n * (uint32_t)K + 16 * kq;
    soff[j] = n * (uint32_t)G;
  }
  // stages on their way: kAhead of them, their codes and scales in registers
  constexpr int kAhead = BUFS - 1;
  u32x4 cn[kAhead][NT][2];
  uint16_t sn[kAhead][NT];
  const auto load_codes = [&](auto to, int s) {
    const int g = min(s * WK + wk, G - 1);     // (past the last group: not used)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        cn[to.value][j][i] = *reinterpret_cast<const u32x4*>(cbase + g * kGroup + 64 * i + coff[j]);
      sn[to.value][j] = sbase[g + soff[j]];
    }
  };
  f32x4 acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[m][j] = {0.f, 0.f, 0.f, 0.f};
  bf16x8 w[NT][4];
  float sc[NT];
  const auto decode = [&](auto from) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      sc[j] = (float)__builtin_bit_cast(_Float16, sn[from.value][j]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t lo = cn[from.value][j][i / 2][2 * (i % 2)], hi = cn[from.value][j][i / 2][2 * (i % 2) + 1];
        // opaque to the compiler: it would take the words apart where they are loaded, and wait for them there
        asm volatile("" : "+v"(lo), "+v"(hi));
        w[j][i] = ll_decode(lo, hi);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  const auto multiply = [&](const uint8_t* xs) {
    // A token tile's fragments are read while the tile before multiplies, and its sums folded while the next one does:
    // the barriers keep the compiler from moving them apart.
    bf16x8 xv[2][4];
    f32x4 p[2][NT];
    const auto read = [&](int m) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int piece = 16 * wk + 8 * (q / 2) + 2 * kq + q % 2;
        xv[m % 2][q] = *reinterpret_cast<const bf16x8*>(xs + ll_place<S::kPieces>(16 * m, 0) +
                                                        ll_place<S::kPieces>(c, piece));
      }
    };
    const auto fold = [&](int m) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[m][j][q] = fmaf(sc[j], p[m % 2][j][q], acc[m][j][q]);
    };
    read(0);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if (m + 1 < MT) read(m + 1);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int j = 0; j < NT; ++j) p[m % 2][j] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int j = 0; j < NT; ++j)
          p[m % 2][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xv[m % 2][q], w[j][q], p[m % 2][j], 0, 0, 0);
      if (m > 0) fold(m - 1);
      __builtin_amdgcn_sched_barrier(0);
    }
    fold(MT - 1);
  };

  const auto nth = [&](int i) { return i + turn < stages ? i + turn : i + turn - stages; };
  // The copies of a stage are awaited by count: those of the kAhead - 1 stages behind it may be on their way (the codes'
  // loads among them only make the wait longer). At the end of K there are fewer, and all are awaited.
  const auto stage = [&](auto slot, int i) {   // slot = i % kAhead
    decode(slot);
    if (i + kAhead < stages) {
      load_x(nth(i + kAhead), (i + kAhead) % BUFS);
      load_codes(slot, nth(i + kAhead));
    }
    if (nth(i) * WK + wk < G) multiply(sm + i % BUFS * S::kStage);
    if (i + kAhead < stages) __builtin_amdgcn_s_waitcnt(ll_vmcnt((kAhead - 1) * S::kLoads));
    else __builtin_amdgcn_s_waitcnt(ll_vmcnt(0));
    __syncthreads();
  };
  const std::integral_constant<int, 0> s0;
  const std::integral_constant<int, kAhead - 1 < 1 ? kAhead - 1 : 1> s1;
  const std::integral_constant<int, kAhead - 1 < 2 ? kAhead - 1 : 2> s2;
  static_assert(kAhead == 1 || kAhead == 3, "stages are written out below");
  load_x(nth(0), 0);
  load_codes(s0, nth(0));
  if constexpr (kAhead == 3) {
    if (stages > 1) {
      load_x(nth(1), 1);
      load_codes(s1, nth(1));
    }
    if (stages > 2) {
      load_x(nth(2), 2);
      load_codes(s2, nth(2));
    }
  }
  if (stages >= kAhead) __builtin_amdgcn_s_waitcnt(ll_vmcnt((kAhead - 1) * S::kLoads));
  else __builtin_amdgcn_s_waitcnt(ll_vmcnt(0));
  __syncthreads();
#pragma unroll 1
  for (int i = 0; i < stages; i += kAhead) {
    stage(s0, i);
    if constexpr (kAhead == 3) {
      if (i + 1 < stages) stage(s1, i + 1);
      if (i + 2 < stages) stage(s2, i + 2);
    }
  }

  // the WK waves' results of a column meet in LDS: wave wk keeps the token tiles wk, wk + WK, .. (res[o]: tile wk + o WK)
  constexpr int MO = MT < WK ? 1 : MT / WK;
  const bool keeps = wk < MT;
  f32x4* part = reinterpret_cast<f32x4*>(sm);          // [wave][tile][lane]
  f32x4 res[MO][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      if (m % WK != wk) part[((wave * MT + m) * NT + j) * kWave + lane] = acc[m][j];
      else res[m / WK][j] = acc[m][j];
    }
  __syncthreads();
  // the adapters of its tiles, the first one's B and the thread's first item of h are on their way meanwhile
  const int rc0 = min(R, kLlRank);
  const auto load_b = [&](int l, int r, int rc, bf16x8 (&to)[NT]) {
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      u32x4 v = {0u, 0u, 0u, 0u};
      if (r % kLlRank + 8 * kq < rc)
        v = *reinterpret_cast<const u32x4*>(b + ((size_t)l * N + min(n0 + 16 * j + c, N - 1)) * R + r + 8 * kq);
      to[j] = __builtin_bit_cast(bf16x8, v);
    }
  };
  bf16x8 bv[MO][NT];
  LoraItem<kLoraSlices> item;
  const int item_row = tid / (rc0 / 8), item_r = 8 * (tid % (rc0 / 8));
  const bool has_item = item_row < S::kRows, has_sum = has_item && lora_row_adapter(adapter, t0, T, L, item_row) >= 0;
  if (has_sum) item.load(h, 0, slices, T, R, t0 + item_row, item_r);
  if (keeps) {
#pragma unroll
    for (int o = 0; o < MO; ++o) {
      const uint32_t rows = lora_rows(ad[o] >= 0);
      if (rows != 0) load_b(__builtin_amdgcn_readlane(ad[o], __ffs(rows) - 1), 0, rc0, bv[o]);
    }
#pragma unroll
    for (int o = 0; o < MO; ++o)
#pragma unroll
      for (int v = 1; v < WK; ++v) {
        const int from = (wk + v) % WK * WN + wn;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const f32x4 u = part[((from * MT + wk + o * WK) * NT + j) * kWave + lane];
#pragma unroll
          for (int i = 0; i < 4; ++i) res[o][j][i] += u[i];
        }
      }
  }
  __syncthreads();

  // the adapters: h of the workgroup's rows in LDS, kLlRank of R at a time
  const int ld = lora_split_stride(rc0);
  if (has_item) {
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (has_sum) item.add(0, slices, v);
    lora_split_store<S::kRows>(v, item_row, item_r, sm, ld);
  }
  for (int r0 = 0; r0 < R; r0 += kLlRank) {
    const int rc = min(R - r0, kLlRank);
    lora_split_rows<S::kRows, S::kThreads>(h, slices, T, R, r0, rc, adapter, L, t0, sm, ld,
                                           tid + (r0 == 0 ? S::kThreads : 0));
    __syncthreads();
    if (keeps) {
#pragma unroll
      for (int o = 0; o < MO; ++o) {
        const int row0 = 16 * (wk + o * WK);
        uint32_t left = lora_rows(ad[o] >= 0);
        bool ready = r0 == 0;                          // bv[o] holds this adapter's first piece
        while (left != 0) {
          const int l = __builtin_amdgcn_readlane(ad[o], __ffs(left) - 1);
          const uint32_t mine = lora_rows(ad[o] == l);
          left &= ~mine;
          f32x4 d[NT];
          const auto products = [&](auto finite) {
#pragma unroll
            for (int j = 0; j < NT; ++j) d[j] = {0.f, 0.f, 0.f, 0.f};
            for (int r = 0; r < rc; r += 32) {
              if (!ready) load_b(l, r0 + r, rc, bv[o]);
              ready = false;
#pragma unroll
              for (int p = 0; p < 3; ++p) {
                bf16x8 hv = __builtin_bit_cast(bf16x8, u32x4{0u, 0u, 0u, 0u});
                if (r + 8 * kq < rc)
                  hv = *reinterpret_cast<const bf16x8*>(sm + (p * S::kRows + row0 + c) * ld + 2 * (r + 8 * kq));
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                  d[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hv, bv[o][j], d[j], 0, 0, 0);
                  if constexpr (decltype(finite)::value) bv[o][j] = lora_finite(bv[o][j]);
                }
              }
            }
          };
          products(std::false_type{});
          const float all = lora_total(d);
          if (__builtin_expect(__ballot(all != all) != 0, 0)) products(std::true_type{});
          // the rows of other adapters keep what they have, whatever this one holds
#pragma unroll
          for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if ((mine >> (4 * kq + i)) & 1) res[o][j][i] += d[j][i];
        }
      }
    }
    __syncthreads();
  }
  if (keeps) {
#pragma unroll
    for (int o = 0; o < MO; ++o)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = t0 + 16 * (wk + o * WK) + 4 * kq + i, n = n0 + 16 * j + c;
          if (t < T && n < N) y[(size_t)t * N + n] = res[o][j][i];
        }
  }
}

template <int MT, int NT, int WN, int WAVES, int BUFS>
hipError_t launch(const uint16_t* x, int T, int K, const int8_t* codes, const uint16_t* scales, int N,
                  const uint16_t* b, int L, int R, const int32_t* adapter, const float* h, int slices, float* y,
                  hipStream_t st) {
  using S = LlShape<MT, NT, WN, WAVES, BUFS>;
  const int ttiles = cdiv(T, S::kRows), wgs = ttiles * cdiv(N, S::kCols), grid = cdiv(wgs, kLlXcds) * kLlXcds;
  const size_t lds = std::max<size_t>({(size_t)BUFS * S::kStage, (size_t)S::kJoin,
                                       (size_t)3 * S::kRows * lora_split_stride(std::min(R, kLlRank))});
  k_linear_lora<MT, NT, WN, WAVES, BUFS><<<grid, S::kThreads, lds, st>>>(x, T, K, codes, scales, N, b, L, R, adapter, h, slices,
                                                           ttiles, wgs, y);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_linear_i8f16_lora(const uint16_t* x, int T, int K, const int8_t* codes, const uint16_t* scales,
                                    int N, const uint16_t* b, int L, int R, const int32_t* adapter, const float* h,
                                    int slices, float* y, hipStream_t st) {
#define I8H_LL(MT, NT, WN, WAVES, BUFS) \
  return launch<MT, NT, WN, WAVES, BUFS>(x, T, K, codes, scales, N, b, L, R, adapter, h, slices, y, st)
  // The smallest tile whose workgroups the 256 CUs hold in about one turn: small ones cost least where there is little
  // to do, large ones read and decode a code for more tokens. Measured with the shrink, K = 2048, rank 16, us:
  //   tokens x columns    16 x 16   32 x 32   64 x 128   128 x 128
  //     32 x 4096          13.5      14.3       24.8       28.5       (512 workgroups of 16 x 16)
  //     64 x 4096          20.9      14.9       26.2       29.8
  //    512 x 1024          34.6      19.6       26.8       33.4       (512 workgroups of 32 x 32)
  //    256 x 4096          58.7      29.2       27.0       32.7
  //    512 x 4096         107        48.7       28.6       33.8       (256 workgroups of 64 x 128)
  //   1024 x 4096         225       104         52.3       40.7
  const auto within = [&](int rows, int cols, int wgs) { return (int64_t)cdiv(T, rows) * cdiv(N, cols) <= wgs; };
  if (within(16, 16, 512)) I8H_LL(1, 1, 1, 8, 2);
  if (within(32, 32, 512)) I8H_LL(2, 1, 2, 8, 2);
  if (within(64, 128, 256)) I8H_LL(4, 2, 4, 8, 4);
  I8H_LL(8, 2, 4, 8, 2);
#undef I8H_LL
}

}  // namespace i8h
