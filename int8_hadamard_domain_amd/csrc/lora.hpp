// Pieces that the kernels with low-rank adapters share. A tile is 16 rows of
// the batch; lane c + 16 q of a wave stands for row c.
#pragma once

#include "common.hpp"

namespace i8h {

// The adapter of row c, -1 for none (outside [0, L), or past the batch).
__device__ __forceinline__ int lora_row_adapter(const int32_t* __restrict__ adapter, int64_t t0, int T, int L, int c) {
  const int ad = t0 + c < T ? adapter[t0 + c] : -1;
  return (uint32_t)ad < (uint32_t)L ? ad : -1;
}

// The rows of the tile where a lane's condition holds, one bit a row.
__device__ __forceinline__ uint32_t lora_rows(bool cond) { return (uint32_t)__ballot(cond) & 0xffffu; }

// Eight float32 values as three bf16 parts whose sum they are: each takes the
// 8 leading bits of what the ones before leave, so the split is exact above
// float32's smallest normal value times 2^16 (below that the last part rounds).
// An infinity or NaN is the first part alone.
struct Bf16Split {
  bf16x8 p[3];
};
__device__ __forceinline__ Bf16Split split3(const float (&v)[8]) {
  uint32_t w[3][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = __float_as_uint(v[i]);
    const bool number = (u & 0x7f800000u) != 0x7f800000u;
    w[0][i] = number ? u & 0xffff0000u : (u & 0x007fffffu) != 0 ? 0x7fc00000u : u;
    const float r1 = number ? v[i] - __uint_as_float(w[0][i]) : 0.0f;
    w[1][i] = __float_as_uint(r1) & 0xffff0000u;
    const float r2 = r1 - __uint_as_float(w[1][i]);
    w[2][i] = __float_as_uint(r2) & 0xffff0000u;
  }
  Bf16Split s;
#pragma unroll
  for (int j = 0; j < 3; ++j) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = (w[j][2 * i] >> 16) | (w[j][2 * i + 1] & 0xffff0000u);
    s.p[j] = __builtin_bit_cast(bf16x8, o);
  }
  return s;
}

// acc[j] += the adapters' part of a tile: row c of the lane, columns
// n0 + 16 j + 4 (lane / 16) .. + 3, for each adapter the rows name in turn.
template <int TILES>
__device__ __forceinline__ void lora_expand(const uint16_t* __restrict__ b, int N, int R, const float* __restrict__ h,
                                            int64_t t0, int T, int n0, int ad, int lane, f32x4 (&acc)[TILES]) {
  const int c = lane % 16, kq = lane / 16;
  uint32_t left = lora_rows(ad >= 0);
  while (left != 0) {
    const int l = __builtin_amdgcn_readlane(ad, __ffs(left) - 1);
    left &= ~lora_rows(ad == l);
    const uint16_t* bl = b + (size_t)l * N * R;
    f32x4 d[TILES];
#pragma unroll
    for (int j = 0; j < TILES; ++j) d[j] = {0.f, 0.f, 0.f, 0.f};
    for (int r0 = 0; r0 < R; r0 += 32) {
      const int r = r0 + 8 * kq;
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (ad == l && r < R) {
        const float* hr = h + (t0 + c) * R + r;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = hr[i];
      }
      const Bf16Split s = split3(v);
#pragma unroll
      for (int j = 0; j < TILES; ++j) {
        const int n = n0 + 16 * j + c;
        u32x4 w = {0u, 0u, 0u, 0u};
        if (n < N && r < R) w = *reinterpret_cast<const u32x4*>(bl + (size_t)n * R + r);
        const bf16x8 bv = __builtin_bit_cast(bf16x8, w);
#pragma unroll
        for (int p = 0; p < 3; ++p) d[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv, s.p[p], d[j], 0, 0, 0);
      }
    }
    // the rows of other adapters keep what they have, whatever this one holds
    if (ad == l) {
#pragma unroll
      for (int j = 0; j < TILES; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[j][i] += d[j][i];
    }
  }
}

}  // namespace i8h
