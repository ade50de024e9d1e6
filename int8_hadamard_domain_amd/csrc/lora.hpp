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

// Bytes between rows of a part of h in LDS: 16 bytes of padding, so that the
// fragment reads of 16 rows spread over the banks.
__host__ __device__ constexpr inline int lora_split_stride(int R) { return 2 * R + 16; }

constexpr int kLoraSlices = 8;               // most slices of K

// Eight inner sums of a row: the loads of up to S slices at once, added up in
// the slices' order, and the store of the sum in three bf16 parts.
template <int S>
struct LoraItem {
  f32x4 u[S][2];
  __device__ __forceinline__ void load(const float* __restrict__ h, int s0, int slices, int T, int R, int64_t t,
                                       int r) {
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (s0 + s < slices) {
        const f32x4* p = reinterpret_cast<const f32x4*>(h + ((int64_t)(s0 + s) * T + t) * R + r);
        u[s][0] = p[0];
        u[s][1] = p[1];
      }
  }
  __device__ __forceinline__ void add(int s0, int slices, float (&v)[8]) const {
#pragma unroll
    for (int s = 0; s < S; ++s)
      if (s0 + s < slices) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] += u[s][0][j];
          v[4 + j] += u[s][1][j];
        }
      }
  }
};
template <int ROWS>
__device__ __forceinline__ void lora_split_store(const float (&v)[8], int row, int r, uint8_t* sm, int ld) {
  const Bf16Split q = split3(v);
#pragma unroll
  for (int p = 0; p < 3; ++p) *reinterpret_cast<bf16x8*>(sm + (p * ROWS + row) * ld + 2 * r) = q.p[p];
}

// The inner sums r0 .. r0 + rc - 1 of ROWS rows from t0 on, added up over the
// slices of K, in three bf16 parts: part p of row r at sm + (p ROWS + r) ld.
// Rows without an adapter are zero. By a workgroup of THREADS threads, from
// item `from` on (a thread's next one is THREADS further); a barrier must follow.
template <int ROWS, int THREADS>
__device__ __forceinline__ void lora_split_rows(const float* __restrict__ h, int slices, int T, int R, int r0, int rc,
                                                const int32_t* __restrict__ adapter, int L, int64_t t0, uint8_t* sm,
                                                int ld, int from) {
#pragma unroll 1
  for (int i = from; i < ROWS * (rc / 8); i += THREADS) {
    const int row = i / (rc / 8), r = 8 * (i % (rc / 8));
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (lora_row_adapter(adapter, t0, T, L, row) >= 0)
      for (int s = 0; s < slices; s += 4) {
        LoraItem<4> item;
        item.load(h, s, slices, T, R, t0 + row, r0 + r);
        item.add(s, slices, v);
      }
    lora_split_store<ROWS>(v, row, r, sm, ld);
  }
}

// LDS that a wave's lanes hand on to each other: writes before, reads after.
__device__ __forceinline__ void lora_wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Infinities of B. Of an inner sum's parts the first has its sign, and is 0 only
// where it is (a subnormal one aside), but the others are often 0, and 0 times an
// infinity is NaN. So where the products hold a NaN they are done again without
// B's infinities and NaN in the second and third part: what is finite comes out
// with the same bits, and the first part decides about the rest. The check is a
// few additions; no finite adapter gets further.

// The sum of a lane's products: NaN if one is (or if there are infinities of both
// signs: then they are done again for nothing).
template <int N>
__device__ __forceinline__ float lora_total(const f32x4 (&d)[N]) {
  float t = 0.0f;
#pragma unroll
  for (int j = 0; j < N; ++j) t += (d[j][0] + d[j][1]) + (d[j][2] + d[j][3]);
  return t;
}

// Eight bf16 values, 0 for infinities and NaN.
__device__ __forceinline__ bf16x8 lora_finite(const bf16x8& v) {
  u32x4 w = __builtin_bit_cast(u32x4, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if ((w[i] & 0x7f80u) == 0x7f80u) w[i] &= 0xffff0000u;
    if ((w[i] & 0x7f800000u) == 0x7f800000u) w[i] &= 0x0000ffffu;
  }
  return __builtin_bit_cast(bf16x8, w);
}

// The products of the adapters' second half, 32 of R from r0 on: d[m][j] += B h
// for the 16 MT rows in LDS (lora_split_rows) and 32 NT columns, bv[j] holding
// row 16 j + lane % 16 of B: the lane gets row 16 m + lane % 16, columns
// 16 j + 4 (lane / 16) .. + 3. FINITE: see above; bv is changed.
template <int MT, int NT, bool FINITE>
__device__ __forceinline__ void lora_multiply(bf16x8 (&bv)[2 * NT], int R, int r0, const uint8_t* sm, int ld,
                                              int lane, f32x4 (&d)[MT][2 * NT]) {
  const int c = lane % 16, r = r0 + 8 * (lane / 16);
  const auto part = [&](int m, int p) {
    bf16x8 hv = __builtin_bit_cast(bf16x8, u32x4{0u, 0u, 0u, 0u});
    if (r < R) hv = *reinterpret_cast<const bf16x8*>(sm + (p * 16 * MT + 16 * m + c) * ld + 2 * r);
#pragma unroll
    for (int j = 0; j < 2 * NT; ++j)
      d[m][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bv[j], hv, d[m][j], 0, 0, 0);
  };
  if constexpr (FINITE) {
#pragma unroll 1
    for (int p = 0; p < 3; ++p) {
#pragma unroll
      for (int m = 0; m < MT; ++m) part(m, p);
#pragma unroll
      for (int j = 0; j < 2 * NT; ++j) bv[j] = lora_finite(bv[j]);
    }
  } else {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int p = 0; p < 3; ++p) part(m, p);
  }
}

}  // namespace i8h
