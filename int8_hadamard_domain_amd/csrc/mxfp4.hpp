// MXFP4 (OCP Microscaling Formats v1.0: blocks of 32 E2M1 values with one
// E8M0 scale) on gfx950: the quantiser's block step and the scaled FP4 matrix
// instruction, shared by the MXFP4 kernels.
#pragma once

#include "common.hpp"
#include "xlane.hpp"

namespace i8h {

constexpr int kMxBlock = 32;   // values per scale

// Eight consecutive values of a block held by four neighbouring lanes ->
// packed codes, and the block's scale byte (the same in all four lanes).
// With a = max |x| of the block and e its biased exponent field, the scale is
// 2^(floor(log2 a) - 2), at least 2^-127: byte max(e - 2, 0), also where a is
// zero or subnormal (e = 0). The quotient x / scale is one exact multiply by
// 2^(127 - s), and v_cvt_scalef32_pk_fp4_f32 (scale 1) rounds it to the
// nearest E2M1 value, ties to the even code, 6 at most. An infinity or NaN
// (e = 255 in the largest magnitude's bits) marks the block with s = 255.
__device__ __forceinline__ uint32_t mx_quant8(const float (&v)[8], int& s) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  m = max(m, (uint32_t)xor_lane_i<1>((int)m));
  m = max(m, (uint32_t)xor_lane_i<2>((int)m));
  const int e = (int)(m >> 23);
  s = e == 255 ? 255 : max(e - 2, 0);
  const float f = __uint_as_float((uint32_t)(254 - min(s, 252)) << 23);   // 2^(127 - s)
  uint32_t c = 0;
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[0] * f, v[1] * f, 1.0f, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[2] * f, v[3] * f, 1.0f, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[4] * f, v[5] * f, 1.0f, 2);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, v[6] * f, v[7] * f, 1.0f, 3);
  return e == 255 ? 0u : c;
}

// eight values as they lie in memory, and as floats
struct MxRaw32 {
  f32x4 a, b;
};
__device__ __forceinline__ MxRaw32 mx_raw8(const float* p) {
  return {reinterpret_cast<const f32x4*>(p)[0], reinterpret_cast<const f32x4*>(p)[1]};
}
__device__ __forceinline__ u32x4 mx_raw8(const uint16_t* p) { return *reinterpret_cast<const u32x4*>(p); }
// the same for data that is read once
__device__ __forceinline__ MxRaw32 mx_raw8_once(const float* p) {
  return {__builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p)),
          __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p) + 1)};
}
__device__ __forceinline__ u32x4 mx_raw8_once(const uint16_t* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
}
__device__ __forceinline__ void mx_floats(const MxRaw32& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = r.a[i];
    v[4 + i] = r.b[i];
  }
}
__device__ __forceinline__ void mx_floats(const u32x4 r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(r[i]);
    v[2 * i + 1] = bf16_hi(r[i]);
  }
}

template <typename T>
__device__ __forceinline__ void mx_load8_once(const T* p, float (&v)[8]) {
  mx_floats(mx_raw8_once(p), v);
}

// LDS that a wave's lanes write for its other lanes: what stands before is done
// when what follows begins, in each lane's program (no instruction; the hardware
// takes a wave's LDS accesses in order)
__device__ __forceinline__ void wave_lds_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
}

// 32 x 32 x 64 with both operands E2M1: lane l holds the 32 codes of row (A) or
// column (B) l % 32 for k = 32 (l / 32) .. +31 of the step, and in byte SA / SB
// of its scale word that block's E8M0 scale; result register r of lane l is
// row 8 (r / 4) + 4 (l / 32) + r % 4, column l % 32 (checked against exact sums).
template <int SA, int SB>
__device__ __forceinline__ f32x16 mx_mfma32(const u32x4 a, const u32x4 b, f32x16 c, uint32_t sa, uint32_t sb) {
  const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(av, bv, c, 4, 4, SA, (int)sa, SB, (int)sb);
}

}  // namespace i8h
