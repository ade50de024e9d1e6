// MXFP4 quantiser and its inverse.
//
// Per block of 32 (OCP Microscaling Formats v1.0, conversion to E2M1):
//   s = max(floor(log2 max|x|) - 2, -127) + 127,  code = E2M1(x 2^(127 - s)).
// Both are streams: the quantiser reads 2 or 4 bytes a value and writes 17/32,
// the inverse the other way round. A lane takes 8 values (one or two 16-byte
// loads, one 4-byte store of codes), four lanes a block.

#include "launch.hpp"
#include "mxfp4.hpp"

namespace i8h {

namespace {

constexpr int kMxThreads = 256;
// Groups of eight values a thread takes. Bound by HBM: 24576 x 2048 float32 to
// codes in 43 us (228 MB, 5.3 TB/s; with one group a thread 52.5), back in 35 us
// (6.5 TB/s); a large copy moves 5.1 TB/s.
constexpr int kMxGroups = 2;

template <typename XT>
__global__ void __launch_bounds__(kMxThreads)
k_mxfp4_quantize(const XT* __restrict__ x, int64_t n8, uint32_t* __restrict__ codes, uint8_t* __restrict__ scales) {
  // rows are whole blocks, so the matrix is one run of blocks
  const int64_t i0 = (int64_t)blockIdx.x * (kMxGroups * kMxThreads) + threadIdx.x;
  float v[kMxGroups][8] = {};
#pragma unroll
  for (int g = 0; g < kMxGroups; ++g) {
    const int64_t i = i0 + g * kMxThreads;
    if (i < n8) mx_load8_once(x + 8 * i, v[g]);   // n8 is a multiple of 4: a block's lanes are all in or all out
  }
#pragma unroll
  for (int g = 0; g < kMxGroups; ++g) {
    const int64_t i = i0 + g * kMxThreads;
    int s;
    const uint32_t c = mx_quant8(v[g], s);
    if (i < n8) {
      codes[i] = c;
      if ((threadIdx.x & 3) == 0) scales[i / 4] = (uint8_t)s;
    }
  }
}

// E2M1 code -> float: codes 0..7 are 0, 0.5, 1, 1.5, 2, 3, 4, 6
template <int SEL>
__device__ __forceinline__ void mx_values(uint32_t c, float (&v)[8]) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  const f32x2 p = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, SEL);
  v[2 * SEL] = p[0];
  v[2 * SEL + 1] = p[1];
}

template <typename OT>
__global__ void __launch_bounds__(kMxThreads)
k_mxfp4_dequantize(const uint32_t* __restrict__ codes, const uint8_t* __restrict__ scales, int64_t n8,
                   OT* __restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * kMxThreads + threadIdx.x;
  if (i >= n8) return;
  const uint32_t c = codes[i];
  const int s = scales[i / 4];
  float v[8];
  mx_values<0>(c, v);
  mx_values<1>(c, v);
  mx_values<2>(c, v);
  mx_values<3>(c, v);
  // v 2^(s - 127): exact in float32 down to its subnormals (the product has one
  // to two significand bits and is at least 2^-128)
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = s == 255 ? __builtin_nanf("") : ldexpf(v[j], s - 127);
  if constexpr (sizeof(OT) == 4) {
    f32x4* o = reinterpret_cast<f32x4*>(out + 8 * i);
    o[0] = f32x4{v[0], v[1], v[2], v[3]};
    o[1] = f32x4{v[4], v[5], v[6], v[7]};
  } else {
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
    *reinterpret_cast<u32x4*>(out + 8 * i) = o;
  }
}

}  // namespace

hipError_t launch_mxfp4_quantize(const void* x, bool bf16, int64_t values, uint8_t* codes, uint8_t* scales,
                                 hipStream_t st) {
  const int64_t n8 = values / 8, per = kMxGroups * kMxThreads, grid = (n8 + per - 1) / per;
  uint32_t* c = reinterpret_cast<uint32_t*>(codes);
  if (bf16)
    k_mxfp4_quantize<<<(unsigned)grid, kMxThreads, 0, st>>>(static_cast<const uint16_t*>(x), n8, c, scales);
  else
    k_mxfp4_quantize<<<(unsigned)grid, kMxThreads, 0, st>>>(static_cast<const float*>(x), n8, c, scales);
  return hipGetLastError();
}

hipError_t launch_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t values, void* out, bool bf16,
                                   hipStream_t st) {
  const int64_t n8 = values / 8, grid = (n8 + kMxThreads - 1) / kMxThreads;
  const uint32_t* c = reinterpret_cast<const uint32_t*>(codes);
  if (bf16)
    k_mxfp4_dequantize<<<(unsigned)grid, kMxThreads, 0, st>>>(c, scales, n8, static_cast<uint16_t*>(out));
  else
    k_mxfp4_dequantize<<<(unsigned)grid, kMxThreads, 0, st>>>(c, scales, n8, static_cast<float*>(out));
  return hipGetLastError();
}

}  // namespace i8h
