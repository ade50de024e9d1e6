// MXFP4 products for a few tokens (decode): one launch each, latency first.
//
// gate_up: a workgroup owns 4 x (8 gate + the matching 8 up rows) of one expert
// for all of the expert's pairs. It quantises every token's row itself (a few
// KB from L2, into LDS), which waits for nothing, while the expert is found and
// its weights, all of them at once, are on their way: two dependent loads from
// launch to weights, and no second launch. Tokens are few, so quantising them in
// every workgroup costs less than a launch that does it once.
//
// down: a workgroup owns 16 output rows of one token and all its slots; each of
// 8 waves takes a slot, quantises that slot's act row into LDS of its own, and
// the slots' sums meet in LDS to be merged in slot order: out comes straight
// from one launch, with no y.
//
// Bound by latency more than by HBM (one token, 8 of 128 experts: gate_up 13.4 MB
// in 8.3 us; down 6.7 MB in 6.6 us): a launch, then the chain offsets, weights,
// products, sums. 7 tokens of 4 of 60 experts: 33 MB in 12.8 us, 2.6 TB/s.
//
// Both use v_mfma_scale_f32_16x16x128_f8f6f4: lane l holds block 4 j + l / 16
// (of step j, K = 128) of weight row l % 16 (A) and of column l % 16 (B), and
// results of rows 4 (l / 16) .. +3, column l % 16. An expert's pairs are the
// columns.

#include "launch.hpp"
#include "mxfp4.hpp"

namespace i8h {

namespace {

// Steps of a chunk held in registers: K = 2048. With all of a row's loads in
// flight at once gate_up of one token takes 8.3 us; with the activation rows
// loaded before them 9.4.
constexpr int kFewSteps = 16;

__device__ __forceinline__ f32x4 mx_mfma16(const u32x4 a, const u32x4 b, f32x4 c, uint32_t sa, uint32_t sb) {
  const i32x8 av = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8 bv = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

// --------------------------------------------------------------------- gate_up

constexpr int kFgThreads = 256;
constexpr int kFgWaves = kFgThreads / kWave;
constexpr int kFgLds = 64 * 1024;    // quantised tokens: rows of codes and scales
constexpr int kFgAhead = 8;          // groups of eight values a thread loads at once: 8 tokens of K = 2048

// bytes of a token's row in LDS: codes, then scales, padded to an odd number of
// 16-byte pieces (columns then lie in different banks)
__host__ __device__ constexpr int few_row_bytes(int nb) { return (cdiv(17 * nb, 16) | 1) * 16; }

template <typename AT>
__global__ void __launch_bounds__(kFgThreads)
k_gateup_mx_few(const uint16_t* __restrict__ x, int T, int nb, const uint8_t* __restrict__ wq,
                const uint8_t* __restrict__ ws, int E, int N, int topk, const int32_t* __restrict__ off,
                const int32_t* __restrict__ sorted_pairs, float* __restrict__ gu, AT* __restrict__ act) {
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  const int tid = threadIdx.x, lane = tid % kWave, g = lane / 16, c = lane % 16;
  const int I = N / 2, K = nb * kMxBlock, row_bytes = few_row_bytes(nb);

  // the y-th expert that has pairs, from one batch of loads a 64 experts; the
  // workgroups past the last such expert come last in the grid
  int e = 0, r0 = 0, m = 0, seen = 0;
  for (int e0 = 0; e0 < E; e0 += kWave) {
    const int i = e0 + lane;
    const int lo = i < E ? off[i] : 0, hi = i < E ? off[i + 1] : 0;
    const uint64_t some = __ballot(lo < hi);
    const int rank = seen + __popcll(some & ((1ull << lane) - 1));
    const uint64_t here = __ballot(lo < hi && rank == (int)blockIdx.y);
    if (here != 0) {
      const int src = __ffsll((unsigned long long)here) - 1;
      e = __builtin_amdgcn_readfirstlane(e0 + src);
      r0 = __builtin_amdgcn_readfirstlane(__shfl(lo, src, kWave));
      m = __builtin_amdgcn_readfirstlane(__shfl(hi, src, kWave)) - r0;
      break;
    }
    seen += __popcll(some);
  }
  if (m == 0) return;

  // weight row of this lane: rows 4 G, 4 G + 1 of a tile are gate rows 2 G, 2 G + 1,
  // rows 4 G + 2, 4 G + 3 the matching up rows
  const int tile = blockIdx.x * kFgWaves + tid / kWave;
  const int i0 = tile * 8 + 2 * (c / 4) + (c & 1);   // N % 64 == 0: the tiles fill the grid's waves
  const size_t n = (size_t)e * N + ((c & 2) ? I + i0 : i0);
  const uint8_t* wr = wq + n * (16 * nb) + 16 * g;
  const uint8_t* wsr = ws + n * nb;
  int token = sorted_pairs[r0 + min(c, m - 1)];   // of this lane's column: its pair for now
  const int steps = nb / 4;            // K % 128 == 0
  u32x4 w[kFewSteps];
  uint32_t s[kFewSteps];
  auto load = [&](int j0) {
#pragma unroll
    for (int j = 0; j < kFewSteps; ++j)
      if (j0 + j < steps) {
        w[j] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(wr + 64 * (j0 + j)));
        s[j] = *reinterpret_cast<const uint32_t*>(wsr + 4 * (j0 + j));
      }
  };
  load(0);

  // every token's row, eight values a thread and a time, kFgAhead loads at once
  const int groups = T * (K / 8);
  auto raw = [&](int p) { return mx_raw8(x + (size_t)min(p, groups - 1) * 8); };
  u32x4 xv[kFgAhead];
#pragma unroll
  for (int i = 0; i < kFgAhead; ++i)
    if (i * kFgThreads < groups) xv[i] = raw(i * kFgThreads + tid);

  auto quantise = [&](int p, const u32x4 r) {
    float v[8];
    mx_floats(r, v);
    int sc;
    const uint32_t q = mx_quant8(v, sc);   // whole blocks: a block's four lanes are all in or all out
    if (p < groups) {
      const int t = p / (K / 8), k8 = p - t * (K / 8);
      *reinterpret_cast<uint32_t*>(&lds[t * row_bytes + 4 * k8]) = q;
      if ((k8 & 3) == 0) lds[t * row_bytes + 16 * nb + k8 / 4] = (uint8_t)sc;
    }
  };
#pragma unroll
  for (int i = 0; i < kFgAhead; ++i)
    if (i * kFgThreads < groups) quantise(i * kFgThreads + tid, xv[i]);
  for (int p0 = kFgAhead * kFgThreads; p0 < groups; p0 += kFgThreads) quantise(p0 + tid, raw(p0 + tid));
  token /= topk;
  __syncthreads();

  for (int c0 = 0; c0 < m; c0 += 16) {
    const int r = r0 + min(c0 + c, m - 1);
    if (c0 > 0) token = sorted_pairs[r] / topk;
    const uint8_t* xr = lds + token * row_bytes;
    f32x4 acc = {};
    for (int j0 = 0; j0 < steps; j0 += kFewSteps) {
      if (j0 > 0 || (c0 > 0 && steps > kFewSteps)) load(j0);
#pragma unroll
      for (int j = 0; j < kFewSteps; ++j)
        if (j0 + j < steps) {
          const u32x4 b = *reinterpret_cast<const u32x4*>(xr + 64 * (j0 + j) + 16 * g);
          const uint32_t xs = *reinterpret_cast<const uint32_t*>(xr + 16 * nb + 4 * (j0 + j));
          acc = mx_mfma16(w[j], b, acc, s[j] >> (8 * g), xs >> (8 * g));
        }
    }
    if (c0 + c < m) {
      // rows 4 g .. +3: gate 2 g, 2 g + 1, then up
      const size_t o = (size_t)r * I + tile * 8 + 2 * g;
      if (gu) {
        float* gr = gu + (size_t)r * N + tile * 8 + 2 * g;
        gr[0] = acc[0];
        gr[1] = acc[1];
        gr[I] = acc[2];
        gr[I + 1] = acc[3];
      }
      if (act) {
        put_act(act, o, gelu_tanh(acc[0]) * acc[2]);
        put_act(act, o + 1, gelu_tanh(acc[1]) * acc[3]);
      }
    }
  }
}

// ------------------------------------------------------------------------ down

constexpr int kFdThreads = 512;
constexpr int kFdWaves = kFdThreads / kWave;
constexpr int kFdMaxI = 2048;
constexpr int kFdRow = kFdMaxI / 2 + kFdMaxI / 32;   // LDS of a wave's act row: codes, then scales

template <typename XT>
__global__ void __launch_bounds__(kFdThreads)
k_down_mx_few(const XT* __restrict__ act, int nb, const uint8_t* __restrict__ wq, const uint8_t* __restrict__ ws, int H,
              int k, const int32_t* __restrict__ ids, const float* __restrict__ tw, const int32_t* __restrict__ pos,
              float* __restrict__ out) {
  __shared__ __attribute__((aligned(16))) uint8_t rows[kFdWaves][kFdRow];
  __shared__ float part[kMaxTopk][16];
  const int tid = threadIdx.x, lane = tid % kWave, g = lane / 16, c = lane % 16, wave = tid / kWave;
  const int t = blockIdx.y, h0 = 16 * blockIdx.x, waves = blockDim.x / kWave;
  const int steps = (nb + 3) / 4;      // the last one may hold fewer than four blocks
  uint8_t* row = rows[wave];
  for (int j = wave; j < k; j += waves) {
    const int e = ids[t * k + j];
    const int64_t r = pos[t * k + j];
    const size_t n = (size_t)e * H + h0 + c;
    const uint8_t* wr = wq + n * (16 * nb);
    const uint8_t* wsr = ws + n * nb;
    u32x4 w[kFewSteps];
    uint32_t s[kFewSteps];
    // a block past the row's last one re-reads that one with scale 1; its act codes are zero
#pragma unroll
    for (int i = 0; i < kFewSteps; ++i)
      if (i < steps) {
        const int b = 4 * i + g;
        w[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(wr + 16 * min(b, nb - 1)));
        s[i] = b < nb ? wsr[b] : 127u;
      }
    // the slot's act row, eight values a lane at a time
    constexpr int kPer = kFewSteps * 16 / kWave;
    decltype(mx_raw8(act)) xv[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (4 * i < steps) xv[i] = mx_raw8(act + r * (nb * kMxBlock) + 8 * min(i * kWave + lane, 4 * nb - 1));
    wave_lds_order();   // every lane has read the last slot's row
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (4 * i < steps) {
        const int p = i * kWave + lane;
        const bool in = p < 4 * nb;
        float v[8];
        mx_floats(xv[i], v);
        int sc;
        const uint32_t q = mx_quant8(v, sc);   // whole blocks: a block's four lanes are all in or all out
        if (p < 16 * steps) {
          *reinterpret_cast<uint32_t*>(&row[4 * p]) = in ? q : 0u;
          if ((p & 3) == 0) row[kFdMaxI / 2 + p / 4] = (uint8_t)(in ? sc : 127);
        }
      }
    wave_lds_order();
    f32x4 acc = {};
#pragma unroll
    for (int i = 0; i < kFewSteps; ++i)
      if (i < steps)
        acc = mx_mfma16(w[i], *reinterpret_cast<const u32x4*>(&row[64 * i + 16 * g]), acc, s[i],
                        row[kFdMaxI / 2 + 4 * i + g]);
    // every column holds the same sums: column 0's, rows 4 g .. +3
    if (c == 0)
#pragma unroll
      for (int i = 0; i < 4; ++i) part[j][4 * g + i] = acc[i];
  }
  __syncthreads();
  if (tid < 16) {
    float o = 0.0f;
    for (int j = 0; j < k; ++j) o = fmaf(tw[t * k + j], part[j][tid], o);
    out[(size_t)t * H + h0 + tid] = o;
  }
}

}  // namespace

// Up to 8 tokens and 32 pairs, the tokens' rows within LDS. Both ways, this form
// and k_mx_stream, 128 experts, top 8: gate_up (K = 2048, N = 1536) one token 8.3
// and 11.0 us, 2 12.9 and 14.5, 4 17.8 and 21.1, 8 26.6 and 25.3; down (I = 768,
// H = 2048) 6.6 and 10.5, 7.3 and 12.7, 12.7 and 15.8, 22.3 and 18.9.
static bool mx_few(int T, int topk) { return T <= 8 && T * topk <= 32; }
bool mx_few_gateup(int T, int K, int topk) {
  return mx_few(T, topk) && T * few_row_bytes(K / kMxBlock) <= kFgLds;
}
bool mx_few_down(int T, int I, int topk) { return mx_few(T, topk) && I <= kFdMaxI; }

hipError_t launch_gateup_mxfp4_few(const uint16_t* x, int T, int K, const uint8_t* codes, const uint8_t* scales, int E,
                                   int N, int k, const int32_t* expert_off, const int32_t* sorted_pairs, float* gu,
                                   void* act, bool act_bf16, hipStream_t st) {
  const int nb = K / kMxBlock;
  const dim3 grid(N / (16 * kFgWaves), T * k < E ? T * k : E);
  const size_t lds = (size_t)T * few_row_bytes(nb);
  if (act_bf16)
    k_gateup_mx_few<<<grid, kFgThreads, lds, st>>>(x, T, nb, codes, scales, E, N, k, expert_off, sorted_pairs, gu,
                                                   static_cast<uint16_t*>(act));
  else
    k_gateup_mx_few<<<grid, kFgThreads, lds, st>>>(x, T, nb, codes, scales, E, N, k, expert_off, sorted_pairs, gu,
                                                   static_cast<float*>(act));
  return hipGetLastError();
}

hipError_t launch_down_mxfp4_few(const void* act, bool act_bf16, int T, int I, const uint8_t* codes,
                                 const uint8_t* scales, int H, int k, const int32_t* ids, const float* tw,
                                 const int32_t* pos, float* out, hipStream_t st) {
  const dim3 grid(H / 16, T);
  const int threads = kWave * (k < kFdWaves ? k : kFdWaves);
  const int nb = I / kMxBlock;
  if (act_bf16)
    k_down_mx_few<<<grid, threads, 0, st>>>(static_cast<const uint16_t*>(act), nb, codes, scales, H, k, ids, tw, pos,
                                               out);
  else
    k_down_mx_few<<<grid, threads, 0, st>>>(static_cast<const float*>(act), nb, codes, scales, H, k, ids, tw, pos,
                                               out);
  return hipGetLastError();
}

}  // namespace i8h
