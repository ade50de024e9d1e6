// Grouped MXFP4 products of the routed experts: gate_up with its GELU
// epilogue, and the down projection with the weighted combine.
//
// Both operands are MXFP4 (activations quantised per token, or per act row,
// just before): for sorted row r of expert e
//   c[r, n] = sum_b 2^(sw[e,n,b] + sx[r,b] - 254) sum_{k in b} qw[e,n,k] qx[r,k]
// v_mfma_scale_f32_32x32x64_f8f6f4 takes the codes as they lie in memory and
// the block scales beside them, so there is no decode and no fold: a product
// step is the instruction alone. Its float32 sums keep the full significand
// (products far below the largest of an instruction are kept, unlike the E4M3
// forms), so the result is as exact as a float32 sum.
//
// The weights are the A operand (32 rows: for gate_up 16 gate rows and the
// matching 16 up rows, so both halves of an output meet in one lane), the
// activation rows the B operand (32 columns).
//
// Work item = one pass of up to 32 MT rows of one expert x 128 weight rows, a
// workgroup of 4 waves, a 32-row weight tile each. The weights go straight from
// memory into operand registers, PD stages of K = 256 ahead (lane l reads 64
// contiguous bytes of row l % 32; this pattern streams at 5.8 TB/s by itself,
// 16-byte loads in address order at 5.9): every wave has its own, so LDS would
// only add a copy. The activation rows are shared: double-buffered in LDS,
// loaded up to three stages ahead through registers.
// Within a stage, step j takes block 4 (lane / 32) + j of both operands, so a
// lane's four scale bytes are one dword, picked by the instruction's byte select.

#include <type_traits>

#include "launch.hpp"
#include "mxfp4.hpp"

namespace i8h {

namespace {

constexpr int kMgThreads = 256;   // 4 waves, a 32-row weight tile each
constexpr int kMgWaves = kMgThreads / kWave;
constexpr int kMgRows = 32 * kMgWaves;   // weight rows of a work item
constexpr int kStB = 8;                  // blocks of a stage (K = 256)
constexpr int kRowBytes = 144;           // LDS row: 128 B of codes, 8 B of scales, 8 B so that 16 rows meet all 64 banks
constexpr int kXcds = 8;

struct MxArgs {
  const uint8_t* xq;   // activation codes, rows of 128 stages bytes (padded to whole stages)
  const uint8_t* xs;   // activation scales, rows of 8 stages
  const uint8_t* wq;   // [E, R, K/2]
  const uint8_t* ws;   // [E, R, K/32]
  uint32_t xq_n;       // bytes of xq (xs has a sixteenth)
  int E, R, nb, topk, ntiles, items;
  const int32_t* expert_off;
  const int32_t* sorted_pairs;   // gate_up: activation row of sorted row r is sorted_pairs[r] / topk
};

// Item i of the passes of up to `rows` rows, experts in order: its expert,
// first sorted row and row count; false past the last item. Every wave of the
// workgroup finds it by itself, from one batch of expert_off loads.
__device__ __forceinline__ bool mx_item(const int32_t* __restrict__ off, int E, int i, int rows, int& e, int& r0,
                                        int& m) {
  const int lane = threadIdx.x % kWave;
  int before = 0;
  for (int e0 = 0; e0 < E; e0 += kWave) {
    const int x = e0 + lane;
    const int lo = off[min(x, E)], hi = off[min(x + 1, E)];
    const int n = (hi - lo + rows - 1) / rows;
    int inc = n;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int o = __shfl_up(inc, d, kWave);
      if (lane >= d) inc += o;
    }
    const uint64_t past = __ballot(before + inc > i);
    if (past != 0) {
      const int src = __ffsll((unsigned long long)past) - 1;
      const int first = i - (before + __shfl(inc - n, src, kWave));   // pass of that expert
      const int l = __shfl(lo, src, kWave), h = __shfl(hi, src, kWave);
      e = __builtin_amdgcn_readfirstlane(e0 + src);
      r0 = __builtin_amdgcn_readfirstlane(l + first * rows);
      m = __builtin_amdgcn_readfirstlane(min(rows, h - r0));
      return true;
    }
    before += __shfl(inc, kWave - 1, kWave);
  }
  return false;
}

// LDS writes before it are seen by the workgroup after it; loads from global
// memory stay in flight (__syncthreads may wait for them)
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

struct MxW {
  u32x4 q[4];
  uint32_t s;
};

// Loads go through buffer descriptors: an offset past the descriptor's size
// reads zero and moves nothing, so the loads past the last stage are issued
// like all others, under a descriptor of size 0. With no branch around a load
// the compiler counts those in flight exactly and waits only for what it uses.
typedef __amdgpu_buffer_rsrc_t mx_rsrc;
__device__ __forceinline__ mx_rsrc mx_buffer(const uint8_t* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), 0, (int)bytes, 0x00020000);   // raw, 32-bit data
}
__device__ __forceinline__ u32x4 mx_get16(mx_rsrc r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0);
}
__device__ __forceinline__ uint32_t mx_get4(mx_rsrc r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0);
}

// The lane's four blocks of stage s of its weight row, qo and so the row's
// offsets. TAIL: rows that are not whole stages. What is read past the row's
// last block meets activation codes of zero, and its scale is set to 1, so
// that another row's NaN scale stays out. Rows of scales may then start
// anywhere: two aligned words hold the four bytes.
template <bool TAIL>
__device__ __forceinline__ void mx_load_w(mx_rsrc wq, mx_rsrc ws, uint32_t qo, uint32_t so, int s, int half, int nb,
                                          MxW& w) {
  const uint32_t o = qo + 128 * s + 64 * half;
#pragma unroll
  for (int j = 0; j < 4; ++j) w.q[j] = mx_get16(wq, o + 16 * j);
  const uint32_t c = so + kStB * s + 4 * half;
  if constexpr (!TAIL) {
    w.s = mx_get4(ws, c);
  } else {
    const uint32_t v = __builtin_amdgcn_alignbyte(mx_get4(ws, (c & ~3u) + 4), mx_get4(ws, c & ~3u), c & 3);
    const int left = nb - (kStB * s + 4 * half);   // blocks of the row from here on
    const uint32_t m = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
    w.s = (v & m) | (0x7f7f7f7fu & ~m);
  }
}

__device__ __forceinline__ void put4(float* p, const f32x4 v) { *reinterpret_cast<f32x4*>(p) = v; }
__device__ __forceinline__ void put4(uint16_t* p, const f32x4 v) {
  *reinterpret_cast<u32x2*>(p) = u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
}

// GU: gate_up with epilogue (out0 = gate_up or NULL, out1 = act or NULL);
// otherwise out0 = y [P, R]
template <bool GU, int MT, bool TAIL, int PD, typename AT>
__global__ void __launch_bounds__(kMgThreads, MT == 1 ? 4 : MT == 2 ? 3 : 2)
k_mx_grouped(const MxArgs a, float* __restrict__ out0, AT* __restrict__ out1) {
  static_assert(PD % 2 == 0, "the activation registers and LDS buffers alternate by stage");
  __shared__ __attribute__((aligned(16))) uint8_t buf[2][32 * MT * kRowBytes];
  // the tiles of an item run on one XCD (they share its activation rows) once
  // there are items for every XCD; with fewer, consecutive tiles on all of them
  const int blk = blockIdx.x;
  int i, nt;
  if (a.items >= 4 * kXcds) {
    i = blk % kXcds + kXcds * (blk / (kXcds * a.ntiles));
    nt = (blk / kXcds) % a.ntiles;
  } else {
    i = blk / a.ntiles;
    nt = blk % a.ntiles;
  }
  int e, r0, m;
  if (!mx_item(a.expert_off, a.E, i, 32 * MT, e, r0, m)) return;
  const int tid = threadIdx.x, lane = tid % kWave, half = lane / 32, col = lane % 32;
  const int tile = nt * kMgWaves + __builtin_amdgcn_readfirstlane(tid / kWave);
  const int I = a.R / 2, nb = a.nb, S = (nb + kStB - 1) / kStB;
  const bool live = tile * 32 < a.R;
  // weight row of this lane (dead waves repeat row 0: they still copy and meet the barriers)
  int n = 0;
  if (live) n = GU ? (col < 16 ? tile * 16 + col : I + tile * 16 + col - 16) : tile * 32 + col;
  const uint8_t* wq = a.wq + (size_t)e * a.R * (16 * nb);
  const uint8_t* ws = a.ws + (size_t)e * a.R * nb;
  const uint32_t wq_n = (uint32_t)a.R * (16 * nb), ws_n = (uint32_t)a.R * nb;
  const uint32_t qo = (uint32_t)n * (16 * nb), so = (uint32_t)n * nb;
  auto load_w = [&](int s, MxW& w) __attribute__((always_inline)) {
    mx_load_w<TAIL>(mx_buffer(wq, s < S ? wq_n : 0), mx_buffer(ws, s < S ? ws_n : 0), qo, so, s, half, nb, w);
  };
  MxW w[PD];
#pragma unroll
  for (int d = 0; d < PD; ++d) load_w(d, w[d]);

  auto run = [&](auto na_c) __attribute__((always_inline)) {
    constexpr int NA = decltype(na_c)::value;   // live 32-row tiles of the pass
    // activation pieces this thread copies: 16 bytes of row 32 q + tid / 8; the
    // scales (8 bytes) of row tid % (32 NA): several threads write the same bytes,
    // with no branch (rows past the pass repeat its last one)
    uint32_t xo[NA], xso;
    {
      auto src = [&](int row) {
        const int r = r0 + min(row, m - 1);
        return (uint32_t)(GU ? a.sorted_pairs[r] / a.topk : r);
      };
#pragma unroll
      for (int q = 0; q < NA; ++q) xo[q] = src(32 * q + tid / 8) * (uint32_t)(128 * S) + 16 * (tid % 8);
      xso = src(tid % (32 * NA)) * (uint32_t)(8 * S);
    }
    u32x4 xr[2][NA];
    uint32_t sr[2][2];
    auto load_x = [&](int s, u32x4 (&xr)[NA], uint32_t (&sr)[2]) __attribute__((always_inline)) {
      const mx_rsrc q = mx_buffer(a.xq, s < S ? a.xq_n : 0), c = mx_buffer(a.xs, s < S ? a.xq_n / 16 : 0);
#pragma unroll
      for (int i = 0; i < NA; ++i) xr[i] = mx_get16(q, xo[i] + 128 * s);
      sr[0] = mx_get4(c, xso + 8 * s);
      sr[1] = mx_get4(c, xso + 8 * s + 4);
    };
    auto store_x = [&](int b, const u32x4 (&xr)[NA], const uint32_t (&sr)[2]) __attribute__((always_inline)) {
#pragma unroll
      for (int q = 0; q < NA; ++q)
        *reinterpret_cast<u32x4*>(&buf[b][(32 * q + tid / 8) * kRowBytes + 16 * (tid % 8)]) = xr[q];
      *reinterpret_cast<u32x2*>(&buf[b][(tid % (32 * NA)) * kRowBytes + 128]) = u32x2{sr[0], sr[1]};
    };

    f32x16 acc[NA];
#pragma unroll
    for (int q = 0; q < NA; ++q) acc[q] = f32x16{};
    load_x(0, xr[0], sr[0]);
    load_x(1, xr[1], sr[1]);
    store_x(0, xr[0], sr[0]);
    load_x(2, xr[0], sr[0]);
    lds_barrier();
    // stages past the last one (S up to a multiple of PD) add products with zero codes
    for (int s0 = 0; s0 < S; s0 += PD) {
#pragma unroll
      for (int d = 0; d < PD; ++d) {
        const int s = s0 + d;
        const uint8_t* x = &buf[s & 1][col * kRowBytes + 64 * half];
        uint32_t xs[NA];
#pragma unroll
        for (int q = 0; q < NA; ++q)
          xs[q] = *reinterpret_cast<const uint32_t*>(&buf[s & 1][(32 * q + col) * kRowBytes + 128 + 4 * half]);
        auto step = [&](auto jc) __attribute__((always_inline)) {
          constexpr int J = decltype(jc)::value;
#pragma unroll
          for (int q = 0; q < NA; ++q) {
            const u32x4 xv = *reinterpret_cast<const u32x4*>(x + 32 * q * kRowBytes + 16 * J);
            acc[q] = mx_mfma32<J, J>(w[d].q[J], xv, acc[q], w[d].s, xs[q]);
          }
        };
        step(std::integral_constant<int, 0>{});
        step(std::integral_constant<int, 1>{});
        step(std::integral_constant<int, 2>{});
        step(std::integral_constant<int, 3>{});
        __builtin_amdgcn_sched_barrier(0);   // the next use of these registers is loaded after their products
        load_w(s + PD, w[d]);
        store_x((s + 1) & 1, xr[(d + 1) & 1], sr[(d + 1) & 1]);
        load_x(s + 3, xr[(d + 1) & 1], sr[(d + 1) & 1]);
        lds_barrier();
      }
    }
    if (!live) return;
#pragma unroll
    for (int q = 0; q < NA; ++q) {
      if (32 * q + col >= m) continue;
      const size_t r = (size_t)r0 + 32 * q + col;
      if constexpr (GU) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // gate rows 8 h + 4 half .. +3 of the tile in registers 4 h .. +3, their up rows in 8 + 4 h .. +3
          const int i0 = tile * 16 + 8 * h + 4 * half;
          f32x4 g, u, v;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            g[j] = acc[q][4 * h + j];
            u[j] = acc[q][8 + 4 * h + j];
            v[j] = gelu_tanh(g[j]) * u[j];
          }
          if (out0) {
            put4(out0 + r * a.R + i0, g);
            put4(out0 + r * a.R + I + i0, u);
          }
          if (out1) put4(out1 + r * I + i0, v);
        }
      } else {
#pragma unroll
        for (int h = 0; h < 4; ++h)
          put4(out0 + r * a.R + tile * 32 + 8 * h + 4 * half,
               f32x4{acc[q][4 * h], acc[q][4 * h + 1], acc[q][4 * h + 2], acc[q][4 * h + 3]});
      }
    }
  };
  const int na = (m + 31) / 32;
  if constexpr (MT == 1) {
    run(std::integral_constant<int, 1>{});
  } else if constexpr (MT == 2) {
    if (na == 1) run(std::integral_constant<int, 1>{});
    else run(std::integral_constant<int, 2>{});
  } else {
    switch (na) {
      case 1: run(std::integral_constant<int, 1>{}); break;
      case 2: run(std::integral_constant<int, 2>{}); break;
      case 3: run(std::integral_constant<int, 3>{}); break;
      case 4: run(std::integral_constant<int, 4>{}); break;
      default: run(std::integral_constant<int, 5>{}); break;
    }
  }
}

// out[t, h .. h + 3] = sum_j w[t, j] y[pos[t k + j], h .. h + 3], slot order
__global__ void __launch_bounds__(kMgThreads)
k_mx_combine(const float* __restrict__ y, int H, int k, const float* __restrict__ tw, const int32_t* __restrict__ pos,
             float* __restrict__ out) {
  const int64_t t = blockIdx.x;
  const int h = 4 * (blockIdx.y * kMgThreads + threadIdx.x);
  if (h >= H) return;
  f32x4 o = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < k; ++j) {
    const float wj = tw[t * k + j];
    const f32x4 v = *reinterpret_cast<const f32x4*>(y + (size_t)pos[t * k + j] * H + h);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = fmaf(wj, v[i], o[i]);
  }
  *reinterpret_cast<f32x4*>(out + t * H + h) = o;
}

}  // namespace

template <bool GU, typename AT>
static hipError_t mx_grouped(MxArgs a, int64_t P, int64_t rows, float* out0, AT* out1, hipStream_t st) {
  // rows per pass by the average expert: passes of 32 rows while experts hold a
  // dozen pairs, of 160 (a prefill expert's 128 on average, with its spread) for many
  const int mt = P <= 16 * (int64_t)a.E ? 1 : P <= 40 * (int64_t)a.E ? 2 : 5;
  a.ntiles = cdiv(a.R, kMgRows);
  a.xq_n = (uint32_t)(rows * cdiv(a.nb, kStB) * 128);
  // every non-empty expert has at most one pass that is not full
  const int64_t items = P / (32 * mt) + (P < a.E ? P : a.E);
  const int64_t grid = (items + kXcds - 1) / kXcds * kXcds * a.ntiles;
  if (grid >= ((int64_t)1 << 31)) return hipErrorInvalidValue;
  a.items = (int)items;
  const bool tail = a.nb % kStB != 0;
  const unsigned g = (unsigned)grid;
#define I8H_MX(M, PD)                                                            \
  do {                                                                           \
    if (tail) k_mx_grouped<GU, M, true, PD><<<g, kMgThreads, 0, st>>>(a, out0, out1);  \
    else k_mx_grouped<GU, M, false, PD><<<g, kMgThreads, 0, st>>>(a, out0, out1);      \
  } while (0)
  if (mt == 1) I8H_MX(1, 2);
  else if (mt == 2) I8H_MX(2, 2);
  else I8H_MX(5, 2);
#undef I8H_MX
  return hipGetLastError();
}

hipError_t launch_gateup_mxfp4(const uint8_t* xq, const uint8_t* xs, int T, int K, const uint8_t* codes,
                               const uint8_t* scales, int E, int N, int k, const int32_t* expert_off,
                               const int32_t* sorted_pairs, float* gu, void* act, bool act_bf16, hipStream_t st) {
  const MxArgs a = {xq, xs, codes, scales, 0, E, N, K / kMxBlock, k, 0, 0, expert_off, sorted_pairs};
  const int64_t P = (int64_t)T * k;
  return act_bf16 ? mx_grouped<true>(a, P, T, gu, static_cast<uint16_t*>(act), st)
                  : mx_grouped<true>(a, P, T, gu, static_cast<float*>(act), st);
}

hipError_t launch_down_mxfp4(const uint8_t* aq, const uint8_t* as, int T, int I, const uint8_t* codes,
                             const uint8_t* scales, int E, int H, int k, const float* tw, const int32_t* expert_off,
                             const int32_t* pos, float* y, float* out, hipStream_t st) {
  const MxArgs a = {aq, as, codes, scales, 0, E, H, I / kMxBlock, k, 0, 0, expert_off, nullptr};
  const hipError_t err = mx_grouped<false>(a, (int64_t)T * k, (int64_t)T * k, y, static_cast<float*>(nullptr), st);
  if (err != hipSuccess) return err;
  k_mx_combine<<<dim3(T, cdiv(H / 4, kMgThreads)), kMgThreads, 0, st>>>(y, H, k, tw, pos, out);
  return hipGetLastError();
}

}  // namespace i8h
