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
// The weights are the B operand (tiles of 32 rows, one a lane: for gate_up 16
// gate rows and the matching 16 up rows), the activation rows the A operand, so
// that neighbouring lanes hold neighbouring features and stores write whole
// runs of them. Within a stage of K = 256, step j
// takes block 4 (lane / 32) + j of both operands, so a lane's four scale bytes
// are one dword, picked by the instruction's byte select, and its codes 64
// contiguous bytes of its row.
//
// The rows are cut into passes, up to 32 MT sorted rows of one expert each.
//   k_mx_stream  the passes' weight tiles are dealt to one workgroup of 8 waves
//                per CU. A workgroup keeps a pass's activation rows in LDS, whole
//                K, and its waves stream tiles past them from memory straight into
//                operand registers, PD stages ahead and on into the next tile: no
//                barrier, no wait but for the weights themselves. Passes of one
//                expert start together on neighbouring CUs of an XCD, so most
//                weights leave memory once. With few rows an expert it finds the
//                passes and quantises their rows itself, one launch; else
//   k_mx_prepare has listed the passes and quantised the rows before.
//   k_mx_ring    for K too long for that: activation rows in stages through LDS.
//
// Bounds, at 128 experts, top 8, K = 2048, N = 1536 (I = 768, H = 2048):
//   128 tokens   the weights from HBM: gate_up 216 MB in 44 us, 4.9 TB/s (a large
//                copy: 5.1), down 111 MB and the y round trip in 32 us.
//   2048 tokens  gate_up 75 us, 71 of them k_mx_stream: 255 MB of HBM traffic
//                (weights fetched 1.04 times) at 3.6 TB/s, matrix units 30 % busy,
//                LDS less; the rest are each pass's start (rows to LDS, 5 to 7 us),
//                whole rounds of tiles and the epilogue. down 86 us: y, 131 MB,
//                written (k_mx_stream 53 to 60) and read again (k_mx_combine 22).

#include <type_traits>

#include "launch.hpp"
#include "mxfp4.hpp"

namespace i8h {

// one pass: up to 32 MT sorted rows of one expert (the list's entry 0 holds the
// number of passes in e)
struct MxItem {
  int e, r0, m, pad;
};

namespace {

constexpr int kStB = 8;             // blocks of a stage (K = 256)
constexpr int kXcds = 8;
constexpr int kPrThreads = 256;     // k_mx_prepare, k_mx_combine

struct MxArgs {
  const uint8_t* x;    // activation rows of row_bytes: codes padded to whole stages, then their scales
  const uint8_t* wq;   // [E, R, K/2]
  const uint8_t* ws;   // [E, R, K/32]
  uint32_t x_n;        // bytes of x, rounded up so that 16-byte reads of scales end inside
  int row_bytes;
  int E, R, nb, topk, ntiles;
  const MxItem* items;           // NULL where the kernel finds passes and quantises rows itself, from:
  const void* raw;               // [rows, 32 nb] float32 or bf16
  const int32_t* off;
  const int32_t* sorted_pairs;   // gate_up: activation row of sorted row r is sorted_pairs[r] / topk
};

// Loads go through buffer descriptors: an offset past the descriptor's size
// reads zero and moves nothing, so the loads past the last stage are issued
// like all others, under a descriptor of size 0. With no branch around a load
// the compiler counts those in flight exactly and waits only for what it uses.
typedef __amdgpu_buffer_rsrc_t mx_rsrc;
__device__ __forceinline__ mx_rsrc mx_buffer(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);   // raw, 32-bit data
}
__device__ __forceinline__ u32x4 mx_get16(mx_rsrc r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0);
}
__device__ __forceinline__ uint32_t mx_get4(mx_rsrc r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0);
}

// the same 16 bytes to LDS, lane l's at p + 16 l, with no register between
__device__ __forceinline__ void mx_get16_lds(mx_rsrc r, uint8_t* p, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)p, 16, (int)off, 0, 0, 0);
}

// The four scale bytes v of a lane's blocks, of which the row has `left` from
// there on: what is read past a row's last block meets activation codes of
// zero, and the scale 1 keeps another row's NaN scale out.
__device__ __forceinline__ uint32_t mx_mask_scales(uint32_t v, int left) {
  const uint32_t m = left >= 4 ? ~0u : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
  return (v & m) | (0x7f7f7f7fu & ~m);
}

// LDS writes before it are seen by the workgroup after it; loads from global
// memory stay in flight (__syncthreads may wait for them)
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// A stage of weights as the matrix unit wants it (lane: its row's four pieces of
// 16 bytes, one a register) from how it is loaded (register k: piece lane % 4 of
// the lane's quad's row k). A quad's four lanes then read 64 contiguous bytes,
// which the load path takes at 52 bytes a clock and CU; each lane reading its
// own row's, it takes 15. Two rounds of exchanges between neighbours: a and b
// are registers k and k + HOP, lanes with bit HOP of k set keep b and fetch b of
// the lane HOP below into a, the others keep a and fetch a into b. One
// instruction a word: a select whose one side comes from another lane, which the
// compiler does not form by itself (it makes a lane move and a select of the
// intrinsics: 64 vector instructions a stage instead of 32, times within 1 %). The
// blocks wait out the two cycles between a vector write and a lane move's, or a
// matrix instruction's, read, and write every output before the last input is
// read, so outputs are early-clobber.
#define I8H_SEL(D, MOVED, KEPT) "v_cndmask_b32_dpp " D ", " MOVED ", " KEPT ", vcc " I8H_PERM "\n"
#define I8H_EXCHANGE                                                                                              \
  "s_nop 1\n"                                                                                                     \
  "s_mov_b64 vcc, %[set]\n" /* b of the lanes whose bit is not set comes from a */                                \
  I8H_SEL("%[t0]", "%[a0]", "%[b0]") I8H_SEL("%[t1]", "%[a1]", "%[b1]")                                           \
  I8H_SEL("%[t2]", "%[a2]", "%[b2]") I8H_SEL("%[t3]", "%[a3]", "%[b3]")                                           \
  "s_not_b64 vcc, vcc\n" /* a of the others from b */                                                             \
  I8H_SEL("%[a0]", "%[b0]", "%[a0]") I8H_SEL("%[a1]", "%[b1]", "%[a1]")                                           \
  I8H_SEL("%[a2]", "%[b2]", "%[a2]") I8H_SEL("%[a3]", "%[b3]", "%[a3]")                                           \
  "s_nop 1"
template <int HOP>
__device__ __forceinline__ void mx_exchange(u32x4& a, u32x4& b) {
  uint32_t t0, t1, t2, t3, a0 = a[0], a1 = a[1], a2 = a[2], a3 = a[3];
#define I8H_REGS                                                                                                  \
  : [t0] "=&v"(t0), [t1] "=&v"(t1), [t2] "=&v"(t2), [t3] "=&v"(t3), [a0] "+&v"(a0), [a1] "+&v"(a1), [a2] "+&v"(a2), \
    [a3] "+&v"(a3)                                                                                                \
  : [b0] "v"(b[0]), [b1] "v"(b[1]), [b2] "v"(b[2]), [b3] "v"(b[3]), [set] "s"(lanes)                              \
  : "vcc", "scc"
  if constexpr (HOP == 1) {
    const uint64_t lanes = 0xaaaaaaaaaaaaaaaaull;
#define I8H_PERM "quad_perm:[1,0,3,2] row_mask:0xf bank_mask:0xf"
    asm(I8H_EXCHANGE I8H_REGS);
#undef I8H_PERM
  } else {
    const uint64_t lanes = 0xccccccccccccccccull;
#define I8H_PERM "quad_perm:[2,3,0,1] row_mask:0xf bank_mask:0xf"
    asm(I8H_EXCHANGE I8H_REGS);
#undef I8H_PERM
  }
#undef I8H_REGS
  a = u32x4{a0, a1, a2, a3};
  b = u32x4{t0, t1, t2, t3};
}
#undef I8H_EXCHANGE
#undef I8H_SEL
__device__ __forceinline__ void mx_transpose(u32x4 (&w)[4]) {
  mx_exchange<1>(w[0], w[1]);
  mx_exchange<1>(w[2], w[3]);
  mx_exchange<2>(w[0], w[2]);
  mx_exchange<2>(w[1], w[3]);
}

// one value at offset off, dropped past the descriptor's end
__device__ __forceinline__ void mx_put(mx_rsrc r, float, float v, uint32_t off) {
  __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, (int)off, 0, 0);
}
__device__ __forceinline__ void mx_put(mx_rsrc r, uint16_t, float v, uint32_t off) {
  __builtin_amdgcn_raw_buffer_store_b16((uint16_t)pack_bf16x2(v, 0.f), r, (int)off, 0, 0);
}

// The results of one 32-row weight tile for NA x 32 rows from sorted row r0 (m
// of them live). GU: out0 = gate_up or NULL, out1 = act or NULL; else out0 = y.
// A lane holds one weight row's products with 16 sorted rows, so a store writes
// whole runs of features (down: 128 bytes, a cache line) of two or four rows;
// rows behind m lie past the descriptor and are dropped.
template <bool GU, int NA, typename AT>
__device__ __forceinline__ void mx_store(const f32x16 (&acc)[NA], int tile, int R, int r0, int m, float* out0,
                                         AT* out1) {
  const int lane = threadIdx.x % kWave, half = lane / 32, col = lane % 32, I = R / 2;
#pragma unroll
  for (int q = 0; q < NA; ++q) {
    const uint32_t live = (uint32_t)min(32, m - 32 * q);
    if constexpr (GU) {
      // Lanes 0..15 hold gate rows, 16..31 the matching up rows: swapped with
      // the next register, one register holds the gates of sorted rows j and
      // j + 1 (lanes 0..15, 16..31), the other their ups.
      const mx_rsrc g_r = mx_buffer(out0 + (size_t)(r0 + 32 * q) * R, out0 ? live * R * 4 : 0);
      const mx_rsrc a_r = mx_buffer(out1 + (size_t)(r0 + 32 * q) * I, out1 ? live * I * sizeof(AT) : 0);
      const int row = 4 * half + col / 16, n = tile * 16 + col % 16;
      const uint32_t og = 4 * (uint32_t)(row * R + n), oa = sizeof(AT) * (uint32_t)(row * I + n);
#pragma unroll
      for (int r = 0; r < 16; r += 2) {
        const uint32_t j = 8 * (r / 4) + r % 4;
        if (8 * (r / 4) >= live) break;
        const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(acc[q][r]), __float_as_uint(acc[q][r + 1]),
                                                        false, false);
        const float g = __uint_as_float(s[0]), u = __uint_as_float(s[1]);
        if (out0) {
          mx_put(g_r, 0.f, g, og + 4 * j * R);
          mx_put(g_r, 0.f, u, og + 4 * (I + j * R));
        }
        if (out1) mx_put(a_r, AT{}, gelu_tanh(g) * u, oa + sizeof(AT) * j * I);
      }
    } else {
      const mx_rsrc y_r = mx_buffer(out0 + (size_t)(r0 + 32 * q) * R, live * R * 4);
      const uint32_t oy = 4 * (uint32_t)(4 * half * R + tile * 32 + col);
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        if (8 * (r / 4) >= live) break;
        mx_put(y_r, 0.f, acc[q][r], oy + 4 * (8 * (r / 4) + r % 4) * R);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Activation rows resident in LDS, weights streamed

constexpr int kSmThreads = 512;                   // 8 waves, two a SIMD
constexpr int kSmWaves = kSmThreads / kWave;
constexpr int kSmBlocks = 256;                    // one workgroup a CU
constexpr int kSmX = 128 * 1104;                  // LDS for activation rows: 128 of K = 2048
constexpr int kSmGroup = 64;                      // blocks of a row whose scales a wave holds at a time
// LDS for a wave's scales: a tile's 32 rows, 16 bytes unused behind every 64, or
// the rows of K = 2048 would all begin in the same four banks
constexpr int kSmSc = 32 * kSmGroup / 4 * 5 + 16;
__device__ __forceinline__ int mx_sc_at(int o) { return o + o / 64 * 16; }

// how a wave copies its tile's scales to LDS
enum class MxSc {
  kRun,     // nb <= 64: whole rows, one or two contiguous runs of 16 nb or 32 nb bytes
  kPiece,   // 64 blocks of each row at a time, 16 bytes a load (nb % 16 == 0)
  kWord     // the same, 4 bytes a load (nb % 4 == 0)
};

// XT: element type of the rows that the kernel quantises itself, or void for
// rows and passes that k_mx_prepare made.
template <bool GU, int MT, int PD, MxSc SM, typename XT, typename AT>
__global__ void __launch_bounds__(kSmThreads, 2)
k_mx_stream(const MxArgs a, float* __restrict__ out0, AT* __restrict__ out1) {
  constexpr bool kOwn = !std::is_void_v<XT>;
  __shared__ __attribute__((aligned(16))) uint8_t lds_x[kSmX];
  __shared__ __attribute__((aligned(16))) uint8_t lds_sc[kSmWaves][kSmSc];
  __shared__ uint32_t lds_row[32 * MT];
  __shared__ MxItem lds_item[2];
  __shared__ int lds_wave[kSmWaves];
  const int tid = threadIdx.x, lane = tid % kWave, half = lane / 32, col = lane % 32;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
  const int R = a.R, I = R / 2, nb = a.nb, S = (nb + kStB - 1) / kStB, SP = (S + PD - 1) / PD * PD;
  const int row_bytes = a.row_bytes, pieces = row_bytes / 16, xsc = S * 128;   // xsc: a row's scales
  const uint32_t wq_n = (uint32_t)R * (16 * nb), ws_n = (uint32_t)R * nb;

  // The deal, lane = workgroup, neighbouring lanes on one XCD: whole passes while
  // there are as many as lanes; then of each of the `rest` passes left the first
  // `cut` tiles to a lane of its own, and the tiles behind them to the `others`.
  // Every run begins with its pass's activation rows, so runs are few:
  //   as many others as passes or more: `helpers` a pass, equal runs;
  //   fewer: even runs over all of them, a cut that makes up for a run being
  //     several (its rows taken as four tiles);
  //   fewer, gate_up, clearly (rest : others above 9 : 8): a helper takes the
  //     whole remainder of its passes, a multiple of 8 tiles, as eight waves take
  //     a tile each in one round; often there is no cut at all. The border lies
  //     between 132 and 146 passes of the sizes below, not measured at others.
  // Measured, even runs always and this deal: gate_up K = 2048, 128 tokens (120
  // passes) 48.3 and 46.2 us, 1024 (146) 63.1 and 60.3, 2048 (202) 80 and 75, 640
  // (132, helpers' whole remainders) 56.2 and 58.8; 18 passes 28.5 and 20.8; down
  // I = 768, 1999 tokens, the whole remainders 88 and 96, for its stores of y keep
  // all CUs busy to the end.
  const int lane_id = blockIdx.x % kXcds * (kSmBlocks / kXcds) + blockIdx.x / kXcds, nt = a.ntiles;
  // kOwn: this thread's two experts' rows and first pass, as k_mx_prepare lists them
  static_assert(kMaxExperts == 2 * kSmThreads);
  int r_lo = 0, m_0 = 0, m_1 = 0, first = 0, passes;
  if constexpr (kOwn) {
    r_lo = a.off[min(2 * tid, a.E)];
    const int mid = a.off[min(2 * tid + 1, a.E)];
    m_0 = mid - r_lo;
    m_1 = a.off[min(2 * tid + 2, a.E)] - mid;
    int sum = cdiv(m_0, 32 * MT) + cdiv(m_1, 32 * MT);
    first = -sum;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int o = __shfl_up(sum, d, kWave);
      if (lane >= d) sum += o;
    }
    if (lane == kWave - 1) lds_wave[wave] = sum;
    lds_barrier();
    first += sum;
    passes = 0;
#pragma unroll
    for (int i = 0; i < kSmWaves; ++i) {
      if (i < wave) first += lds_wave[i];
      passes += lds_wave[i];
    }
    passes = __builtin_amdgcn_readfirstlane(passes);
  } else {
    passes = a.items[0].e;
  }
  // pass idx into lds_item: by the thread that has its expert
  auto find = [&](int idx, MxItem* out) __attribute__((always_inline)) {
    const int n0 = cdiv(m_0, 32 * MT), n1 = cdiv(m_1, 32 * MT), i = idx - first;
    if (i < 0 || i >= n0 + n1) return;
    const bool second = i >= n0;
    const int m = second ? m_1 : m_0, per = cdiv(m, second ? n1 : n0), r = (second ? i - n0 : i) * per;
    *out = MxItem{2 * tid + second, (second ? r_lo + m_0 : r_lo) + r, max(0, min(per, m - r)), 0};
  };

  const int full = passes / kSmBlocks, rest = passes % kSmBlocks, others = kSmBlocks - rest;
  const int helpers = rest > 0 ? others / rest : 0;
  int cut = nt, u = 0, end = 0;   // even runs: u .. end - 1 of the tiles behind the cuts
  bool even = false;
  if (helpers > 0) {
    cut = cdiv(nt, helpers + 1);
  } else if (!GU || 8 * rest < 9 * others) {
    even = true;
    cut = min(nt, max(cdiv(rest * nt, kSmBlocks), (rest * (nt + 4) - 4 * others) / kSmBlocks));
    if (lane_id >= rest) {
      const int64_t tiles = (int64_t)rest * (nt - cut);
      u = (int)(tiles * (lane_id - rest) / others);
      end = (int)(tiles * (lane_id - rest + 1) / others);
    }
  } else {
    // a round, a tile a wave, takes S stages, a pass's rows about six: the
    // rounds r at which both are alike, rounded either way, or all
    constexpr int kStart = 6;
    const int rounds = cdiv(nt, kSmWaves), shared = cdiv(rest, others);
    auto cost = [&](int r) { return max(r * S + kStart, r < rounds ? shared * ((rounds - r) * S + kStart) : 0); };
    const int r = (int)(((int64_t)shared * rounds * S + (shared - 1) * kStart) / ((shared + 1) * S));
    if (min(cost(r), cost(r + 1)) < cost(rounds)) cut = min(nt, (cost(r) < cost(r + 1) ? r : r + 1) * kSmWaves);
  }
  struct Run {
    int idx, t0, tend;   // tiles t0 .. tend - 1 of a pass; idx < 0: no more
  };
  auto next_run = [&](int seg) __attribute__((always_inline)) -> Run {
    if (seg < full) return {seg * kSmBlocks + lane_id, 0, nt};
    seg -= full;
    const int j = lane_id - rest;
    if (j < 0) return {seg == 0 ? full * kSmBlocks + lane_id : -1, 0, cut};
    if (helpers > 0) {
      const int i = j / helpers, per = cdiv(nt - cut, helpers), t0 = cut + (j - i * helpers) * per;
      return {seg == 0 && i < rest && t0 < nt ? full * kSmBlocks + i : -1, t0, min(nt, t0 + per)};
    }
    if (even) {
      if (u >= end) return {-1, 0, 0};
      const int i = u / (nt - cut), t0 = cut + (u - i * (nt - cut)), tend = min(nt, t0 + (end - u));
      u += tend - t0;
      return {full * kSmBlocks + i, t0, tend};
    }
    const int i = j * rest / others + seg;
    return {cut < nt && i < (j + 1) * rest / others ? full * kSmBlocks + i : -1, cut, nt};
  };

  Run next = next_run(0);
  if constexpr (kOwn) {
    find(next.idx, &lds_item[0]);
    lds_barrier();
  }
  for (int seg = 0; next.idx >= 0; ++seg) {
    const int idx = next.idx, t0 = next.t0, tend = next.tend;
    next = next_run(seg + 1);
    const MxItem it = kOwn ? lds_item[seg & 1] : a.items[1 + idx];
    const int e = __builtin_amdgcn_readfirstlane(it.e), r0 = __builtin_amdgcn_readfirstlane(it.r0),
              m = __builtin_amdgcn_readfirstlane(it.m);
    const uint8_t* wq = a.wq + (size_t)e * wq_n;
    const uint8_t* ws = a.ws + (size_t)e * ws_n;
    // offsets of the lane's row of tile 0; tstep rows further on for each tile
    const int n0 = GU ? (col < 16 ? col : I + col - 16) : col;
    constexpr int tstep = GU ? 16 : 32;
    // a lane loads piece lane % 4 of its quad's four rows (mx_transpose)
    const uint32_t qo = (uint32_t)(n0 - col % 4) * (16 * nb) + 64 * half + 16 * (lane % 4);

    // stage s of the wave's tile t, or past SP of its next one
    u32x4 w[PD][4];
    auto load_w = [&](int t, int s, int d) __attribute__((always_inline)) {
      if (s >= SP) {
        s -= SP;
        t += kSmWaves;
      }
      const mx_rsrc q = mx_buffer(wq, s < S && t < tend ? wq_n : 0);
      const uint32_t o = qo + ((uint32_t)(t * tstep) * (16 * nb) + 128 * s);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[d][j] = mx_get16(q, o + (uint32_t)(j * 16 * nb));
    };
    // scales of tile t, blocks 64 g and on (g past the last group: of the next tile)
    const int groups = SM == MxSc::kRun ? 1 : (nb + kSmGroup - 1) / kSmGroup;
    u32x4 sr[2];
    auto load_sc = [&](int t, int g) __attribute__((always_inline)) {
      if (g >= groups) {
        g = 0;
        t += kSmWaves;
      }
      const mx_rsrc r = mx_buffer(ws, t < tend ? ws_n : 0);
      const uint32_t b0 = (uint32_t)(t * tstep) * nb;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int p = lane + i * kWave;
        if constexpr (SM == MxSc::kRun) {
          // 2 nb pieces; for gate_up the second half is the run of up rows
          sr[i] = mx_get16(r, b0 + 16 * p + (GU && p >= nb ? (uint32_t)(I - 16) * nb : 0u));
        } else {
          // piece p % 4 of row p / 4
          const int row = p / 4, n = GU && row >= 16 ? I + row - 16 : row;
          const uint32_t o = b0 + (uint32_t)n * nb + kSmGroup * g + 16 * (p % 4);
          if constexpr (SM == MxSc::kPiece) sr[i] = mx_get16(r, o);
          else sr[i] = u32x4{mx_get4(r, o), mx_get4(r, o + 4), mx_get4(r, o + 8), mx_get4(r, o + 12)};
        }
      }
    };
    auto store_sc = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) *reinterpret_cast<u32x4*>(&lds_sc[wave][mx_sc_at(16 * (lane + i * kWave))]) = sr[i];
    };
    const int lsc = col * (SM == MxSc::kRun ? nb : kSmGroup) + 4 * half;

    int t = t0 + wave;
    if constexpr (kOwn) {
      // Rows quantised by the workgroup, eight values a thread and kAhead times
      // at once. The first ones' loads go out between the weights' stages 1 and 2
      // and the stages from 4 on only behind them: with all of them first, the
      // rows arrived after 13 us of weights (128 tokens: 48.5 us; so 47.0).
      // Blocks behind a row: zero codes, scale 1.
      constexpr int kAhead = sizeof(XT) == 4 ? 4 : 8, kFirst = 2, kThen = PD < 4 ? PD : 4;
      const XT* x = static_cast<const XT*>(a.raw);
      const int per = 4 * kStB * S, n = m * per;   // a multiple of 4: a block's four lanes are all in or all out
      decltype(mx_raw8(x)) v[kAhead];
      auto load_x = [&](int p0) __attribute__((always_inline)) {
        int row[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          row[i] = r0 + min(p0 + i * kSmThreads, n - 1) / per;
          if constexpr (GU) row[i] = a.sorted_pairs[row[i]];
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int p = min(p0 + i * kSmThreads, n - 1), g = min(p % per, 4 * nb - 1);
          v[i] = mx_raw8(x + (size_t)(GU ? row[i] / a.topk : row[i]) * (nb * kMxBlock) + 8 * g);
        }
      };
#pragma unroll
      for (int d = 0; d < kFirst; ++d) load_w(t, d, d);
      load_sc(t, 0);
      load_x(tid);
#pragma unroll
      for (int d = kFirst; d < kThen; ++d) load_w(t, d, d);
      lds_barrier();   // no wave still reads the last pass's
      find(next.idx, &lds_item[(seg + 1) & 1]);
      for (int p0 = tid; p0 < n; p0 += kAhead * kSmThreads) {
        if (p0 != tid) load_x(p0);
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int p = p0 + i * kSmThreads, row = p / per, g = p - row * per;
          const bool in = g < 4 * nb;
          float f[8];
          mx_floats(v[i], f);
          int sc;
          const uint32_t c = mx_quant8(f, sc);
          if (p < n) {
            uint8_t* o = &lds_x[row * row_bytes];
            *reinterpret_cast<uint32_t*>(o + 4 * g) = in ? c : 0u;
            if ((g & 3) == 0) o[xsc + g / 4] = (uint8_t)(in ? sc : 127);
          }
        }
      }
#pragma unroll
      for (int d = kThen; d < PD; ++d) load_w(t, d, d);
    } else {
#pragma unroll
      for (int d = 0; d < PD; ++d) load_w(t, d, d);
      load_sc(t, 0);

      // the pass's activation rows
      lds_barrier();   // no wave still reads the last pass's
      if (tid < m) lds_row[tid] = (uint32_t)(GU ? a.sorted_pairs[r0 + tid] / a.topk : r0 + tid) * (uint32_t)row_bytes;
      lds_barrier();
      const int n = m * pieces;
      const mx_rsrc x = mx_buffer(a.x, a.x_n);
      for (int p0 = wave * kWave; p0 < n; p0 += kSmThreads) {
        const int p = p0 + lane, row = p / pieces;
        if (p < n) mx_get16_lds(x, &lds_x[16 * p0], lds_row[row] + 16 * (p - row * pieces));
      }
      __builtin_amdgcn_s_waitcnt(0x0f70);   // vmcnt(0)
    }
    lds_barrier();

    auto run = [&](auto na_c) __attribute__((always_inline)) {
      constexpr int NA = decltype(na_c)::value;   // live 32-row tiles of the pass
      // Operands from LDS run one step ahead of the products (two waves a SIMD
      // do not hide its latency otherwise): the activation codes of step j + 1,
      // and with a stage's last step the next one's codes and scales, on into
      // the next tile, whose stages begin with 0 again.
      u32x4 xv[2][NA];
      uint32_t xs[NA], xn[NA], sw, sn = 0;
      auto read_x = [&](int s, int j, u32x4 (&v)[NA]) __attribute__((always_inline)) {
        const uint8_t* x = &lds_x[col * row_bytes + 128 * s + 64 * half + 16 * j];
#pragma unroll
        for (int q = 0; q < NA; ++q) v[q] = *reinterpret_cast<const u32x4*>(x + 32 * q * row_bytes);
      };
      auto read_xs = [&](int s, uint32_t (&v)[NA]) __attribute__((always_inline)) {
        const uint8_t* x = &lds_x[col * row_bytes + xsc + kStB * s + 4 * half];
#pragma unroll
        for (int q = 0; q < NA; ++q) v[q] = *reinterpret_cast<const uint32_t*>(x + 32 * q * row_bytes);
      };
      // scales of the wave's weight rows, stage s (what is read past the row's last block is masked)
      auto read_sw = [&](int s) __attribute__((always_inline)) {
        uint32_t v;
        if constexpr (SM == MxSc::kRun) {
          const int o = lsc + kStB * s;   // the four bytes may start anywhere
          const uint32_t lo = *reinterpret_cast<const uint32_t*>(&lds_sc[wave][mx_sc_at(o & ~3)]);
          const uint32_t hi = *reinterpret_cast<const uint32_t*>(&lds_sc[wave][mx_sc_at((o & ~3) + 4)]);
          v = __builtin_amdgcn_alignbyte(hi, lo, o & 3);
        } else {
          v = *reinterpret_cast<const uint32_t*>(&lds_sc[wave][mx_sc_at(lsc + kStB * (s % kStB))]);
        }
        return mx_mask_scales(v, nb - kStB * s - 4 * half);
      };
      if (t < tend) {
        read_x(0, 0, xv[0]);
        read_xs(0, xs);
      }
      for (; t < tend; t += kSmWaves) {
        f32x16 acc[NA];
#pragma unroll
        for (int q = 0; q < NA; ++q) acc[q] = f32x16{};
        for (int s0 = 0; s0 < SP; s0 += PD) {
          if (s0 % kStB == 0) {   // this group's scales into LDS, the next one's on their way
            wave_lds_order();   // every lane has read the last group's
            store_sc();
            wave_lds_order();
            load_sc(t, s0 / kStB + 1);
            sn = read_sw(s0);
          }
#pragma unroll
          for (int d = 0; d < PD; ++d) {
            const int s = s0 + d;
            // stages past the last one multiply zero weights with the first stage's codes
            const int sx = s < S ? s : 0, next = s + 1 < S ? s + 1 : 0;
            sw = sn;
            mx_transpose(w[d]);
            auto step = [&](auto jc) __attribute__((always_inline)) {
              constexpr int J = decltype(jc)::value;
              if constexpr (J < 3) {
                read_x(sx, J + 1, xv[(J + 1) % 2]);
              } else {
                read_x(next, 0, xv[0]);
                read_xs(next, xn);
                sn = read_sw(next);
              }
              __builtin_amdgcn_sched_barrier(0);
#pragma unroll
              for (int q = 0; q < NA; ++q) acc[q] = mx_mfma32<J, J>(xv[J % 2][q], w[d][J], acc[q], xs[q], sw);
              __builtin_amdgcn_sched_barrier(0);
            };
            step(std::integral_constant<int, 0>{});
            step(std::integral_constant<int, 1>{});
            step(std::integral_constant<int, 2>{});
            step(std::integral_constant<int, 3>{});
#pragma unroll
            for (int q = 0; q < NA; ++q) xs[q] = xn[q];
            load_w(t, s + PD, d);   // into the registers just used
          }
        }
        mx_store<GU, NA>(acc, t, R, r0, m, out0, out1);
      }
    };
    const int na = (m + 31) / 32;
    if (MT >= 4 && na == 4) run(std::integral_constant<int, 4>{});
    else if (MT >= 3 && na == 3) run(std::integral_constant<int, 3>{});
    else if (MT >= 2 && na == 2) run(std::integral_constant<int, 2>{});
    else run(std::integral_constant<int, 1>{});
  }
}

// ---------------------------------------------------------------------------
// Long rows: activation rows in stages through LDS. A work item is one pass x
// 128 weight rows, a workgroup of 4 waves, a 32-row tile each; weights and
// their scales from memory into registers two stages ahead, activation rows
// double-buffered in LDS.

constexpr int kRgThreads = 256;
constexpr int kRgWaves = kRgThreads / kWave;
constexpr int kRgTile = 144;                 // a row's stage in LDS: 128 B of codes, 8 scales, 8 B unused
constexpr int kRgPieces = kRgTile / 16;
constexpr int kRgMt = 3;

template <bool GU, typename AT>
__global__ void __launch_bounds__(kRgThreads, 2)
k_mx_ring(const MxArgs a, float* __restrict__ out0, AT* __restrict__ out1) {
  constexpr int PD = 2;   // stages of weights in flight; also the parity of the LDS buffers
  __shared__ __attribute__((aligned(16))) uint8_t buf[2][32 * kRgMt * kRgTile];
  const int ntg = (a.ntiles + kRgWaves - 1) / kRgWaves;
  const int i = blockIdx.x / ntg;
  if (i >= a.items[0].e) return;
  const MxItem it = a.items[1 + i];
  const int e = it.e, r0 = it.r0, m = it.m;
  const int tid = threadIdx.x, lane = tid % kWave, half = lane / 32, col = lane % 32;
  const int tile = blockIdx.x % ntg * kRgWaves + __builtin_amdgcn_readfirstlane(tid / kWave);
  const int R = a.R, I = R / 2, nb = a.nb, S = (nb + kStB - 1) / kStB;
  const uint32_t wq_n = (uint32_t)R * (16 * nb), ws_n = (uint32_t)R * nb;
  const uint8_t* wq = a.wq + (size_t)e * wq_n;
  const uint8_t* ws = a.ws + (size_t)e * ws_n;
  const bool live = tile < a.ntiles;   // dead waves read zeros; they still copy and meet the barriers
  const int n = GU ? tile * 16 + (col < 16 ? col : I + col - 16) : tile * 32 + col;
  const uint32_t qo = (uint32_t)n * (16 * nb) + 64 * half, so = (uint32_t)n * nb + 4 * half;
  u32x4 w[PD][4];
  uint32_t wsc[PD];
  auto load_w = [&](int s, int d) __attribute__((always_inline)) {
    const bool on = live && s < S;
    const mx_rsrc q = mx_buffer(wq, on ? wq_n : 0), c = mx_buffer(ws, on ? ws_n : 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) w[d][j] = mx_get16(q, qo + 128 * s + 16 * j);
    // rows of scales may start anywhere: two aligned words hold the four bytes
    const uint32_t o = so + kStB * s;
    wsc[d] = mx_mask_scales(__builtin_amdgcn_alignbyte(mx_get4(c, (o & ~3u) + 4), mx_get4(c, o & ~3u), o & 3),
                            nb - kStB * s - 4 * half);
  };
#pragma unroll
  for (int d = 0; d < PD; ++d) load_w(d, d);

  auto run = [&](auto na_c) __attribute__((always_inline)) {
    constexpr int NA = decltype(na_c)::value;   // live 32-row tiles of the pass
    // activation pieces this thread copies: 16 bytes of a row's stage, pieces
    // tid, tid + 256, .. of the pass (rows past it repeat its last one); piece 8
    // of a row is its stage's scales and the 8 bytes behind them
    constexpr int kPieces = 32 * NA * kRgPieces, kCopies = (kPieces + kRgThreads - 1) / kRgThreads;
    uint32_t xo[kCopies];
    int xstep[kCopies];
#pragma unroll
    for (int q = 0; q < kCopies; ++q) {
      const int p = min(tid + q * kRgThreads, kPieces - 1), row = p / kRgPieces, c = p - row * kRgPieces;
      const int r = r0 + min(row, m - 1);
      xo[q] = (uint32_t)(GU ? a.sorted_pairs[r] / a.topk : r) * (uint32_t)a.row_bytes + (c < kStB ? 16 * c : 128 * S);
      xstep[q] = c < kStB ? 128 : kStB;
    }
    u32x4 xr[2][kCopies];
    auto load_x = [&](int s, u32x4 (&xr)[kCopies]) __attribute__((always_inline)) {
      const mx_rsrc q = mx_buffer(a.x, s < S ? a.x_n : 0);
#pragma unroll
      for (int i = 0; i < kCopies; ++i) xr[i] = mx_get16(q, xo[i] + xstep[i] * s);
    };
    auto store_x = [&](int b, const u32x4 (&xr)[kCopies]) __attribute__((always_inline)) {
      // threads past the last piece write that piece again: no branch
#pragma unroll
      for (int i = 0; i < kCopies; ++i)
        *reinterpret_cast<u32x4*>(&buf[b][16 * min(tid + i * kRgThreads, kPieces - 1)]) = xr[i];
    };

    f32x16 acc[NA];
#pragma unroll
    for (int q = 0; q < NA; ++q) acc[q] = f32x16{};
    load_x(0, xr[0]);
    load_x(1, xr[1]);
    store_x(0, xr[0]);
    load_x(2, xr[0]);
    lds_barrier();
    // a stage past the last one (S odd) adds products with zero codes
    for (int s0 = 0; s0 < S; s0 += PD) {
#pragma unroll
      for (int d = 0; d < PD; ++d) {
        const int s = s0 + d;
        const uint8_t* x = &buf[d][col * kRgTile + 64 * half];
        uint32_t xs[NA];
#pragma unroll
        for (int q = 0; q < NA; ++q)
          xs[q] = *reinterpret_cast<const uint32_t*>(&buf[d][(32 * q + col) * kRgTile + 128 + 4 * half]);
        auto step = [&](auto jc) __attribute__((always_inline)) {
          constexpr int J = decltype(jc)::value;
#pragma unroll
          for (int q = 0; q < NA; ++q) {
            const u32x4 xv = *reinterpret_cast<const u32x4*>(x + 32 * q * kRgTile + 16 * J);
            acc[q] = mx_mfma32<J, J>(xv, w[d][J], acc[q], xs[q], wsc[d]);
          }
        };
        step(std::integral_constant<int, 0>{});
        step(std::integral_constant<int, 1>{});
        step(std::integral_constant<int, 2>{});
        step(std::integral_constant<int, 3>{});
        __builtin_amdgcn_sched_barrier(0);
        load_w(s + PD, d);
        store_x(d ^ 1, xr[d ^ 1]);
        load_x(s + 3, xr[d ^ 1]);
        lds_barrier();
      }
    }
    if (live) mx_store<GU, NA>(acc, tile, R, r0, m, out0, out1);
  };
  const int na = (m + 31) / 32;
  if (na == 3) run(std::integral_constant<int, 3>{});
  else if (na == 2) run(std::integral_constant<int, 2>{});
  else run(std::integral_constant<int, 1>{});
}

// ---------------------------------------------------------------------------

// What the products need ready, in one launch: workgroup 0 lists the passes
// (an expert of m > 0 rows has n = ceil(m / rows) of them, of ceil(m / n) rows
// each, so that they take alike), the others quantise the activation rows, eight
// values a thread, into rows of nbp blocks of codes and their scales; the blocks
// behind a row hold zero codes with scale 1.
template <typename XT>
__global__ void __launch_bounds__(kPrThreads)
k_mx_prepare(const XT* __restrict__ x, int64_t n8, int nb, int nbp, int row_bytes, uint8_t* __restrict__ rows_out,
             const int32_t* __restrict__ off, int E, int rows, MxItem* __restrict__ items) {
  const int tid = threadIdx.x;
  if (blockIdx.x == 0) {
    __shared__ int s_off[kMaxExperts + 1], s_first[kMaxExperts + 1];
    __shared__ int s_wave[kPrThreads / kWave];
    for (int i = tid; i <= E; i += kPrThreads) s_off[i] = off[i];
    __syncthreads();
    constexpr int kPer = kMaxExperts / kPrThreads;   // consecutive experts a thread counts
    int n[kPer], sum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int e = kPer * tid + j;
      n[j] = e < E ? (s_off[e + 1] - s_off[e] + rows - 1) / rows : 0;
      sum += n[j];
    }
    int inc = sum;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
      const int o = __shfl_up(inc, d, kWave);
      if (tid % kWave >= d) inc += o;
    }
    if (tid % kWave == kWave - 1) s_wave[tid / kWave] = inc;
    __syncthreads();
    int first = inc - sum;
    for (int w = 0; w < tid / kWave; ++w) first += s_wave[w];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int e = kPer * tid + j;
      if (e < E) s_first[e] = first;
      first += n[j];
      if (e == E - 1) s_first[E] = first;
    }
    __syncthreads();
    const int total = s_first[E];
    if (tid == 0) items[0] = MxItem{total, 0, 0, 0};
    for (int i = tid; i < total; i += kPrThreads) {
      int lo = 0, hi = E;   // the last expert whose first pass is at or before i: it has passes
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (s_first[mid] <= i) lo = mid;
        else hi = mid;
      }
      const int m = s_off[lo + 1] - s_off[lo], passes = s_first[lo + 1] - s_first[lo];
      const int per = (m + passes - 1) / passes, p = i - s_first[lo];
      items[1 + i] = MxItem{lo, s_off[lo] + p * per, max(0, min(per, m - p * per)), 0};
    }
    return;
  }
  const int64_t i = (int64_t)(blockIdx.x - 1) * kPrThreads + tid;
  float v[8] = {};
  const int64_t row = (i / 4) / nbp;
  const int b = (int)(i / 4 - row * nbp);
  if (i < n8 && b < nb) mx_load8_once(x + (row * nb + b) * kMxBlock + 8 * (i & 3), v);
  int s;
  const uint32_t c = mx_quant8(v, s);   // n8 is a multiple of 4: a block's four lanes are all in or all out
  if (i >= n8) return;
  uint8_t* o = rows_out + row * row_bytes;
  *reinterpret_cast<uint32_t*>(o + 16 * b + 4 * (i & 3)) = c;
  if ((i & 3) == 0) o[16 * nbp + b] = (uint8_t)(b < nb ? s : 127);
}

// out[t, h .. h + 3] = sum_j w[t, j] y[pos[t k + j], h .. h + 3], slot order.
// Bound by the read of y: 1999 tokens, top 8, H = 2048 in 22 us, 147 MB at 6.7 TB/s.
__global__ void __launch_bounds__(kPrThreads)
k_mx_combine(const float* __restrict__ y, int H, int k, const float* __restrict__ tw, const int32_t* __restrict__ pos,
             float* __restrict__ out) {
  const int64_t t = blockIdx.x;
  const int h = 4 * (blockIdx.y * kPrThreads + threadIdx.x);
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

// How a product of rows of K is run: the passes' rows and the kernel
struct MxPlan {
  int nb, nbp, row_bytes, mt;
  bool stream, own;   // own: the stream kernel finds the passes and quantises the rows itself
  MxPlan(int K, int64_t P, int E) {
    nb = K / kMxBlock;
    nbp = cdiv(nb, kStB) * kStB;
    row_bytes = (cdiv(17 * nbp, 16) | 1) * 16;   // an odd number of 16-byte pieces: 16 rows meet all LDS banks
    // Rows per pass: 32, quantised by the kernel itself (no second launch), while
    // an expert has eight on average; up to 128, as far as they fit LDS, for more.
    // Both at K = 2048, N = 1536, 32 and 128 rows: 128 experts, 4 pairs each 40.5
    // and 41.0 us, 8 each 46.9 and 47.5, 16 each 57.6 and 50.7, 32 each 73 and 55;
    // 8 experts, 8 pairs each 13.5 and 11.9 (the launch not counted), 16 each 18.5
    // and 12.4. 64 rows are within 1 us of 128 up to 20 pairs an expert and 7 us
    // behind at 64.
    const int want = P <= 8 * (int64_t)E ? 1 : 4;
    // Longer rows than 64 blocks: this kernel as far as one pass of 32 rows fits, also
    // where the other takes passes of 96. Both, 32 experts, top 4, N = 1536: K = 2304,
    // 128 and 2048 tokens 22.9 and 25.8 us, 53 and 60; 4096 30.6 and 42.8, 76 and 101;
    // 7168 47 and 69, 163 and 170; 8192 58 and 79, 166 and 190.
    const int fit = kSmX / 32 / row_bytes;   // the product overflows for the longest rows
    stream = fit >= 1 && (nb <= kSmGroup || nb % 4 == 0);
    mt = stream ? (want <= fit ? want : fit >= 2 ? 2 : 1) : kRgMt;
    own = stream && mt == 1 && nb <= kSmGroup;
  }
  // every non-empty expert has at most one pass that is not full
  int64_t passes(int64_t P, int E) const { return P / (32 * mt) + (P < E ? P : E); }
};

MxWorkspace::MxWorkspace(int64_t rows, int K, int64_t P, int E) {
  const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  const MxPlan plan(K, P, E);
  items = total = 0;
  if (plan.own) return;
  items = up((size_t)rows * plan.row_bytes + 16);   // reads of a row's scales run up to 8 bytes past it
  total = items + up((size_t)(1 + plan.passes(P, E)) * sizeof(MxItem));
}

// workgroups of k_mx_ring
static int64_t mx_ring_grid(const MxPlan& plan, int64_t P, int E, int R) {
  return plan.passes(P, E) * cdiv(R / 32, kRgWaves);
}

// a launch holds fewer than 2^32 threads; the other kernels' grids stay far below
bool mx_launch_fits(int K, int64_t P, int E, int R) {
  const MxPlan plan(K, P, E);
  return plan.stream || mx_ring_grid(plan, P, E, R) * kRgThreads < (int64_t)1 << 32;
}

template <bool GU, typename XT, typename AT>
static hipError_t mx_grouped(const XT* x, int64_t rows, int K, int64_t P, const uint8_t* codes, const uint8_t* scales,
                             int E, int R, int topk, const int32_t* expert_off, const int32_t* sorted_pairs,
                             uint8_t* ws, float* out0, AT* out1, hipStream_t st) {
  const MxWorkspace lay(rows, K, P, E);
  const MxPlan plan(K, P, E);
  const int64_t n8 = rows * plan.nbp * 4, qgrid = 1 + (n8 + kPrThreads - 1) / kPrThreads;
  const int ntiles = R / 32;
#define I8H_MX(M, D, S, X) k_mx_stream<GU, M, D, MxSc::S, X><<<kSmBlocks, kSmThreads, 0, st>>>(a, out0, out1)
  if (plan.own) {
    const MxArgs a = {nullptr, codes, scales, 0, plan.row_bytes, E, R, plan.nb, topk, ntiles, nullptr, x, expert_off,
                      sorted_pairs};
    // Depth of the prefetch: what the registers leave, less for short rows, whose
    // stages are rounded up to it: those past the last are products of zeros (up to
    // two of three at K <= 256, three of eight at five stages)
    if (plan.nb <= 3 * kStB) I8H_MX(1, 3, kRun, XT);
    else if (plan.nb <= 4 * kStB) I8H_MX(1, 4, kRun, XT);
    else I8H_MX(1, 8, kRun, XT);
    return hipGetLastError();
  }
  MxItem* items = reinterpret_cast<MxItem*>(ws + lay.items);
  k_mx_prepare<<<(unsigned)qgrid, kPrThreads, 0, st>>>(x, n8, plan.nb, plan.nbp, plan.row_bytes, ws, expert_off, E,
                                                       32 * plan.mt, items);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const MxArgs a = {ws, codes, scales, (uint32_t)(rows * plan.row_bytes + 16), plan.row_bytes, E, R, plan.nb, topk,
                    ntiles, items, nullptr, nullptr, sorted_pairs};
  if (!plan.stream) {
    k_mx_ring<GU><<<(unsigned)mx_ring_grid(plan, P, E, R), kRgThreads, 0, st>>>(a, out0, out1);
  } else if (plan.nb <= kSmGroup) {
    if (plan.nb <= 3 * kStB) I8H_MX(4, 3, kRun, void);   // K = 768, 2048 tokens: 84 us, two deep 87; K = 2048: 85, 81
    else I8H_MX(4, 2, kRun, void);
  } else if (plan.nb % 16 == 0) {
    if (plan.mt == 1) I8H_MX(1, 8, kPiece, void);
    else I8H_MX(2, 2, kPiece, void);
  } else {
    if (plan.mt == 1) I8H_MX(1, 8, kWord, void);
    else I8H_MX(2, 2, kWord, void);
  }
#undef I8H_MX
  return hipGetLastError();
}

hipError_t launch_gateup_mxfp4(const uint16_t* x, int T, int K, const uint8_t* codes, const uint8_t* scales, int E,
                               int N, int k, const int32_t* expert_off, const int32_t* sorted_pairs, float* gu,
                               void* act, bool act_bf16, uint8_t* ws, hipStream_t st) {
  const int64_t P = (int64_t)T * k;
  return act_bf16 ? mx_grouped<true>(x, T, K, P, codes, scales, E, N, k, expert_off, sorted_pairs, ws, gu,
                                     static_cast<uint16_t*>(act), st)
                  : mx_grouped<true>(x, T, K, P, codes, scales, E, N, k, expert_off, sorted_pairs, ws, gu,
                                     static_cast<float*>(act), st);
}

hipError_t launch_down_mxfp4(const void* act, bool act_bf16, int T, int I, const uint8_t* codes,
                             const uint8_t* scales, int E, int H, int k, const float* tw, const int32_t* expert_off,
                             const int32_t* pos, uint8_t* ws, float* y, float* out, hipStream_t st) {
  const int64_t P = (int64_t)T * k;
  float* const none = nullptr;
  const hipError_t err =
      act_bf16 ? mx_grouped<false>(static_cast<const uint16_t*>(act), P, I, P, codes, scales, E, H, k, expert_off,
                                   nullptr, ws, y, none, st)
               : mx_grouped<false>(static_cast<const float*>(act), P, I, P, codes, scales, E, H, k, expert_off,
                                   nullptr, ws, y, none, st);
  if (err != hipSuccess) return err;
  k_mx_combine<<<dim3(T, cdiv(H / 4, kPrThreads)), kPrThreads, 0, st>>>(y, H, k, tw, pos, out);
  return hipGetLastError();
}

}  // namespace i8h
