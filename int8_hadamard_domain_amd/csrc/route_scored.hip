// Experts by scores: softmax or sigmoid over all experts, a bias for balance,
// groups, top-k, weights with or without renormalisation; then the stable
// permutation of moe_route_permute.
//
// The order of the choice values s + bias is that of float64: two experts
// whose float32 values round alike must not change places. A token is chosen
// in float32 first, with a bound on the error of each comparison that decides
// (the border of the groups that stay, the border of the chosen, neighbours
// among them); only where two values lie within that bound is the token done
// again in float64. Without a bias the logits themselves are compared, exactly.
//
// Kernels
//   k_scored_small    up to 32 tokens: everything in one workgroup
//   k_scored_rows     per chunk of tokens: a wave per token chooses its
//                     experts; the chunk's histogram
//   k_scored_scan     more than 256 chunks: the histograms' running sums
//   k_scored_scatter  per chunk: first rows of the experts, stable ranks
//
// Measured (medians on MI355X): one token of 128 experts 5.2 us in one launch;
// 128 tokens 4.6 (rows) + 4.2 (scatter); 1999 tokens of 160 experts, 3 of 8
// groups, 9.3 + 5.3; 16384 tokens of 256 experts, 4 of 8 groups, 23.9 + 5.9
// (the bytes alone 3.7). Few tokens: the chain of dependent steps of one token,
// 2.3 us, and of the permutation. Many: the vector unit's issue, 372
// instructions a token by a whole wave. The rule, the lists and the float64 path
// need more scalar registers than there are: 33 to 51 of them (148 past 512
// experts) are kept in lanes of vector registers, which costs vector instructions.

#include <algorithm>

#include "common.hpp"
#include "launch.hpp"
#include "topk.hpp"

namespace i8h {

namespace {

constexpr int kScChunkTokens = 64;           // most tokens of a chunk; its counts fit in bytes
constexpr int kScFill = 256;                 // chunks while there are tokens for them: one a CU
constexpr int kScScanFrom = 256;             // chunks above which the running sums take a launch of their own
constexpr int kScPairs = 512;                // most pairs of a scatter workgroup: a thread each
constexpr int kScScatterThreads = kScPairs;
constexpr int kScScanThreads = 1024;
constexpr int kScScanExperts = 16;           // experts a workgroup of the scan
constexpr int kScSmallTokens = 32;
constexpr int kScSmallThreads = 1024;

// waves of a workgroup that chooses: as many as the float64 scratch (E doubles a wave) leaves room for
template <int VPL>
constexpr int sc_waves() { return VPL <= 4 ? 16 : 64 / VPL; }

struct ScoredRule {
  const float* bias;       // [E] or NULL
  int E, k, groups, keep, top;
  int size;                // experts a group
  int lanes;               // log2 of a group's lanes, -1 where a group is not a power of two of whole lanes
  bool sigmoid, renorm;
  float scale;
};

// a lane's chosen expert; rank is its place, k or more for none
struct Choice {
  int id, rank;
  float w;
};

// a wave's scratch: the entries that may be chosen, at most one a lane, in the experts' order
struct Candidates {
  uint64_t key[kWave];       // float64's choice keys
  uint32_t k32[kWave];       // float32's choice value, or a logit's key
  int e[kWave];
  float v[kWave];            // the logit
};

// LDS that a wave's lanes hand on to each other: writes before, reads after
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Reductions over the wave to a uniform value, one vector instruction a step:
// within rows of 16 lanes by shifts, then row 0 into 1, 2 into 3, both into
// the last. `none` is the value that lanes without a partner take.
template <typename Op>
__device__ __forceinline__ uint32_t wave_reduce(uint32_t v, uint32_t none, const Op& op) {
#define I8H_STEP(CTRL, ROWS) v = op(v, (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, CTRL, ROWS, 0xF, false));
  I8H_STEP(0x111, 0xF) I8H_STEP(0x112, 0xF) I8H_STEP(0x114, 0xF) I8H_STEP(0x118, 0xF)   // row_shr 1, 2, 4, 8
  I8H_STEP(0x142, 0xA) I8H_STEP(0x143, 0xC)                                             // row_bcast 15, 31
#undef I8H_STEP
  return (uint32_t)__builtin_amdgcn_readlane((int)v, kWave - 1);
}
__device__ __forceinline__ uint32_t reduce_max(uint32_t v) {
  return wave_reduce(v, 0u, [](uint32_t a, uint32_t b) { return max(a, b); });
}
__device__ __forceinline__ int reduce_add(int v) {
  return (int)wave_reduce((uint32_t)v, 0u, [](uint32_t a, uint32_t b) { return a + b; });
}
__device__ __forceinline__ float reduce_add(float v) {
  return __uint_as_float(wave_reduce(__float_as_uint(v), 0u, [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}
__device__ __forceinline__ float reduce_max(float v) {      // NaN only where all are
  return __uint_as_float(wave_reduce(__float_as_uint(v), __float_as_uint(-INFINITY), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}

// Order-preserving map of a float64 to an unsigned key; NaN to 0, below every number.
__device__ __forceinline__ uint64_t order_key64(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);   // -0 + 0 = +0
  const uint64_t k = (b >> 63) ? ~b : (b | 0x8000000000000000ull);
  return v == v ? k : 0ull;
}

__device__ __forceinline__ double key_value64(uint64_t k) {
  return k == 0 ? __builtin_nan("") : __builtin_bit_cast(double, (k >> 63) ? k & 0x7fffffffffffffffull : ~k);
}

template <int M>
__device__ __forceinline__ uint64_t xor_lane_u64(uint64_t v) {
  return (uint64_t)(uint32_t)xor_lane_i<M>((int)(uint32_t)v) |
         (uint64_t)(uint32_t)xor_lane_i<M>((int)(uint32_t)(v >> 32)) << 32;
}
__device__ __forceinline__ uint64_t wave_max_u64(uint64_t v) {
  v = max(v, xor_lane_u64<1>(v));
  v = max(v, xor_lane_u64<2>(v));
  v = max(v, xor_lane_u64<4>(v));
  v = max(v, xor_lane_u64<8>(v));
  v = max(v, xor_lane_u64<16>(v));
  v = max(v, xor_lane_u64<32>(v));
  return v;
}
template <int M>
__device__ __forceinline__ double add_xor(double v) {
  return v + __builtin_bit_cast(double, xor_lane_u64<M>(__builtin_bit_cast(uint64_t, v)));
}
__device__ __forceinline__ double wave_sum64(double v) {
  return add_xor<1>(add_xor<2>(add_xor<4>(add_xor<8>(add_xor<16>(add_xor<32>(v))))));
}
__device__ __forceinline__ uint64_t readlane_u64(uint64_t v, int lane) {
  return (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane) |
         (uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(v >> 32), lane) << 32;
}

// (a, b) = the two largest of (a, b) and (c, d), each pair in order
__device__ __forceinline__ void merge2(float& a, float& b, float c, float d) {
  const float low = fminf(a, c);
  a = fmaxf(a, c);
  b = fmaxf(low, fmaxf(b, d));
}

// lanes below this one whose bit is set
__device__ __forceinline__ int lanes_below_with(uint64_t m) {
  return (int)__builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0u));
}

template <int VPL>
__device__ __forceinline__ int count_from(const uint32_t (&kv)[VPL], uint32_t from) {
  int n = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) n += __popcll(__ballot(kv[i] >= from));
  return n;
}

// exp(x) to about 2 units, the rounding of x log2(e) carried along; x is held in [-128, 88] (0 there, and 2^127).
__device__ __forceinline__ float exp_carried(float x) {
  const float l2e = 1.4426950408889634f, rest = 1.925963033500e-08f;   // log2(e) = l2e + rest
  const float c = fminf(fmaxf(x, -128.0f), 88.0f), h = c * l2e;
  const float r = fmaf(c, rest, fmaf(c, l2e, -h));
  const float e = __builtin_amdgcn_exp2f(h);
  return fmaf(e * r, 0.6931471805599453f, e);
}

// Which groups stay, one bit a group, in float64 (exact order, ties to the
// lower group). `value` holds a key per entry; lds is the wave's (E keys).
template <int VPL>
__device__ __forceinline__ uint64_t groups_float64(const uint64_t (&value)[VPL], const ScoredRule& R, bool sum, int lane,
                                                   uint64_t* lds) {
  const int size = R.size;
  wave_order();
#pragma unroll
  for (int i = 0; i < VPL; ++i)
    if (VPL * lane + i < R.E) lds[VPL * lane + i] = value[i];
  wave_order();
  uint64_t worth = 0;
  if (lane < R.groups) {
    uint64_t a = 0, b = 0;                             // the two largest
#pragma unroll 4
    for (int i = 0; i < size; ++i) {
      const uint64_t x = lds[lane * size + i];
      b = max(b, min(a, x));
      a = max(a, x);
    }
    worth = sum ? order_key64(key_value64(a) + key_value64(b)) : a;
  }
  int rank = 0;
  for (int g = 0; g < R.groups; ++g) {
    const uint64_t o = readlane_u64(worth, g);
    rank += o > worth || (o == worth && g < lane) ? 1 : 0;
  }
  wave_order();
  return __ballot(lane < R.groups && rank < R.keep);
}

// One token by one wave. Lane l holds the logits v and biases b of experts
// VPL l .. VPL l + VPL - 1; lds is the wave's own (E doubles).
//
// F64 false: in float32; returns false where a comparison that decides lies
// within the error of its values, or one of them is no number. Errors, in
// units of 2^-24 (hardware exponential and reciprocal 2, a rounded product, sum
// or constant 1, an exponential's argument x its size |x|):
//   sigmoid: s (1 - s) (1.5 |l| + 2) + 3 s <= 4
//   softmax, e = exp(l - max): 3;  s = e / S: the sum's relative error is at
//     most 2.5 mean|l - max| + 2 + 10 <= 30 (the mean under the softmax is at
//     most ln 1024), so 36 / S
// A difference of two such values plus their roundings is surely of the right
// sign beyond `unit` + 2^-22 |c|, with unit twice those errors or more:
// 2^-20, for a softmax with a bias 2^-17 / S. The worth of two values takes
// twice that.
// F64 true: in float64, exactly as defined; always returns true.
template <int VPL, bool F64>
__device__ __forceinline__ bool choose(const float (&v)[VPL], const float (&b)[VPL], const ScoredRule& R, int lane,
                                       double* lds, Candidates& sc, Choice& ch) {
  const int E = R.E, k = R.k;
  const bool by_logit = R.bias == nullptr;
  const bool limited = R.keep < R.groups;
  const float log2e = 1.4426950408889634f;
  float mx = 0.0f, S = 1.0f;
  double S64 = 1.0;
  float c[VPL];              // float32's choice values, or the scores that a worth adds up
  uint64_t key[VPL];         // float64's choice keys
  uint32_t kv[VPL];          // choice keys (their upper halves), 0 for what cannot be chosen
  float unit = 0x1p-20f;
  if (!R.sigmoid) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < VPL; ++i) m = fmaxf(m, v[i]);
    mx = reduce_max(m);
    if (mx == -INFINITY || mx != mx) mx = 0.0f;        // masked whole: every score is 0
  }
  if constexpr (F64) {
    double s[VPL], sum = 0.0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      const double l = (double)v[i];
      if (R.sigmoid) s[i] = 1.0 / (1.0 + exp(-l));
      else s[i] = v[i] == -INFINITY ? 0.0 : exp(l - (double)mx);
      sum += s[i];
    }
    if (!R.sigmoid) {
      sum = wave_sum64(sum);
      S64 = sum == 0.0 ? 1.0 : sum;
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      s[i] /= S64;
      key[i] = by_logit ? (uint64_t)order_key(v[i]) << 32 : order_key64(s[i] + (double)b[i]);
    }
    if (limited) {
      uint64_t value[VPL];
#pragma unroll
      for (int i = 0; i < VPL; ++i) value[i] = by_logit && R.top == 2 ? order_key64(s[i]) : key[i];
      const uint64_t stays = groups_float64<VPL>(value, R, R.top == 2, lane, reinterpret_cast<uint64_t*>(lds));
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        const int e = min(VPL * lane + i, E - 1);
        kv[i] = (stays >> (e / R.size)) & 1 ? max((uint32_t)(key[i] >> 32), 1u) : 0u;
      }
    } else {
#pragma unroll
      for (int i = 0; i < VPL; ++i) kv[i] = max((uint32_t)(key[i] >> 32), 1u);   // NaN: 1, below every number
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (VPL * lane + i >= E) kv[i] = 0u;
  } else {
    if (mx == INFINITY) return false;
    if (!by_logit || (limited && R.top == 2) || (!R.sigmoid && !R.renorm)) {
      if (R.sigmoid) {
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          c[i] = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v[i] * -log2e));
      } else {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          c[i] = __builtin_amdgcn_exp2f((v[i] - mx) * log2e);   // 0 past E and at -inf
          sum += c[i];
        }
        S = reduce_add(sum);
        if (S == 0.0f) S = 1.0f;
      }
    }
    // a NaN among the logits (or +inf beside -inf), or no finite choice value: float64 does it
    float test = 0.0f;
    if (by_logit) {
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        kv[i] = VPL * lane + i < E ? order_key(v[i]) : 0u;
        test += v[i];
      }
      if (__ballot(test != test) != 0) return false;
    } else {
      float inv = 1.0f;
      if (!R.sigmoid) {
        inv = __builtin_amdgcn_rcpf(S);
        unit = 0x1p-17f * inv;
      }
#pragma unroll
      for (int i = 0; i < VPL; ++i) {
        c[i] = R.sigmoid ? c[i] + b[i] : c[i] * inv + b[i];
        kv[i] = VPL * lane + i < E ? order_key(c[i]) : 0u;
        test += c[i];
      }
      if (__ballot(!(fabsf(test) < INFINITY)) != 0) return false;
    }
    if (limited) {
      const int size = R.size;
      const bool lanes = R.lanes >= 0;                 // (no division here: a third of this block's instructions)
      const int lpg = lanes ? 1 << R.lanes : 0;
      const bool exact = by_logit && R.top == 1;
      uint32_t wk = 0;                                 // exact: the largest key
      float wa = -INFINITY, wb = -INFINITY;            // else the two largest values
      if (lanes) {
        if (exact) {
#pragma unroll
          for (int i = 0; i < VPL; ++i) wk = max(wk, kv[i]);
#define I8H_STEP(M) if (lpg > M) wk = max(wk, (uint32_t)xor_lane_i<M>((int)wk));
          I8H_STEP(1) I8H_STEP(2) I8H_STEP(4) I8H_STEP(8) I8H_STEP(16) I8H_STEP(32)
#undef I8H_STEP
        } else {
          // (lanes past the last group hold whole groups' worth of padding: nobody reads theirs)
#pragma unroll
          for (int i = 0; i < VPL; ++i) {
            wb = fmaxf(wb, fminf(wa, c[i]));
            wa = fmaxf(wa, c[i]);
          }
#define I8H_STEP(M) if (lpg > M) merge2(wa, wb, xor_lane<M>(wa), xor_lane<M>(wb));
          I8H_STEP(1) I8H_STEP(2) I8H_STEP(4) I8H_STEP(8) I8H_STEP(16) I8H_STEP(32)
#undef I8H_STEP
        }
      } else {
        // the values by way of LDS, a lane a group
        float* f = reinterpret_cast<float*>(lds);
        wave_order();
#pragma unroll
        for (int i = 0; i < VPL; ++i)
          if (VPL * lane + i < E) f[VPL * lane + i] = exact ? __uint_as_float(kv[i]) : c[i];
        wave_order();
        if (lane < R.groups) {
#pragma unroll 4
          for (int i = 0; i < size; ++i) {
            const float x = f[lane * size + i];
            wk = max(wk, __float_as_uint(x));
            wb = fmaxf(wb, fminf(wa, x));
            wa = fmaxf(wa, x);
          }
        }
      }
      const int shift = lanes ? R.lanes : 0;           // group g's worth is lane g << shift's
      const int mine = lane >> shift;
      const bool live = mine < R.groups;
      int above = 0;                                   // groups (surely) of more worth
      if (exact) {
        for (int g = 0; g < R.groups; ++g) {
          const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)wk, g << shift);
          above += o > wk || (o == wk && g < mine) ? 1 : 0;
        }
      } else {
        const float w = R.top == 2 ? wa + wb : wa;
        const float up = w + (2.0f * unit + 0x1p-21f * (fabsf(wa) + (R.top == 2 ? fabsf(wb) : 0.0f)));
        for (int g = 0; g < R.groups; ++g)
          above += __int_as_float(__builtin_amdgcn_readlane(__float_as_int(w), g << shift)) > up ? 1 : 0;
        // the `keep` best are below that many at most: no others, or the border is not sure
        if (__popcll(__ballot(live && above < R.keep)) != R.keep << shift) return false;
      }
      if (lanes) {
#pragma unroll
        for (int i = 0; i < VPL; ++i) kv[i] = above < R.keep ? kv[i] : 0u;
      } else {
        const uint64_t all = __ballot(live && above < R.keep);
        const float inv = 1.0f / (float)size;          // (e + 1/2) / size: never within rounding of a whole number
#pragma unroll
        for (int i = 0; i < VPL; ++i) {
          const int g = (int)(((float)(VPL * lane + i) + 0.5f) * inv);
          kv[i] = (all >> (g & 63)) & 1 ? kv[i] : 0u;
        }
      }
    }
  }
  // Candidates: every entry from a threshold `lo` on that leaves k of them or more, but no more than the wave has
  // lanes. The k-th largest of the lanes' own maxima is such a threshold for most rows, and is nearly found by
  // bisection with one comparison a step: from the largest key down in growing steps (2^22 float32 keys are half a
  // factor of two in value), then by halves, until at most k / 2 + 4 maxima too many lie above.
  uint32_t m = kv[0];
#pragma unroll
  for (int i = 1; i < VPL; ++i) m = max(m, kv[i]);
  const uint32_t most = reduce_max(m) + 1u;
  uint32_t hi = most, lo = most, step = 1u << 22;
  int n = 0;
  while (n < k && lo > 1u) {
    hi = lo;
    lo = step != 0u && hi > step ? hi - step : 1u;     // every open key is above 0: all count at 1
    step <<= 2;
    n = __popcll(__ballot(m >= lo));
  }
  while (n > k + k / 2 + 4 && hi - lo > 1u) {
    const uint32_t mid = lo + (hi - lo) / 2u;
    const int at = __popcll(__ballot(m >= mid));
    if (at >= k) {
      lo = mid;
      n = at;
    } else {
      hi = mid;
    }
  }
  n = count_from<VPL>(kv, lo);
  if (n > kWave) {
    // too many: bisection over all entries, count(lo) >= k > count(hi)
    hi = most;
    while (n > kWave && hi - lo > 1u) {
      const uint32_t mid = lo + (hi - lo) / 2u;
      const int at = count_from<VPL>(kv, mid);
      if (at >= k) {
        lo = mid;
        n = at;
      } else {
        hi = mid;
      }
    }
  }
  uint32_t taken = 0;                                  // bit i: entry i of this lane is a candidate
  if (n <= kWave) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) taken |= kv[i] >= lo ? 1u << i : 0u;
  } else if (by_logit) {
    // more than 64 logits equal the k-th: those above, and of the equal ones the lowest indices
    int need = k, before = 0;
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
      taken |= kv[i] > lo ? 1u << i : 0u;
      need -= __popcll(__ballot(kv[i] > lo));
      before += lanes_below_with(__ballot(kv[i] == lo));
    }
#pragma unroll
    for (int i = 0; i < VPL; ++i)
      if (kv[i] == lo) taken |= before++ < need ? 1u << i : 0u;
    n = k;
  } else if constexpr (F64) {
    // more than 64 values within a float64's upper half: the k largest one by one
    for (int j = 0; j < k; ++j) {
      uint64_t top = 0;
#pragma unroll
      for (int i = 0; i < VPL; ++i)
        if (kv[i] != 0u && !((taken >> i) & 1u)) top = max(top, key[i] + 1u);   // (no key is the largest integer)
      const uint64_t all = wave_max_u64(top);
      const int owner = __ffsll((unsigned long long)__ballot(top == all)) - 1;
      if (lane == owner) {
        int at = VPL;
#pragma unroll
        for (int i = VPL - 1; i >= 0; --i)
          if (kv[i] != 0u && !((taken >> i) & 1u) && key[i] + 1u == all) at = i;
        taken |= 1u << at;
      }
    }
    n = k;
  } else {
    return false;
  }
  // one candidate a lane, in the experts' order
  int at = 0;
#pragma unroll
  for (int i = 0; i < VPL; ++i) at += lanes_below_with(__ballot((taken >> i) & 1u));
  wave_order();
#pragma unroll
  for (int i = 0; i < VPL; ++i) {
    if ((taken >> i) & 1u) {
      if constexpr (F64) sc.key[at] = key[i];
      else sc.k32[at] = by_logit ? kv[i] : __float_as_uint(c[i]);
      sc.e[at] = VPL * lane + i;
      sc.v[at] = v[i];
      ++at;
    }
  }
  wave_order();
  const int j = lane < n ? lane : 0;
  const float l = sc.v[j];
  ch.id = sc.e[j];
  int rank = 0;
  if constexpr (F64) {
    const uint64_t mine = sc.key[j];
    for (int r = 0; r < n; ++r) {
      const uint64_t o = sc.key[r];
      rank += o > mine || (o == mine && r < j) ? 1 : 0;
    }
  } else if (by_logit) {
    const uint32_t mine = sc.k32[j];
    for (int r = 0; r < n; ++r) rank += sc.k32[r] > mine ? 1 : 0;
    if (reduce_add(lane < n ? rank : 0) != n * (n - 1) / 2) {   // equal ones among them: the lower index first
      rank = 0;
      for (int r = 0; r < n; ++r) rank += sc.k32[r] + (r < j ? 1u : 0u) > mine ? 1 : 0;
    }
  } else {
    const float mine = __uint_as_float(sc.k32[j]), near = unit + 0x1p-22f * fabsf(mine), up = mine + near;
    for (int r = 0; r < n; ++r) rank += __uint_as_float(sc.k32[r]) > up ? 1 : 0;
    // The rank counts the entries surely above, the true place or less. The chosen places are sure if each of them is
    // taken (their sum is whole and there are k), and the entries left out lie surely below the last.
    const bool in = lane < n && rank < k;
    if (__popcll(__ballot(in)) != k || reduce_add(in ? rank : 0) != k * (k - 1) / 2) return false;
    if (lo > 1u && __ballot(in && mine - near < key_logit(lo)) != 0) return false;
  }
  const bool chosen = lane < n && rank < k;
  if constexpr (F64) {
    double w = 0.0;
    if (chosen) {
      if (R.sigmoid) w = 1.0 / (1.0 + exp(-(double)l));
      else w = (l == -INFINITY ? 0.0 : exp((double)l - (double)mx)) / S64;
    }
    if (R.renorm) {
      const double total = wave_sum64(w);
      w = total == 0.0 ? 0.0 : w / total;
    }
    ch.w = (float)(w * (double)R.scale);
  } else {
    // In float32, an exponential of about 2 units and an argument of |l - max| (softmax) of rounding a score, 10 for a
    // sum: within 40 units of 2^-24, and 2 |l - max|. (In float64 and rounded once: 16384 tokens of 256 experts 31.5 us in
    // place of 29.5.) The score before the softmax's sum, its exponential's argument x. Below e^-746 it is 0 in float64 too.
    const float x = R.sigmoid ? l : l - mx;
    const bool some = chosen && x > -746.0f;
    float w = R.sigmoid ? __builtin_amdgcn_rcpf(1.0f + exp_carried(-l)) : exp_carried(x);
    w = some ? w : 0.0f;
    const float total = R.renorm ? reduce_add(w) : R.sigmoid ? 1.0f : S;
    const float by = R.scale * (total == 0.0f ? 1.0f : __builtin_amdgcn_rcpf(total));
    if (!(fabsf(by) < INFINITY)) return false;
    // A score near float32's smallest normal value, or below, may be short of bits or 0. It is about e^x at most, so its
    // weight is below 2^-127, and 0 here, unless x lies above the border; one that counts is left to float64, and so is a
    // total that such scores may have a part in.
    const bool small = some && w < 0x1p-125f;
    if (__ballot(small) != 0) {
      const float border = -88.1f - 0.6931472f * __builtin_amdgcn_logf(fabsf(by));
      if (total < 0x1p-90f || __ballot(small && x > border) != 0) return false;
      w = small ? 0.0f : w;
    }
    ch.w = w * by;                                     // (the scale first: w / total may have too few bits)
  }
  ch.rank = chosen ? rank : kMaxTopk;
  return true;
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(uint16_t v) { return bf16_to_f32(v); }

// The lane's VPL logits; vec: rows and lanes on whole vectors of them.
template <int VPL, typename X>
__device__ __forceinline__ void load_row(const X* __restrict__ row, int E, int lane, bool vec, float (&v)[VPL]) {
  constexpr int kVec = VPL * sizeof(X) > 16 ? 16 / (int)sizeof(X) : VPL;
  typedef X vec_t __attribute__((ext_vector_type(kVec)));
  if (vec) {
#pragma unroll
    for (int i = 0; i < VPL; i += kVec) {
      vec_t x;
      if (VPL * lane + i < E) x = *reinterpret_cast<const vec_t*>(row + VPL * lane + i);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        if constexpr (kVec == 1) v[i] = VPL * lane + i < E ? to_f32((X)x[0]) : -INFINITY;
        else v[i + j] = VPL * lane + i < E ? to_f32((X)x[j]) : -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = VPL * lane + i < E ? to_f32(row[VPL * lane + i]) : -INFINITY;
  }
}

template <int VPL>
__device__ __forceinline__ void load_bias(const ScoredRule& R, int lane, float (&b)[VPL]) {
#pragma unroll
  for (int i = 0; i < VPL; ++i) b[i] = R.bias != nullptr && VPL * lane + i < R.E ? R.bias[VPL * lane + i] : 0.0f;
}

// The tokens t0 .. t1 of a workgroup of `waves` waves: put(t, choice) for each. Tokens that float32 cannot settle
// are listed and done after the others: the float64 code's registers and the loop's are not held at once.
template <int VPL, typename X, typename Put>
__device__ __forceinline__ void choose_tokens(const X* __restrict__ logits, int64_t t0, int64_t t1, const ScoredRule& R,
                                              bool vec, int lane, int wave, int waves, double* lds, Candidates& sc,
                                              int* again, int* listed, const Put& put) {
  float v[VPL], next[VPL], b[VPL];
  if (t0 + wave < t1) load_row<VPL>(logits + (t0 + wave) * R.E, R.E, lane, vec, next);
  load_bias<VPL>(R, lane, b);
  for (int64_t t = t0 + wave; t < t1; t += waves) {
#pragma unroll
    for (int i = 0; i < VPL; ++i) v[i] = next[i];
    if (t + waves < t1) load_row<VPL>(logits + (t + waves) * R.E, R.E, lane, vec, next);
    Choice ch;
    if (choose<VPL, false>(v, b, R, lane, lds, sc, ch)) put(t, ch);
    else if (lane == 0) listed[atomicAdd(again, 1)] = (int)(t - t0);   // any order: a token's results are its own
  }
  __syncthreads();
  const int n = *again;
  for (int i = wave; i < n; i += waves) {
    const int64_t t = t0 + listed[i];
    load_row<VPL>(logits + t * R.E, R.E, lane, vec, v);
    Choice ch;
    choose<VPL, true>(v, b, R, lane, lds, sc, ch);
    put(t, ch);
  }
}

// A workgroup chooses for a chunk of up to 64 tokens and counts its experts in
// bytes. 16 waves a workgroup and a chunk a CU: four waves a SIMD keep the vector
// unit issuing 92 % of the time at 16384 tokens of 256 experts (5,500 cycles a
// token and wave: scores 640, groups 1,850, threshold 550, candidates 620, ranks
// 1,200, weights 470). The candidates' ranks by way of LDS or of scalar registers
// take the same time.
template <int VPL, typename X>
__global__ void __launch_bounds__(kWave * sc_waves<VPL>())
k_scored_rows(const X* __restrict__ logits, int T, ScoredRule R, int tpc, bool vec, int32_t* __restrict__ ids,
              float* __restrict__ w, uint8_t* __restrict__ hist, int epad) {
  constexpr int kWaves = sc_waves<VPL>();
  __shared__ int cnt[kWave * VPL];             // (epad of them are in use)
  __shared__ double lds[kWaves][kWave * VPL];
  __shared__ Candidates sc[kWaves];
  __shared__ int again, listed[kScChunkTokens];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t t0 = (int64_t)blockIdx.x * tpc, t1 = min((int64_t)T, t0 + tpc);
  for (int e = threadIdx.x; e < epad; e += blockDim.x) cnt[e] = 0;
  if (threadIdx.x == 0) again = 0;
  __syncthreads();
  choose_tokens<VPL>(logits, t0, t1, R, vec, lane, wave, (int)blockDim.x / kWave, lds[wave], sc[wave], &again, listed,
                     [&](int64_t t, const Choice& ch) {
                       if (ch.rank < R.k) {
                         ids[t * R.k + ch.rank] = ch.id;
                         w[t * R.k + ch.rank] = ch.w;
                         atomicAdd(&cnt[ch.id], 1);   // counts only: order does not matter
                       }
                     });
  __syncthreads();
  uint32_t* h = reinterpret_cast<uint32_t*>(hist + (size_t)blockIdx.x * epad);
  for (int e = threadIdx.x; e < epad / 4; e += blockDim.x)
    h[e] = (uint32_t)cnt[4 * e] | (uint32_t)cnt[4 * e + 1] << 8 | (uint32_t)cnt[4 * e + 2] << 16 |
           (uint32_t)cnt[4 * e + 3] << 24;
}

// Running sums of the chunks' counts, one for every `mult` chunks (a scatter
// workgroup's), and the totals: a workgroup takes 16 experts, 64 threads an
// expert, each a run of scatter workgroups.
__global__ void __launch_bounds__(kScScanThreads)
k_scored_scan(const uint8_t* __restrict__ hist, int epad, int nchunks, int mult, int nwg, int E,
              int32_t* __restrict__ pre, int32_t* __restrict__ tot) {
  constexpr int kRuns = kScScanThreads / kScScanExperts;
  __shared__ int run[kRuns][kScScanExperts];
  const int x = threadIdx.x % kScScanExperts, r = threadIdx.x / kScScanExperts;
  const int e = blockIdx.x * kScScanExperts + x;       // < epad
  const int per = (nwg + kRuns - 1) / kRuns;
  const int w0 = min(nwg, r * per), w1 = min(nwg, w0 + per);
  const int c0 = w0 * mult, c1 = min(nchunks, w1 * mult);
  int s = 0;
  for (int c = c0; c < c1; ++c) s += hist[(size_t)c * epad + e];
  run[r][x] = s;
  __syncthreads();
  int before = 0;
  for (int i = 0; i < r; ++i) before += run[i][x];
  for (int w = w0; w < w1; ++w) {
    if (e < E) pre[(size_t)w * E + e] = before;
    for (int c = w * mult, end = min(nchunks, c + mult); c < end; ++c) before += hist[(size_t)c * epad + e];
  }
  if (r == kRuns - 1 && e < E) tot[e] = before;
}

// off[e] = sum of tot[0..e) for e < E, by the whole workgroup of WAVES waves
// (1024 / (64 WAVES) consecutive experts a thread).
template <int WAVES>
__device__ __forceinline__ void exclusive_scan(const int* tot, int* off, int E, int* wave_tot) {
  constexpr int kPer = kMaxExperts / (kWave * WAVES);
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave, e0 = threadIdx.x * kPer;
  int a[kPer], s = 0;
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    a[i] = e0 + i < E ? tot[e0 + i] : 0;
    s += a[i];
  }
  int inc = s;
#pragma unroll
  for (int d = 1; d < kWave; d <<= 1) {
    const int o = __shfl_up(inc, d, kWave);
    if (lane >= d) inc += o;
  }
  if (lane == kWave - 1) wave_tot[wave] = inc;
  __syncthreads();
  int at = inc - s;
#pragma unroll
  for (int i = 0; i < WAVES - 1; ++i) at += i < wave ? wave_tot[i] : 0;      // (all read at once)
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    if (e0 + i < E) off[e0 + i] = at;
    at += a[i];
  }
}

// Rank of the thread's pair among the workgroup's pairs of the same expert
// with a lower thread index. count [waves][ld] in LDS, zero on entry.
template <int WAVES>
__device__ __forceinline__ int stable_rank(bool valid, int e, int E, int ld, int* count) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  uint64_t same = __ballot(valid);
  for (int b = 0, bits = bits_for(E); b < bits; ++b) {
    const bool bit = valid && ((e >> b) & 1);
    const uint64_t with = __ballot(bit);
    same &= bit ? with : ~with;
  }
  int rank = __popcll(same & lanes_below(lane));
  if (valid && rank == 0) count[wave * ld + e] = __popcll(same);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < WAVES - 1; ++i) {
    const int c = count[i * ld + e];           // (all read at once)
    rank += i < wave ? c : 0;
  }
  return rank;
}

// Adds the packed counts of a wave, `cols` (a power of two) lanes a chunk, and puts lane c's sums at part[16 c ..]. A step
// at a time for all of them: a branch a count and step took 2,000 cycles. Over lanes 16 and 32 apart two counts share
// an exchange, each half of the lanes keeping one of them.
__device__ __forceinline__ void put_sums(uint32_t (&v)[16], int cols, int epad, int lane, uint32_t* part) {
#define I8H_STEP(M)                                                                               \
  if (cols <= M) {                                                                                \
    _Pragma("unroll") for (int i = 0; i < 16; ++i) v[i] += (uint32_t)xor_lane_i<M>((int)v[i]);    \
  }
  I8H_STEP(1) I8H_STEP(2) I8H_STEP(4) I8H_STEP(8)
  if (cols <= 16) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const auto s = __builtin_amdgcn_permlane16_swap(v[i], v[i + 8], false, false);
      v[i] = s[0] + s[1];                      // odd rows of 16 lanes: i + 8
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const auto s = __builtin_amdgcn_permlane32_swap(v[i], v[i + 4], false, false);
      v[i] = s[0] + s[1];                      // the upper half: i + 4
    }
    uint32_t* to = part + 16 * (lane % 16) + 4 * (lane / 32) + 8 * (lane / 16 % 2);
    if (lane % 16 < cols && 16 * (lane % 16) < epad) *reinterpret_cast<u32x4*>(to) = u32x4{v[0], v[1], v[2], v[3]};
  } else {
    I8H_STEP(32)
    if (lane < cols && 16 * lane < epad) {
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<u32x4*>(part + 16 * lane + i) = u32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
    }
  }
#undef I8H_STEP
}

// The permutation of `mult` chunks' pairs, a thread each: 5.9 us for 131072 pairs
// of 256 experts, of which most is the chain counts, sums, scan, ranks, store (the
// bytes would take 0.6). SCANNED: pre and
// total hold the chunks' running sums and the totals, else the workgroup adds
// up the counts of all chunks itself: 16 experts a load, `cols` (a power of
// two) lanes a chunk, sums in pairs of 16 bits (at most 256 chunks of 64).
template <bool SCANNED>
__global__ void __launch_bounds__(kScScatterThreads)
k_scored_scatter(const int32_t* __restrict__ ids, int P, int E, int epad, int cols, int nchunks, int mult, int cp,
                 const uint8_t* __restrict__ hist, const int32_t* __restrict__ before,
                 const int32_t* __restrict__ total, int32_t* __restrict__ expert_off,
                 int32_t* __restrict__ sorted_pairs, int32_t* __restrict__ pair_pos) {
  constexpr int kWaves = kScScatterThreads / kWave;
  extern __shared__ __align__(16) int sm[];    // tot, base, pre [epad] each, count [waves][epad]
  int *tot = sm, *base = tot + epad, *pre = base + epad, *count = pre + epad;
  __shared__ int wave_tot[kWaves];
  const int tid = threadIdx.x, lane = tid % kWave, wave = tid / kWave, wg = blockIdx.x;
  const int64_t p = (int64_t)wg * cp + tid;
  const bool valid = tid < cp && p < P;
  const int id = valid ? ids[p] : 0;
  if constexpr (SCANNED) {
    for (int e = tid; e < E; e += kScScatterThreads) {
      tot[e] = total[e];
      pre[e] = before[(size_t)wg * E + e];
    }
  } else {
    // waves' sums in the counts' place: [waves][epad] packed words each, all chunks' and those before
    uint32_t* part = reinterpret_cast<uint32_t*>(count);
    const int col = tid % cols, rows = kScScatterThreads / cols;
    const bool live = 16 * col < epad;
    uint32_t sums[16] = {};                    // [2 i + h]: bytes 4 i + h and 4 i + h + 2 of the 16; 8 on: of chunks before
    for (int c0 = tid / cols; c0 < nchunks; c0 += 4 * rows) {
      u32x4 h[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        h[u] = {0u, 0u, 0u, 0u};
        const int c = c0 + u * rows;
        if (live && c < nchunks) h[u] = *reinterpret_cast<const u32x4*>(hist + (size_t)c * epad + 16 * col);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t mask = c0 + u * rows < wg * mult ? ~0u : 0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t even = h[u][i] & 0x00ff00ffu, odd = (h[u][i] >> 8) & 0x00ff00ffu;
          sums[2 * i] += even;
          sums[2 * i + 1] += odd;
          sums[8 + 2 * i] += even & mask;
          sums[9 + 2 * i] += odd & mask;
        }
      }
    }
    put_sums(sums, cols, epad, lane, part + wave * epad);
    __syncthreads();
    for (int e = tid; e < epad; e += kScScatterThreads) {
      const int b = e % 16, word = 2 * (b / 4) + b % 2, shift = b & 2 ? 16 : 0;
      int t = 0, q = 0;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) {
        t += (part[i * epad + e - b + word] >> shift) & 0xffffu;
        q += (part[i * epad + e - b + 8 + word] >> shift) & 0xffffu;
      }
      tot[e] = t;
      pre[e] = q;
    }
    __syncthreads();
  }
  for (int i = tid; i < kWaves * epad; i += kScScatterThreads) count[i] = 0;
  __syncthreads();
  exclusive_scan<kWaves>(tot, base, E, wave_tot);
  const int rank = stable_rank<kWaves>(valid, id, E, epad, count);   // (its barrier also orders base)
  if (wg == 0) {
    for (int e = tid; e < E; e += kScScatterThreads) expert_off[e] = base[e];
    if (tid == 0) expert_off[E] = P;
  }
  if (valid) {
    const int dst = base[id] + pre[id] + rank;
    sorted_pairs[dst] = (int32_t)p;
    pair_pos[p] = dst;
  }
}

// Few tokens in one workgroup, up to 32 of them, where a wave has two; us here and
// in two launches, 128 experts, top 8: 16 tokens 7.1 and 7.8, 32 tokens 9.2 and 8.0,
// 64 tokens 14.1 and 8.6, 128 tokens 22.8 and 8.7. A call of 32 tokens takes the
// host 14.8 us with one launch and no workspace, 19.6 with two.
template <int VPL, typename X>
__global__ void __launch_bounds__(kScSmallThreads)
k_scored_small(const X* __restrict__ logits, int T, ScoredRule R, bool vec, int32_t* __restrict__ ids,
               float* __restrict__ w, int32_t* __restrict__ expert_off, int32_t* __restrict__ sorted_pairs,
               int32_t* __restrict__ pair_pos) {
  constexpr int kWaves = kScSmallThreads / kWave;
  // the float64 scratch (a wave's E doubles), then the counts of the ranks in its place
  __shared__ double lds[kWaves][kWave * VPL];
  __shared__ Candidates sc[kWaves];
  __shared__ int tot[kWave * VPL], base[kWave * VPL], chosen[kScSmallThreads], wave_tot[kWaves];
  __shared__ int again, listed[kScSmallTokens];
  const int lane = threadIdx.x % kWave;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  for (int e = threadIdx.x; e < R.E; e += kScSmallThreads) tot[e] = 0;
  if (threadIdx.x == 0) again = 0;
  __syncthreads();
  choose_tokens<VPL>(logits, 0, T, R, vec, lane, wave, kWaves, lds[wave], sc[wave], &again, listed,
                     [&](int64_t t, const Choice& ch) {
                       if (ch.rank < R.k) {
                         const int at = (int)t * R.k + ch.rank;
                         ids[at] = chosen[at] = ch.id;
                         w[at] = ch.w;
                         atomicAdd(&tot[ch.id], 1);
                       }
                     });
  __syncthreads();
  int* count = reinterpret_cast<int*>(lds);
  for (int i = threadIdx.x; i < kWaves * R.E; i += kScSmallThreads) count[i] = 0;
  const int P = T * R.k, p = threadIdx.x;
  const bool valid = p < P;
  const int id = valid ? chosen[p] : 0;
  exclusive_scan<kWaves>(tot, base, R.E, wave_tot);   // (its barrier also orders count)
  const int rank = stable_rank<kWaves>(valid, id, R.E, R.E, count);
  for (int e = threadIdx.x; e < R.E; e += kScSmallThreads) expert_off[e] = base[e];
  if (p == 0) expert_off[R.E] = P;
  if (valid) {
    const int dst = base[id] + rank;
    sorted_pairs[dst] = p;
    pair_pos[p] = dst;
  }
}

inline int vpl_of(int E) { return E <= 64 ? 1 : E <= 128 ? 2 : E <= 256 ? 4 : E <= 512 ? 8 : 16; }

// one workgroup: 16 waves have the registers for up to 256 experts
inline bool small_form(int T, int E) { return T <= kScSmallTokens && E <= 256; }

// How the tokens are dealt: chunks of a choosing workgroup, and how many of
// them a scatter workgroup takes (whole ones, at most 512 pairs).
struct Deal {
  int tokens, mult, epad, cols;
  int64_t chunks, wgs;
  Deal(int T, int E, int k) {
    const int most = std::min(kScChunkTokens, kScPairs / k);
    tokens = std::max(1, (int)std::min<int64_t>(most, ((int64_t)T + kScFill - 1) / kScFill));
    mult = kScPairs / (tokens * k);
    chunks = ((int64_t)T + tokens - 1) / tokens;
    wgs = (chunks + mult - 1) / mult;
    epad = (E + 15) / 16 * 16;
    cols = 1;
    while (16 * cols < epad) cols *= 2;
  }
  bool scanned() const { return chunks > kScScanFrom; }
  size_t hist_bytes() const { return ((size_t)chunks * epad + 255) / 256 * 256; }
};

template <int VPL, typename X>
hipError_t launch(const X* l, int T, const ScoredRule& R, int32_t* ids, float* w, int32_t* expert_off,
                  int32_t* sorted_pairs, int32_t* pair_pos, void* ws, hipStream_t st) {
  // whole vectors: VPL logits a lane, at most 16 bytes of them
  constexpr int kBytes = VPL * sizeof(X) > 16 ? 16 : VPL * (int)sizeof(X);
  const bool vec = R.E % VPL == 0 && ((int64_t)R.E * (int64_t)sizeof(X)) % kBytes == 0 &&
                   reinterpret_cast<uintptr_t>(l) % kBytes == 0;
  if constexpr (VPL <= 4) {
    if (small_form(T, R.E)) {
      k_scored_small<VPL, X><<<1, kScSmallThreads, 0, st>>>(l, T, R, vec, ids, w, expert_off, sorted_pairs, pair_pos);
      return hipGetLastError();
    }
  }
  const Deal d(T, R.E, R.k);
  uint8_t* hist = static_cast<uint8_t*>(ws);
  int32_t* tot = reinterpret_cast<int32_t*>(hist + d.hist_bytes());
  int32_t* pre = tot + R.E;
  const int threads = kWave * std::min(sc_waves<VPL>(), d.tokens), nc = (int)d.chunks, nwg = (int)d.wgs;
  k_scored_rows<VPL, X><<<nc, threads, 0, st>>>(l, T, R, d.tokens, vec, ids, w, hist, d.epad);
  const size_t lds = (size_t)(3 + kScScatterThreads / kWave) * d.epad * sizeof(int);
  const int P = T * R.k, cp = d.mult * d.tokens * R.k;
  if (d.scanned()) {
    k_scored_scan<<<d.epad / kScScanExperts, kScScanThreads, 0, st>>>(hist, d.epad, nc, d.mult, nwg, R.E, pre, tot);
    k_scored_scatter<true><<<nwg, kScScatterThreads, lds, st>>>(ids, P, R.E, d.epad, d.cols, nc, d.mult, cp, hist, pre,
                                                                tot, expert_off, sorted_pairs, pair_pos);
  } else {
    k_scored_scatter<false><<<nwg, kScScatterThreads, lds, st>>>(ids, P, R.E, d.epad, d.cols, nc, d.mult, cp, hist,
                                                                 pre, tot, expert_off, sorted_pairs, pair_pos);
  }
  return hipGetLastError();
}

template <typename X>
hipError_t launch(const void* logits, int T, const ScoredRule& R, int32_t* ids, float* w, int32_t* expert_off,
                  int32_t* sorted_pairs, int32_t* pair_pos, void* ws, hipStream_t st) {
  const X* l = static_cast<const X*>(logits);
  switch (vpl_of(R.E)) {
    case 1: return launch<1, X>(l, T, R, ids, w, expert_off, sorted_pairs, pair_pos, ws, st);
    case 2: return launch<2, X>(l, T, R, ids, w, expert_off, sorted_pairs, pair_pos, ws, st);
    case 4: return launch<4, X>(l, T, R, ids, w, expert_off, sorted_pairs, pair_pos, ws, st);
    case 8: return launch<8, X>(l, T, R, ids, w, expert_off, sorted_pairs, pair_pos, ws, st);
    default: return launch<16, X>(l, T, R, ids, w, expert_off, sorted_pairs, pair_pos, ws, st);
  }
}

}  // namespace

bool scored_fits(int T, int E, int k) {
  // offsets into the counts and the chunks' first pairs are 64-bit; a launch holds fewer than 2^32 threads, and a chunk
  // takes up to 1024
  return Deal(T, E, k).chunks * kWave * sc_waves<1>() < ((int64_t)1 << 32);
}

// Never less for more tokens: up to kScFill chunks their number goes up and down with T (256 tokens are 256 chunks, 257
// are 129), so that from kScFill tokens on there is room for kScFill of them.
size_t scored_workspace_bytes(int T, int E, int k) {
  if (small_form(T, E)) return 0;
  Deal d(T, E, k);
  const size_t sums = d.scanned() ? (size_t)(d.wgs + 1) * E * sizeof(int32_t) : 0;
  d.chunks = std::max<int64_t>(d.chunks, std::min(T, kScFill));
  return d.hist_bytes() + sums;
}

hipError_t launch_route_scored(const void* logits, bool bf16, int T, int E, int k, bool sigmoid, const float* bias,
                               int groups, int keep, int top, bool renorm, float scale, int32_t* ids, float* w,
                               int32_t* expert_off, int32_t* sorted_pairs, int32_t* pair_pos, void* ws,
                               hipStream_t st) {
  const int size = E / groups, vpl = vpl_of(E), lpg = size / vpl;
  const bool whole = size == lpg * vpl && (lpg & (lpg - 1)) == 0;
  const ScoredRule R = {bias, E, k, groups, keep, top, size, whole ? __builtin_ctz(lpg) : -1, sigmoid, renorm, scale};
  if (bf16) return launch<uint16_t>(logits, T, R, ids, w, expert_off, sorted_pairs, pair_pos, ws, st);
  return launch<float>(logits, T, R, ids, w, expert_off, sorted_pairs, pair_pos, ws, st);
}

}  // namespace i8h
