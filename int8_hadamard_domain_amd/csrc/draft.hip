// Verification of drafted tokens (speculative sampling's acceptance rule).
//
//   token i stays while u_i q_i(x_i) < p_i(x_i); at the first that does not
//   (row n) the next token is drawn from rest = max(p_n - q_n, 0), after the
//   last drafted one from rest = p_len: the lowest v with
//   rest(0) + .. + rest(v) > u_next sum(rest).
//
// Only one row of p and q is read whole, so the step is a read of 8 V bytes a
// sequence, bound by HBM for many sequences and by latency for one. The row is
// cut into chunks, a workgroup each (k_draft_sums: the chunk's sum in float64,
// fixed order, no atomics on floats), and one workgroup a sequence then finds
// the chunk that the draw falls into and reads only that one again
// (k_draft_pick). Which row it is costs a handful of loads, so every workgroup
// finds it for itself.
//
// Sums are float64: a token is right only if the draw falls on the right side
// of a running sum, and float32 sums over 2^18 entries would be off by more
// than a typical entry's share.

#include "common.hpp"
#include "launch.hpp"

namespace i8h {

namespace {

constexpr int kDrThreads = 256;
constexpr int kDrPer = 16;                          // entries a thread takes of a chunk
constexpr int kDrChunk = kDrThreads * kDrPer;

__device__ __forceinline__ float prob(const float* p, int64_t i) { return p[i]; }
__device__ __forceinline__ float prob(const uint16_t* p, int64_t i) { return bf16_to_f32(p[i]); }

struct DraftArgs {
  const int32_t* drafted;
  const int32_t* draft_len;
  const float* u;
  const float* u_next;
  int D, V;
};

// the sequence's drafted length and the number of tokens that stay (wave-uniform)
template <typename PT>
__device__ __forceinline__ int draft_kept(const DraftArgs& a, const PT* p, const PT* q, int b, int& len) {
  const int lane = threadIdx.x % kWave;
  len = a.draft_len ? min(max(a.draft_len[b], 0), a.D) : a.D;
  for (int i0 = 0; i0 < len; i0 += kWave) {
    const int i = i0 + lane;
    bool stop = false;
    if (i < len) {
      const int x = a.drafted[(int64_t)b * a.D + i];
      stop = true;
      if (x >= 0 && x < a.V) {
        const double pv = prob(p, ((int64_t)b * (a.D + 1) + i) * a.V + x);
        const double qv = q ? (double)prob(q, ((int64_t)b * a.D + i) * a.V + x) : 1.0;
        stop = !((double)a.u[(int64_t)b * a.D + i] * qv < pv);
      }
    }
    const uint64_t m = __ballot(stop);
    if (m != 0) return i0 + __ffsll((unsigned long long)m) - 1;
  }
  return len;
}

__device__ __forceinline__ double positive(double d) { return d > 0.0 && d < __builtin_inf() ? d : 0.0; }

// what row n leaves to draw from: rows of p and q (NULL: nothing subtracted),
// and the entry left out (-1: none)
template <typename PT>
struct DraftRow {
  const PT* p;
  const PT* q;
  int skip;
  __device__ __forceinline__ DraftRow(const DraftArgs& a, const PT* pb, const PT* qb, int b, int n, int len) {
    p = pb + ((int64_t)b * (a.D + 1) + n) * a.V;
    q = nullptr;
    skip = -1;
    if (n < len) {
      if (qb) q = qb + ((int64_t)b * a.D + n) * a.V;
      else skip = a.drafted[(int64_t)b * a.D + n];
    }
  }
  __device__ __forceinline__ void at(int v, double& rest, double& all) const {
    const double pv = prob(p, v);
    all = positive(pv);
    rest = v == skip ? 0.0 : q ? positive(pv - (double)prob(q, v)) : all;
  }
};

__device__ __forceinline__ double shfl_xor_f64(double v, int m) { return __shfl_xor(v, m, kWave); }

template <typename PT>
__global__ void __launch_bounds__(kDrThreads)
k_draft_sums(const DraftArgs a, const PT* __restrict__ p, const PT* __restrict__ q, double* __restrict__ sums) {
  __shared__ double part[2][kDrThreads / kWave];
  const int b = blockIdx.y, c = blockIdx.x;
  int len;
  const int n = draft_kept(a, p, q, b, len);
  const DraftRow<PT> row(a, p, q, b, n, len);
  double rest = 0.0, all = 0.0;
#pragma unroll
  for (int i = 0; i < kDrPer; ++i) {
    const int64_t v = (int64_t)c * kDrChunk + i * kDrThreads + threadIdx.x;
    if (v < a.V) {
      double r, w;
      row.at((int)v, r, w);
      rest += r;
      all += w;
    }
  }
  for (int m = 32; m >= 1; m >>= 1) {
    rest += shfl_xor_f64(rest, m);
    all += shfl_xor_f64(all, m);
  }
  if (threadIdx.x % kWave == 0) {
    part[0][threadIdx.x / kWave] = rest;
    part[1][threadIdx.x / kWave] = all;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double* o = sums + 2 * ((int64_t)b * gridDim.x + c);
    o[0] = (part[0][0] + part[0][1]) + (part[0][2] + part[0][3]);
    o[1] = (part[1][0] + part[1][1]) + (part[1][2] + part[1][3]);
  }
}

// sum of v over the threads below this one; total over the workgroup
__device__ __forceinline__ double block_scan(double v, double* wave_sum, double& total) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  double inc = v;
  for (int d = 1; d < kWave; d <<= 1) {
    const double o = __shfl_up(inc, d, kWave);
    if (lane >= d) inc += o;
  }
  __syncthreads();
  if (lane == kWave - 1) wave_sum[wave] = inc;
  __syncthreads();
  double base = 0.0;
  total = 0.0;
  for (int w = 0; w < kDrThreads / kWave; ++w) {
    if (w < wave) base += wave_sum[w];
    total += wave_sum[w];
  }
  double ex = __shfl_up(inc, 1, kWave);
  if (lane == 0) ex = 0.0;
  return base + ex;
}

template <typename PT>
__global__ void __launch_bounds__(kDrThreads)
k_draft_pick(const DraftArgs a, const PT* __restrict__ p, const PT* __restrict__ q, const double* __restrict__ sums,
             int nchunks, int32_t* __restrict__ tokens, int32_t* __restrict__ accepted) {
  __shared__ double wave_sum[kDrThreads / kWave];
  __shared__ double s_base;
  __shared__ int s_first, s_last;
  const int b = blockIdx.x, tid = threadIdx.x;
  int len;
  const int n = draft_kept(a, p, q, b, len);
  const DraftRow<PT> row(a, p, q, b, n, len);
  const double* sb = sums + 2 * (int64_t)b * nchunks;

  // the sums' total, and whether anything is left of rest
  double rest = 0.0, all = 0.0;
  for (int c = tid; c < nchunks; c += kDrThreads) {
    rest += sb[2 * c];
    all += sb[2 * c + 1];
  }
  double rt, at;
  block_scan(rest, wave_sum, rt);
  block_scan(all, wave_sum, at);
  const int kind = rt > 0.0 ? 0 : 1;
  const double total = kind == 0 ? rt : at;
  const double target = (double)a.u_next[b] * total;

  // the first chunk whose running sum passes the target (the last one that
  // holds anything, if rounding leaves none), and the sum before it
  if (tid == 0) {
    s_first = nchunks;
    s_last = -1;
  }
  double before = 0.0;
  int chunk = -1;
  for (int c0 = 0; c0 < nchunks; c0 += kDrThreads) {
    const int c = c0 + tid;
    const double v = c < nchunks ? sb[2 * c + kind] : 0.0;
    double tile;
    const double ex = before + block_scan(v, wave_sum, tile);
    if (c < nchunks && ex + v > target) atomicMin(&s_first, c);
    if (v > 0.0) atomicMax(&s_last, c);
    __syncthreads();
    const int hit = s_first < nchunks ? s_first : c0 + kDrThreads >= nchunks ? s_last : -1;
    // the sum before the chosen chunk, if it is in this tile of chunks
    if (c < nchunks && c == hit) s_base = ex;
    __syncthreads();
    if (s_first < nchunks) {
      chunk = s_first;
      break;
    }
    before += tile;
  }
  int next = a.V - 1;
  if (chunk < 0) {
    // no running sum passes (the target rounds up to the total): the last entry
    // that holds anything; with an empty row the last of all
    chunk = s_last;
    if (chunk >= 0) {
      __syncthreads();
      if (tid == 0) s_base = __builtin_inf();
    }
  }
  __syncthreads();
  if (chunk >= 0) {
    const double base = s_base;
    double v[kDrPer], sum = 0.0;
    int last = -1;
    const int64_t v0 = (int64_t)chunk * kDrChunk + tid * kDrPer;
#pragma unroll
    for (int i = 0; i < kDrPer; ++i) {
      v[i] = 0.0;
      if (v0 + i < a.V) {
        double r, w;
        row.at((int)(v0 + i), r, w);
        v[i] = kind == 0 ? r : w;
        if (v[i] > 0.0) last = (int)(v0 + i);
      }
      sum += v[i];
    }
    double unused;
    double run = block_scan(sum, wave_sum, unused);
    if (tid == 0) {
      s_first = a.V;
      s_last = -1;
    }
    __syncthreads();
    // base is infinite where the last entry is wanted: then nothing counts as passed
    if (base < __builtin_inf()) {
      run += base;
      int first = a.V;
#pragma unroll
      for (int i = 0; i < kDrPer; ++i) {
        run += v[i];
        if (first == a.V && v[i] > 0.0 && run > target) first = (int)(v0 + i);
      }
      if (first < a.V) atomicMin(&s_first, first);
    }
    if (last >= 0) atomicMax(&s_last, last);
    __syncthreads();
    next = s_first < a.V ? s_first : s_last >= 0 ? s_last : a.V - 1;
  }
  for (int i = tid; i <= a.D; i += kDrThreads)
    tokens[(int64_t)b * (a.D + 1) + i] = i < n ? a.drafted[(int64_t)b * a.D + i] : i == n ? next : -1;
  if (tid == 0) accepted[b] = n;
}

template <typename PT>
hipError_t draft(const DraftArgs& a, const void* pv, const void* qv, int B, double* sums, int32_t* tokens,
                 int32_t* accepted, hipStream_t st) {
  const PT* p = static_cast<const PT*>(pv);
  const PT* q = a.D > 0 ? static_cast<const PT*>(qv) : nullptr;
  const int nchunks = draft_chunks(a.V);
  k_draft_sums<PT><<<dim3(nchunks, B), kDrThreads, 0, st>>>(a, p, q, sums);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_draft_pick<PT><<<B, kDrThreads, 0, st>>>(a, p, q, sums, nchunks, tokens, accepted);
  return hipGetLastError();
}

}  // namespace

int draft_chunks(int V) { return (int)(((int64_t)V + kDrChunk - 1) / kDrChunk); }

hipError_t launch_draft_verify(const void* p, const void* q, bool bf16, const int32_t* drafted,
                               const int32_t* draft_len, const float* u, const float* u_next, int B, int D, int V,
                               double* sums, int32_t* tokens, int32_t* accepted, hipStream_t st) {
  const DraftArgs a = {drafted, draft_len, u, u_next, D, V};
  return bf16 ? draft<uint16_t>(a, p, q, B, sums, tokens, accepted, st)
              : draft<float>(a, p, q, B, sums, tokens, accepted, st);
}

}  // namespace i8h
