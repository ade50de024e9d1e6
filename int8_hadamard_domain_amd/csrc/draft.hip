// Verification of drafted tokens (speculative sampling's acceptance rule).
//
//   token i stays while u_i q_i(x_i) < p_i(x_i); at the first that does not
//   (row n) the next token is drawn from rest = max(p_n - q_n, 0), after the
//   last drafted one from rest = p_len: the lowest v with
//   rest(0) + .. + rest(v) > u_next sum(rest).
//
// Only one row of p and q is read whole, so the step is a read of 8 V bytes a
// sequence, bound by HBM for many sequences (64 of 2^17 entries: 67 MB in 23 us,
// 19 of them k_draft_sums, whose read waits for the search for the row) and by
// latency for one (2^18 entries: 7.6 us, two launches). The row is
// cut into chunks, a workgroup each (k_draft_sums: the chunk's sum in float64,
// fixed order, no atomics on floats), and one workgroup a sequence then finds
// the chunk that the draw falls into and reads only that one again
// (k_draft_pick). Which row it is costs two dependent loads, so every workgroup
// of the first kernel finds it for itself; the second is told.
//
// Sums are float64: a token is right only if the draw falls on the right side
// of a running sum, and float32 sums over 2^18 entries would be off by more
// than a typical entry's share.

#include "common.hpp"
#include "launch.hpp"

namespace i8h {

namespace {

constexpr int kDrThreads = 256;
constexpr int kDrWaves = kDrThreads / kWave;

__device__ __forceinline__ float prob(const float* p) { return *p; }
__device__ __forceinline__ float prob(const uint16_t* p) { return bf16_to_f32(*p); }

// entries v .. v + 3 of a row of V (zero past its end); vec: rows are aligned for one load
__device__ __forceinline__ void prob4(const float* p, int64_t v, int V, bool vec, float (&o)[4]) {
  if (vec && v + 4 <= V) {
    const f32x4 a = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p + v));
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = a[j];
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = v + j < V ? p[v + j] : 0.0f;
  }
}
__device__ __forceinline__ void prob4(const uint16_t* p, int64_t v, int V, bool vec, float (&o)[4]) {
  if (vec && v + 4 <= V) {
    const u32x2 a = __builtin_nontemporal_load(reinterpret_cast<const u32x2*>(p + v));
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      o[2 * j] = bf16_lo(a[j]);
      o[2 * j + 1] = bf16_hi(a[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = v + j < V ? bf16_to_f32(p[v + j]) : 0.0f;
  }
}

struct DraftArgs {
  const int32_t* drafted;
  const int32_t* draft_len;
  const float* u;
  const float* u_next;
  int D, V;
  bool vec;
};

__device__ __forceinline__ int draft_length(const DraftArgs& a, int b) {
  return a.draft_len ? min(max(a.draft_len[b], 0), a.D) : a.D;
}

// the number of tokens that stay (wave-uniform). A position's loads do not wait
// for the sequence's length, which only ends the count.
template <typename PT>
__device__ __forceinline__ int draft_kept(const DraftArgs& a, const PT* p, const PT* q, int b, int len) {
  const int lane = threadIdx.x % kWave;
  for (int i0 = 0; i0 < a.D; i0 += kWave) {
    const int i = i0 + lane;
    bool stop = true;
    if (i < a.D) {
      const int x = a.drafted[(int64_t)b * a.D + i];
      if (x >= 0 && x < a.V) {
        const double pv = prob(p + ((int64_t)b * (a.D + 1) + i) * a.V + x);
        const double qv = q ? (double)prob(q + ((int64_t)b * a.D + i) * a.V + x) : 1.0;
        stop = !((double)a.u[(int64_t)b * a.D + i] * qv < pv);
      }
    }
    const uint64_t m = __ballot(stop || i >= len);
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
};

// entries v0 + 4 i stride .. +3 of the row's p and q, i < N
template <int N, typename PT>
__device__ __forceinline__ void draft_load(const DraftArgs& a, const DraftRow<PT>& row, int64_t v0, int stride,
                                           float (&pv)[N][4], float (&qv)[N][4]) {
#pragma unroll
  for (int i = 0; i < N; ++i) prob4(row.p, v0 + (int64_t)4 * i * stride, a.V, a.vec, pv[i]);
  if (row.q) {
#pragma unroll
    for (int i = 0; i < N; ++i) prob4(row.q, v0 + (int64_t)4 * i * stride, a.V, a.vec, qv[i]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) qv[i][j] = 0.0f;
  }
}
template <typename PT>
__device__ __forceinline__ double draft_rest(const DraftRow<PT>& row, int64_t v, float p, float q) {
  return v == row.skip ? 0.0 : positive((double)p - (double)q);
}

// Sum over the lanes up to this one, in lane order within rows of 16 and then
// over rows: data-parallel-primitive moves on the vector ALU (a scan through LDS
// shuffles costs their latency twelve times).
template <int CTRL, int ROWS>
__device__ __forceinline__ double dpp_f64(double v) {
  const u32x2 w = __builtin_bit_cast(u32x2, v);
  u32x2 o;
  o[0] = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w[0], CTRL, ROWS, 0xF, true);
  o[1] = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)w[1], CTRL, ROWS, 0xF, true);
  return __builtin_bit_cast(double, o);   // 0.0 where no lane gives one
}
__device__ __forceinline__ double wave_scan(double v) {
  v += dpp_f64<0x111, 0xF>(v);   // row_shr 1, 2, 4, 8
  v += dpp_f64<0x112, 0xF>(v);
  v += dpp_f64<0x114, 0xF>(v);
  v += dpp_f64<0x118, 0xF>(v);
  v += dpp_f64<0x142, 0xA>(v);   // row_bcast 15: lane 15 of rows 0, 2 to rows 1, 3
  v += dpp_f64<0x143, 0xC>(v);   // row_bcast 31: lane 31 to rows 2, 3
  return v;
}

// N: groups of four entries a thread takes of a chunk of kDrThreads * 4 N
template <int N, typename PT>
__global__ void __launch_bounds__(kDrThreads)
k_draft_sums(const DraftArgs a, const PT* __restrict__ p, const PT* __restrict__ q, double* __restrict__ sums,
             int32_t* __restrict__ kept) {
  __shared__ double part[2][kDrWaves];
  const int b = blockIdx.y, c = blockIdx.x;
  const int len = draft_length(a, b);
  const int n = draft_kept(a, p, q, b, len);
  const DraftRow<PT> row(a, p, q, b, n, len);
  const int64_t v0 = (int64_t)c * (kDrThreads * 4 * N) + 4 * threadIdx.x;
  float pv[N][4], qv[N][4];
  draft_load<N>(a, row, v0, kDrThreads, pv, qv);
  double rest = 0.0, all = 0.0;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      all += positive(pv[i][j]);
      rest += draft_rest(row, v0 + (int64_t)4 * i * kDrThreads + j, pv[i][j], qv[i][j]);
    }
  rest = wave_scan(rest);
  all = wave_scan(all);
  if (threadIdx.x % kWave == kWave - 1) {
    part[0][threadIdx.x / kWave] = rest;
    part[1][threadIdx.x / kWave] = all;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    double* o = sums + 2 * ((int64_t)b * gridDim.x + c);
    o[0] = (part[0][0] + part[0][1]) + (part[0][2] + part[0][3]);
    o[1] = (part[1][0] + part[1][1]) + (part[1][2] + part[1][3]);
    if (c == 0) kept[b] = n;
  }
}

// sum of v over the threads below this one; total over the workgroup
__device__ __forceinline__ double block_scan(double v, double* wave_sum, double& total) {
  const int lane = threadIdx.x % kWave, wave = threadIdx.x / kWave;
  const double inc = wave_scan(v);
  __syncthreads();
  if (lane == kWave - 1) wave_sum[wave] = inc;
  __syncthreads();
  double base = 0.0;
  total = 0.0;
#pragma unroll
  for (int w = 0; w < kDrWaves; ++w) {
    const double s = wave_sum[w];
    if (w < wave) base += s;
    total += s;
  }
  return base + dpp_f64<0x138, 0xF>(inc);   // wave_shr 1
}

// the lowest thread index at which `hit` holds, and the highest at which `any`
// does (-1: none), over the workgroup
__device__ __forceinline__ void block_find(bool hit, bool any, int (*found)[2], int& first, int& last) {
  const int wave = threadIdx.x / kWave;
  const uint64_t h = __ballot(hit), a = __ballot(any);
  __syncthreads();
  if (threadIdx.x % kWave == 0) {
    found[wave][0] = h ? wave * kWave + __ffsll((unsigned long long)h) - 1 : -1;
    found[wave][1] = a ? wave * kWave + 63 - __clzll((long long)a) : -1;
  }
  __syncthreads();
  first = last = -1;
#pragma unroll
  for (int w = 0; w < kDrWaves; ++w) {
    if (first < 0) first = found[w][0];
    if (found[w][1] >= 0) last = found[w][1];
  }
}

template <int N, typename PT>
__global__ void __launch_bounds__(kDrThreads)
k_draft_pick(const DraftArgs a, const PT* __restrict__ p, const PT* __restrict__ q, const double* __restrict__ sums,
             int nchunks, const int32_t* __restrict__ kept, int32_t* __restrict__ tokens,
             int32_t* __restrict__ accepted) {
  constexpr int kPer = 4 * N;
  __shared__ double wave_sum[kDrWaves];
  __shared__ double s_base;
  __shared__ int s_next;
  __shared__ int found[kDrWaves][2];
  const int b = blockIdx.x, tid = threadIdx.x;
  const double* sb = sums + 2 * (int64_t)b * nchunks;
  const int n = kept[b], len = draft_length(a, b);
  const DraftRow<PT> row(a, p, q, b, n, len);
  const double un = a.u_next[b];

  // the first chunk whose running sum passes the target (the last one that
  // holds anything, if rounding leaves none), and the sum before it. Nearly
  // always the row's chunks fit one tile of 256.
  double total, chunk_sum = tid < nchunks ? sb[2 * tid] : 0.0, ex = block_scan(chunk_sum, wave_sum, total);
  int kind = 0;
  if (nchunks > kDrThreads) {
    double more = 0.0, rest;
    for (int c = kDrThreads + tid; c < nchunks; c += kDrThreads) more += sb[2 * c];
    block_scan(more, wave_sum, rest);
    total += rest;
  }
  if (!(total > 0.0)) {   // nothing is left of rest: p itself
    kind = 1;
    double all = 0.0;
    for (int c = tid; c < nchunks; c += kDrThreads) all += sb[2 * c + 1];
    block_scan(all, wave_sum, total);
    chunk_sum = tid < nchunks ? sb[2 * tid + 1] : 0.0;
    double unused;
    ex = block_scan(chunk_sum, wave_sum, unused);
  }
  const double target = un * total;
  int chunk = -1, last_chunk = -1;
  for (int c0 = 0;;) {
    int first, last;
    // only a chunk that holds something: ex is rounded in another order than the
    // sums before it, so an empty chunk's may pass where theirs did not
    const bool some = chunk_sum > 0.0;
    block_find(some && ex + chunk_sum > target, some, found, first, last);
    if (last >= 0) last_chunk = c0 + last;
    if (first >= 0) {
      chunk = c0 + first;
      if (tid == first) s_base = ex;
      break;
    }
    c0 += kDrThreads;
    if (c0 >= nchunks) break;
    if (tid == kDrThreads - 1) s_base = ex + chunk_sum;   // the running sum so far
    __syncthreads();
    const double before = s_base;
    const int c = c0 + tid;
    double tile;
    chunk_sum = c < nchunks ? sb[2 * c + kind] : 0.0;
    ex = before + block_scan(chunk_sum, wave_sum, tile);
  }
  // no running sum passes (the target rounds up to the total): the last entry
  // that holds anything; with an empty row the last of all
  const bool last_one = chunk < 0;
  if (last_one) chunk = last_chunk;
  if (tid == 0) s_next = a.V - 1;
  __syncthreads();
  if (chunk >= 0) {
    float pv[N][4], qv[N][4];
    const int64_t v0 = (int64_t)chunk * (kDrThreads * kPer) + tid * kPer;
    draft_load<N>(a, row, v0, 1, pv, qv);
    double rest[kPer], sum = 0.0;
    int mine = -1;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const float pi = pv[i / 4][i % 4], qi = qv[i / 4][i % 4];
      rest[i] = kind == 1 ? positive(pi) : draft_rest(row, v0 + i, pi, qi);
      if (rest[i] > 0.0) mine = i;
      sum += rest[i];
    }
    double unused, run = s_base + block_scan(sum, wave_sum, unused);
    const bool any = mine >= 0;
    int hit = -1;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      run += rest[i];
      if (hit < 0 && rest[i] > 0.0 && run > target && !last_one) hit = i;
    }
    int first, last;
    block_find(hit >= 0, any, found, first, last);
    if (first >= 0 ? tid == first : tid == last) s_next = (int)(v0 + (first >= 0 ? hit : mine));
    __syncthreads();
  }
  const int next = s_next;
  for (int i = tid; i <= a.D; i += kDrThreads)
    tokens[(int64_t)b * (a.D + 1) + i] = i < n ? a.drafted[(int64_t)b * a.D + i] : i == n ? next : -1;
  if (tid == 0) accepted[b] = n;
}

// Groups of four entries a thread takes: chunks of 1024 entries, so that one
// sequence of 2^18 entries fills the chip, while they make up to four times the
// workgroups that run at once; chunks of 4096 beyond, where each workgroup's
// search for its row costs more than the parallelism gives. Both, of 1024 and of
// 4096 entries: 1 sequence of 2^18 7.4 and 11.9 us, 32 of 2^17 15.4 and 17.2, 64
// (8192 workgroups) 23.4 and 23.3, 128 34.4 and 27.5, 256 58 and 40.
int draft_groups(int B, int V) { return B * (((int64_t)V + 1023) / 1024) <= 8192 ? 1 : 4; }

template <typename PT>
hipError_t draft(const DraftArgs& a, const void* pv, const void* qv, int B, void* ws, int32_t* tokens,
                 int32_t* accepted, hipStream_t st) {
  const PT* p = static_cast<const PT*>(pv);
  const PT* q = a.D > 0 ? static_cast<const PT*>(qv) : nullptr;
  const int nchunks = draft_chunks(B, a.V);
  double* sums = static_cast<double*>(ws);
  int32_t* kept = reinterpret_cast<int32_t*>(sums + (int64_t)2 * B * nchunks);
  const dim3 grid(nchunks, B);
  const bool small = draft_groups(B, a.V) == 1;
  if (small) k_draft_sums<1, PT><<<grid, kDrThreads, 0, st>>>(a, p, q, sums, kept);
  else k_draft_sums<4, PT><<<grid, kDrThreads, 0, st>>>(a, p, q, sums, kept);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (small) k_draft_pick<1, PT><<<B, kDrThreads, 0, st>>>(a, p, q, sums, nchunks, kept, tokens, accepted);
  else k_draft_pick<4, PT><<<B, kDrThreads, 0, st>>>(a, p, q, sums, nchunks, kept, tokens, accepted);
  return hipGetLastError();
}

}  // namespace

int draft_chunks(int B, int V) {
  const int64_t chunk = (int64_t)kDrThreads * 4 * draft_groups(B, V);
  return (int)((V + chunk - 1) / chunk);
}

// the chunks' sums, two doubles each, then the sequences' counts
size_t draft_workspace_bytes(int B, int V) {
  return (size_t)B * draft_chunks(B, V) * 2 * sizeof(double) + (size_t)B * sizeof(int32_t);
}

hipError_t launch_draft_verify(const void* p, const void* q, bool bf16, const int32_t* drafted,
                               const int32_t* draft_len, const float* u, const float* u_next, int B, int D, int V,
                               void* ws, int32_t* tokens, int32_t* accepted, hipStream_t st) {
  // one load of four entries where every row starts at its alignment
  const uintptr_t align = bf16 ? 8 : 16;
  const bool vec = V % 4 == 0 && (reinterpret_cast<uintptr_t>(p) | reinterpret_cast<uintptr_t>(q)) % align == 0;
  const DraftArgs a = {drafted, draft_len, u, u_next, D, V, vec};
  return bf16 ? draft<uint16_t>(a, p, q, B, ws, tokens, accepted, st)
              : draft<float>(a, p, q, B, ws, tokens, accepted, st);
}

}  // namespace i8h
