// Verification of drafted tokens: a request's drafts x are kept in turn while u q(x) < p(x); the token at the
// first refused row is the smallest t with draw W < w_0 + .. + w_t, w = max(p - q, 0) (behind the last draft: p).
//
// What bounds it: one row of p and one of q per request, read once from HBM; for few requests the two
// launches. Rows are cut into segments of kSegment tokens: the first kernel sums each (fp64: exact products and
// differences, and borders between tokens that do not move with the order of the sums by more than 1e-13), the
// second finds the segment that holds the draw and walks its tokens. Every workgroup finds the request's first
// refused row by itself, from a few gathered values.
#include "attend.hpp"
#include "common.hpp"

namespace seed {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr int kRun = 16;  // tokens of a thread
constexpr int kSegment = kThreads * kRun;

// Weights of a row's tokens: p less q, or p with token x taken out; NaN and negative ones are 0.
template <int DT>
struct Weights {
  const stor_t<DT>* p;
  const stor_t<DT>* q;  // nullptr: nothing to take away
  int x;                // -1: no token taken out
  // of tokens [t0, t0 + N), and of p alone
  template <int N>
  __device__ __forceinline__ void load(int t0, int vocab, double (&w)[N], double (&full)[N]) const {
    float pt[N], qt[N];
    values<N>(p, t0, vocab, pt);
    if (q != nullptr) values<N>(q, t0, vocab, qt);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      full[e] = pt[e] > 0.f ? static_cast<double>(pt[e]) : 0.0;
      if (q != nullptr) {
        const double d = static_cast<double>(pt[e]) - static_cast<double>(qt[e]);
        w[e] = d > 0.0 ? d : 0.0;
      } else {
        w[e] = t0 + e == x ? 0.0 : full[e];
      }
    }
  }

 private:
  template <int N>
  static __device__ __forceinline__ void values(const stor_t<DT>* row, int t0, int vocab, float (&v)[N]) {
    if (t0 <= vocab - N && (reinterpret_cast<uintptr_t>(row + t0) & 15) == 0) {
      load_f32<DT, N>(row + t0, v);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] = t0 < vocab - e ? to_f32<DT>(row[t0 + e]) : 0.f;
    }
  }
};

// Row of the request's first refused draft, or its last row; by every wavefront for itself.
template <int DT>
__device__ __forceinline__ int64_t first_refused(const VerifyArgs& A, int64_t lo, int64_t hi) {
  using T = stor_t<DT>;
  const int lane = threadIdx.x & 63;
  for (int64_t r0 = lo; r0 < hi - 1; r0 += kWave) {
    const int64_t r = r0 + lane;
    bool keep = true;
    if (r < hi - 1) {
      const int x = A.drafts[r];
      keep = false;
      if (x >= 0 && x < A.vocab) {
        const double p = to_f32<DT>(static_cast<const T*>(A.target)[r * A.target_stride + x]);
        const double q = A.draft != nullptr ? to_f32<DT>(static_cast<const T*>(A.draft)[r * A.draft_stride + x]) : 1.f;
        keep = static_cast<double>(A.uniforms[r]) * q < p;
      }
    }
    const uint64_t refused = __ballot(!keep);
    if (refused != 0) return r0 + __builtin_ctzll(refused);
  }
  return hi - 1;
}

template <int DT>
__device__ __forceinline__ Weights<DT> weights_at(const VerifyArgs& A, int64_t row, int64_t hi) {
  using T = stor_t<DT>;
  const bool drafted = row < hi - 1;
  Weights<DT> w;
  w.p = static_cast<const T*>(A.target) + row * A.target_stride;
  w.q = drafted && A.draft != nullptr ? static_cast<const T*>(A.draft) + row * A.draft_stride : nullptr;
  w.x = drafted && A.draft == nullptr ? A.drafts[row] : -1;
  return w;
}

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) v += __shfl_xor(v, d, kWave);
  return v;
}

// Sum of the values of the threads before this one, and of all.
__device__ __forceinline__ double sum_before(double v, double* red, double& total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  double run = v;
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const double up = __shfl_up(run, d, kWave);
    if (lane >= d) run += up;
  }
  const double above = __shfl_up(run, 1, kWave);
  __syncthreads();  // the last call's sums have been read
  if (lane == kWave - 1) red[wave] = run;
  __syncthreads();
  double before = 0.0;
  total = 0.0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w == wave) before = total;
    total += red[w];
  }
  return lane == 0 ? before : before + above;
}

}  // namespace

template <int DT>
__global__ __launch_bounds__(kThreads) void k_verify_sums(const VerifyArgs A) {
  __shared__ double red[2][kWaves];
  const int seg = static_cast<int>(blockIdx.x % A.segments), b = static_cast<int>(blockIdx.x / A.segments);
  int64_t lo, hi;
  sequence_rows(A.offsets, b, A.rows, lo, hi);
  if (lo >= hi) return;
  const int64_t row = first_refused<DT>(A, lo, hi);
  if (seg == 0 && threadIdx.x == 0) A.kept[b] = static_cast<int32_t>(row - lo);
  const Weights<DT> W = weights_at<DT>(A, row, hi);
  constexpr int N = DT == 0 ? 4 : 8;
  double s = 0.0, f = 0.0;
#pragma unroll
  for (int i = 0; i < kRun / N; ++i) {
    double w[N], full[N];
    W.load(seg * kSegment + (i * kThreads + static_cast<int>(threadIdx.x)) * N, A.vocab, w, full);
#pragma unroll
    for (int e = 0; e < N; ++e) {
      s += w[e];
      f += full[e];
    }
  }
  s = wave_sum64(s);
  f = wave_sum64(f);
  if ((threadIdx.x & 63) == 0) {
    red[0][threadIdx.x >> 6] = s;
    red[1][threadIdx.x >> 6] = f;
  }
  __syncthreads();
  if (threadIdx.x < 2) {
    const double* r = red[threadIdx.x];
    A.sums[(static_cast<int64_t>(b) * A.segments + seg) * 2 + threadIdx.x] = (r[0] + r[1]) + (r[2] + r[3]);
  }
}

// A workgroup per request: the segment whose sums pass the draw, then the token in it.
template <int DT>
__global__ __launch_bounds__(kThreads) void k_verify_pick(const VerifyArgs A) {
  constexpr int kNone = 0x7fffffff;
  __shared__ double red[kWaves], start;
  __shared__ int hit, last;  // the first of the segments or tokens that passes the draw, the last one of positive weight
  const int b = blockIdx.x, tid = threadIdx.x;
  int64_t lo, hi;
  sequence_rows(A.offsets, b, A.rows, lo, hi);
  if (lo >= hi) {
    if (tid == 0) A.counts[b] = 0;
    return;
  }
  const int kept = A.kept[b];
  Weights<DT> W = weights_at<DT>(A, lo + kept, hi);
  const double* sums = A.sums + static_cast<int64_t>(b) * A.segments * 2;
  const int per = (A.segments + kThreads - 1) / kThreads;
  const int64_t i0 = static_cast<int64_t>(tid) * per, i1 = min(i0 + per, static_cast<int64_t>(A.segments));
  if (tid == 0) {
    hit = kNone;
    last = -1;
  }
  double total = 0.0, c = 0.0;
  int k = 0;
  for (; k < 2; ++k) {  // where no weight is positive: target itself
    double mine = 0.0;
    for (int64_t i = i0; i < i1; ++i) mine += sums[2 * i + k];
    c = sum_before(mine, red, total);
    if (total > 0.0) break;
  }
  if (k == 1) {
    W.q = nullptr;
    W.x = -1;
  }
  int token = -1;
  if (k < 2) {
    const double target = static_cast<double>(A.draws[b]) * total;
    int mine = kNone, positive = -1;
    double base = 0.0;
    for (int64_t i = i0; i < i1; ++i) {
      const double s = sums[2 * i + k];
      if (s > 0.0) positive = static_cast<int>(i);
      if (mine == kNone && s > 0.0 && c + s > target) {
        mine = static_cast<int>(i);
        base = c;
      }
      c += s;
    }
    if (mine != kNone) atomicMin(&hit, mine);
    if (positive >= 0) atomicMax(&last, positive);
    __syncthreads();
    const bool passed = hit != kNone;
    const int seg = passed ? hit : last;
    if (passed && mine == hit) start = base;
    __syncthreads();
    const double from = passed ? start : 0.0;
    if (tid == 0) {
      hit = kNone;
      last = -1;
    }
    double w[kRun], full[kRun];
    const int t0 = seg * kSegment + tid * kRun;
    W.template load<kRun>(t0, A.vocab, w, full);
    double sum = 0.0, all;
#pragma unroll
    for (int e = 0; e < kRun; ++e) sum += w[e];
    c = from + sum_before(sum, red, all);
    mine = kNone;
    positive = -1;
#pragma unroll
    for (int e = 0; e < kRun; ++e) {
      c += w[e];
      if (w[e] > 0.0) positive = t0 + e;
      if (mine == kNone && w[e] > 0.0 && c > target) mine = t0 + e;
    }
    if (passed && mine != kNone) atomicMin(&hit, mine);
    if (positive >= 0) atomicMax(&last, positive);
    __syncthreads();
    token = hit != kNone ? hit : last;
  }
  const int64_t rows = hi - lo;
  for (int64_t i = tid; i < rows; i += kThreads) A.out[lo + i] = i < kept ? A.drafts[lo + i] : (i == kept ? token : -1);
  if (tid == 0) A.counts[b] = kept + 1;
}

int32_t verify_segments(int32_t vocab) { return static_cast<int32_t>((static_cast<int64_t>(vocab) + kSegment - 1) / kSegment); }

hipError_t launch_verify(int32_t io_dtype, const VerifyArgs& a, hipStream_t s) {
  const dim3 sums(static_cast<unsigned>(static_cast<int64_t>(a.batch) * a.segments)), pick(static_cast<unsigned>(a.batch)), threads(kThreads);
  if (io_dtype == SEED_BF16) k_verify_sums<1><<<sums, threads, 0, s>>>(a);
  else k_verify_sums<0><<<sums, threads, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (io_dtype == SEED_BF16) k_verify_pick<1><<<pick, threads, 0, s>>>(a);
  else k_verify_pick<0><<<pick, threads, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace seed
