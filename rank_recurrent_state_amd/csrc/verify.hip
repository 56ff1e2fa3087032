// Verification of drafted tokens: a request's drafts x are kept in turn while u q(x) < p(x); the token at the
// first refused row is the smallest t with draw W < w_0 + .. + w_t, w = max(p - q, 0) (behind the last draft: p).
//
// What bounds it: one row of p, and one of q where a draft is refused, read once from HBM; for few requests the latency of
// what follows from what: the row's number, a few drafts' probabilities, the row, the sums, the segment that holds
// the draw. Rows are cut into segments of 1024 tokens, a wavefront each: it sums them (fp64: exact products and
// differences, and borders between tokens that do not move with the order of the sums by more than 1e-13), then the
// segment that holds the draw is read again and its tokens are walked. Every wavefront finds the request's first
// refused row by itself, from a few gathered values, and no step needs more than one wavefront: a row that one
// workgroup reads as fast as a second launch takes is summed and walked by it, larger ones in two launches.
// Measured: 128 requests, 150001 tokens, fp32, of which 50 refuse a draft and read its row too, 107 MB: 24 us, 4.5 TB/s.
// The sums take 19 to 21 (5.5 TB/s; wavefronts wait 63 % of their time, the vector unit is busy 27 % of it), the choice 5.
// 200 requests, 65536 tokens, bf16, no drafts' probabilities, 26 MB: 13 us, the sums 9.5 (wavefronts wait 69 %, vector unit
// 45 %: neither it nor HBM is the bound, but what waits one after another), the choice 4 to 5, both launches' starts and
// ends among them. The loads that lead to the refused row are 1 us of it (no drafts: 10.4 us from 11.5, captured). 14 us
// with the choice of positive weights and of x in fp64 for all. Two segments a wavefront at once: the same or up to 1 us more.
#include "attend.hpp"
#include "common.hpp"

namespace seed {

namespace {

constexpr int kRun = 16;                  // tokens of a lane
constexpr int kSegment = kWave * kRun;    // and of a segment
constexpr int kWaves = 4;                 // of a workgroup that sums
constexpr int kMany = kAloneThreads / kWave;  // of one that does a request alone
// Segments of such a request. One request of 16384 fp32 tokens: 7.1 us, in two launches 8.2; of 32768: 8.4 and 8.6; of
// 65536: 11 and 8. 64 of 16384: 8 and 10; of 32768: 12 and 10; 200 of 32768: 13 and 14.
constexpr int kMost = 32;

// 16 bytes at any address that holds a value: rows of an odd length start anywhere.
template <int DT> struct Any16;
template <> struct Any16<0> { using T = __attribute__((ext_vector_type(4), aligned(4))) uint32_t; };
template <> struct Any16<1> { using T = __attribute__((ext_vector_type(4), aligned(2))) uint32_t; };

// Weights of a row's tokens: p less q, or p with token x taken out; NaN and negative ones are 0.
template <int DT>
struct Weights {
  static constexpr int N = DT == 0 ? 4 : 8;  // values of 16 bytes
  const stor_t<DT>* p;
  const stor_t<DT>* q;  // nullptr: nothing to take away
  int x;                // -1: no token taken out

  // K times N tokens, the k-th from t0 + k step on; inside: the whole wavefront's tokens are below vocab
  template <int K>
  __device__ __forceinline__ void load(int t0, int step, int vocab, bool inside, double (&w)[K * N]) const {
    float pt[K][N], qt[K][N];
    if (inside) {
#pragma unroll
      for (int k = 0; k < K; ++k) wide(p + t0 + k * step, pt[k]);
      if (q != nullptr) {
#pragma unroll
        for (int k = 0; k < K; ++k) wide(q + t0 + k * step, qt[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < N; ++e) pt[k][e] = qt[k][e] = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (t0 + k * step <= vocab - N) {
          wide(p + t0 + k * step, pt[k]);
          if (q != nullptr) wide(q + t0 + k * step, qt[k]);
        }
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (t0 + k * step > vocab - N && t0 + k * step < vocab) {  // the row's last tokens: one lane's
#pragma unroll
          for (int e = 0; e < N - 1; ++e)
            if (t0 + k * step + e < vocab) {
              pt[k][e] = to_f32<DT>(p[t0 + k * step + e]);
              if (q != nullptr) qt[k][e] = to_f32<DT>(q[t0 + k * step + e]);
            }
        }
    }
    if (q != nullptr) {
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < N; ++e) w[k * N + e] = fmax(static_cast<double>(pt[k][e]) - static_cast<double>(qt[k][e]), 0.0);  // of NaN: 0
    } else {
      bool here = false;  // token x among these
#pragma unroll
      for (int k = 0; k < K; ++k) here = here || static_cast<uint32_t>(x - (t0 + k * step)) < N;
      if (__any(here)) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
          for (int e = 0; e < N; ++e) pt[k][e] = t0 + k * step + e == x ? 0.f : pt[k][e];
      }
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int e = 0; e < N; ++e) w[k * N + e] = __builtin_amdgcn_fmed3f(pt[k][e], 0.f, __builtin_inff());  // of NaN: 0
    }
  }

 private:
  static __device__ __forceinline__ void wide(const stor_t<DT>* p, float (&v)[N]) {
    const auto x = __builtin_nontemporal_load(reinterpret_cast<const typename Any16<DT>::T*>(p));
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (DT == 0) {
        v[e] = __uint_as_float(x[e]);
      } else {
        v[2 * e] = lo16<DT>(x[e]);
        v[2 * e + 1] = hi16<DT>(x[e]);
      }
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

template <int CTRL>
__device__ __forceinline__ double dpp64(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_mov_dpp(static_cast<int>(u), CTRL, 0xF, 0xF, true);
  const uint32_t hi = __builtin_amdgcn_mov_dpp(static_cast<int>(u >> 32), CTRL, 0xF, 0xF, true);
  return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
// Sum over all lanes, the same in each.
__device__ __forceinline__ double wave_sum64(double v) {
  v += dpp64<0xB1>(v);
  v += dpp64<0x4E>(v);
  v += dpp64<0x141>(v);
  v += dpp64<0x140>(v);
  v += __shfl_xor(v, 16, kWave);
  v += __shfl_xor(v, 32, kWave);
  return v;
}
// Sum of the lanes before this one, and of all.
__device__ __forceinline__ double sum_before(double v, double& total) {
  const int lane = threadIdx.x & 63;
  double run = v;
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const double up = __shfl_up(run, d, kWave);
    if (lane >= d) run += up;
  }
  total = __shfl(run, kWave - 1, kWave);
  const double above = __shfl_up(run, 1, kWave);
  return lane == 0 ? 0.0 : above;
}

// Sum of a segment's weights.
template <int DT>
__device__ __forceinline__ double sum_segment(const Weights<DT>& W, int seg, int vocab) {
  constexpr int N = Weights<DT>::N;
  double w[kRun], s = 0.0;
  W.template load<kRun / N>(seg * kSegment + (static_cast<int>(threadIdx.x) & 63) * N, kWave * N, vocab, (seg + 1) * kSegment <= vocab, w);
#pragma unroll
  for (int e = 0; e < kRun; ++e) s += w[e];
  return wave_sum64(s);
}

// The token of segment seg that passes target, base the sum of the segments before; where none does (passes: whether
// one is meant to), the last of positive weight. One wavefront.
template <int DT>
__device__ __forceinline__ int walk(const Weights<DT>& W, int seg, int vocab, double base, double target, bool passes) {
  constexpr int N = Weights<DT>::N;
  const int t0 = seg * kSegment + (static_cast<int>(threadIdx.x) & 63) * kRun;
  double w[kRun], sum = 0.0, all;
  W.template load<kRun / N>(t0, N, vocab, (seg + 1) * kSegment <= vocab, w);
#pragma unroll
  for (int e = 0; e < kRun; ++e) sum += w[e];
  double c = base + sum_before(sum, all);
  int first = -1, last = -1;
#pragma unroll
  for (int e = 0; e < kRun; ++e) {
    c += w[e];
    if (w[e] > 0.0) last = t0 + e;
    if (first < 0 && w[e] > 0.0 && c > target) first = t0 + e;
  }
  const uint64_t passed = passes ? __ballot(first >= 0) : 0, left = __ballot(last >= 0);
  return passed != 0 ? __shfl(first, __builtin_ctzll(passed), kWave) : __shfl(last, 63 - __builtin_clzll(left), kWave);
}

// The token drawn from target alone, where nothing is left of it: every segment is summed here. -1: none has a
// positive weight.
template <int DT>
__device__ __noinline__ int pick_plain(const stor_t<DT>* p, int segments, int vocab, double draw) {
  const Weights<DT> W{p, nullptr, -1};
  double total = 0.0;
  int last = -1;
  for (int i = 0; i < segments; ++i) {
    const double s = sum_segment<DT>(W, i, vocab);
    total += s;
    if (s > 0.0) last = i;
  }
  if (last < 0) return -1;
  const double target = draw * total;
  double c = 0.0;
  for (int i = 0; i < segments; ++i) {
    const double s = sum_segment<DT>(W, i, vocab);
    if (s > 0.0 && c + s > target) return walk<DT>(W, i, vocab, c, target, true);
    c += s;
  }
  return walk<DT>(W, last, vocab, c, target, false);
}

// The token drawn, from the segments' sums: one wavefront.
template <int DT>
__device__ __forceinline__ int pick(const Weights<DT>& W, const double* sums, int segments, int vocab, double draw) {
  const int lane = threadIdx.x & 63, per = (segments + kWave - 1) / kWave;
  const int i0 = min(lane * per, segments), i1 = min(i0 + per, segments);
  double total, mine = 0.0;
  for (int i = i0; i < i1; ++i) mine += sums[i];
  double c = sum_before(mine, total), base = 0.0;
  if (!(total > 0.0)) return pick_plain<DT>(W.p, segments, vocab, draw);
  const double target = draw * total;
  // the first segment that passes the draw, else the last one of positive sum
  int first = -1, last = -1;
  for (int i = i0; i < i1; ++i) {
    const double s = sums[i];
    if (s > 0.0) last = i;
    if (first < 0 && s > 0.0 && c + s > target) {
      first = i;
      base = c;
    }
    c += s;
  }
  const uint64_t hit = __ballot(first >= 0), some = __ballot(last >= 0);
  const int at = hit != 0 ? __builtin_ctzll(hit) : 63 - __builtin_clzll(some);
  const int seg = __shfl(hit != 0 ? first : last, at, kWave);
  return walk<DT>(W, seg, vocab, __shfl(base, at, kWave), target, hit != 0);
}

// A request's results, by one wavefront. out may be drafts: what is read of them here is written by the same lane.
__device__ __forceinline__ void finish(const VerifyArgs& A, int b, int64_t lo, int64_t hi, int64_t row, int token) {
  const int lane = threadIdx.x & 63;
  for (int64_t r = lo + lane; r < hi; r += kWave) A.out[r] = r < row ? A.drafts[r] : (r == row ? token : -1);
  if (lane == 0) A.counts[b] = static_cast<int32_t>(row - lo) + 1;
}

}  // namespace

// A wavefront per segment.
template <int DT>
__global__ __launch_bounds__(kWaves* kWave) void k_verify_sums(const VerifyArgs A) {
  const int groups = (A.segments + kWaves - 1) / kWaves;
  const int b = static_cast<int>(blockIdx.x / groups);
  const int seg = static_cast<int>(blockIdx.x % groups) * kWaves + static_cast<int>(threadIdx.x >> 6);
  int64_t lo, hi;
  sequence_rows(A.offsets, b, A.rows, lo, hi);
  if (lo >= hi || seg >= A.segments) return;
  const int64_t row = first_refused<DT>(A, lo, hi);
  const double sum = sum_segment<DT>(weights_at<DT>(A, row, hi), seg, A.vocab);
  if ((threadIdx.x & 63) == 0) {
    A.sums[static_cast<int64_t>(b) * A.segments + seg] = sum;
    if (seg == 0) A.kept[b] = static_cast<int32_t>(row - lo);
  }
}

// A wavefront per request.
template <int DT>
__global__ __launch_bounds__(kWave) void k_verify_pick(const VerifyArgs A) {
  const int b = blockIdx.x;
  const double draw = A.draws[b];
  const int kept = A.kept[b];  // of a request without rows: anything
  int64_t lo, hi;
  sequence_rows(A.offsets, b, A.rows, lo, hi);
  if (lo >= hi) {
    if (threadIdx.x == 0) A.counts[b] = 0;
    return;
  }
  const int64_t row = lo + kept;
  const int token = pick<DT>(weights_at<DT>(A, row, hi), A.sums + static_cast<int64_t>(b) * A.segments, A.segments, A.vocab, draw);
  finish(A, b, lo, hi, row, token);
}

// A workgroup per request, the sums in LDS.
template <int DT>
__global__ __launch_bounds__(kMany* kWave) void k_verify_whole(const VerifyArgs A) {
  __shared__ double sums[kMost];
  const int b = blockIdx.x, wave = threadIdx.x >> 6;
  const double draw = A.draws[b];
  int64_t lo, hi;
  sequence_rows(A.offsets, b, A.rows, lo, hi);
  if (lo >= hi) {
    if (threadIdx.x == 0) A.counts[b] = 0;
    return;
  }
  const int64_t row = first_refused<DT>(A, lo, hi);
  const Weights<DT> W = weights_at<DT>(A, row, hi);
  for (int seg = wave; seg < A.segments; seg += kMany) {
    const double sum = sum_segment<DT>(W, seg, A.vocab);
    if ((threadIdx.x & 63) == 0) sums[seg] = sum;
  }
  __syncthreads();
  if (wave != 0) return;
  finish(A, b, lo, hi, row, pick<DT>(W, sums, A.segments, A.vocab, draw));
}

namespace {

template <int DT>
hipError_t verify(const VerifyArgs& a, hipStream_t s) {
  if (a.segments <= verify_alone()) {
    k_verify_whole<DT><<<dim3(static_cast<unsigned>(a.batch)), dim3(kMany * kWave), 0, s>>>(a);
    return hipGetLastError();
  }
  const int64_t groups = (a.segments + kWaves - 1) / kWaves;
  k_verify_sums<DT><<<dim3(static_cast<unsigned>(a.batch * groups)), dim3(kWaves * kWave), 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_verify_pick<DT><<<dim3(static_cast<unsigned>(a.batch)), dim3(kWave), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

int32_t verify_segments(int32_t vocab) { return static_cast<int32_t>((static_cast<int64_t>(vocab) + kSegment - 1) / kSegment); }

int32_t verify_alone() { return kMost; }

hipError_t launch_verify(int32_t io_dtype, const VerifyArgs& a, hipStream_t s) {
  return io_dtype == SEED_BF16 ? verify<1>(a, s) : verify<0>(a, s);
}

}  // namespace seed
