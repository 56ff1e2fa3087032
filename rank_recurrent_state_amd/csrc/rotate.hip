// Rotary positions of packed rows, and new keys and values stored into a paged cache:
//   (a, b) <- amplitude (a cos - b sin, a sin + b cos), the angle 2 pi frac(position turns_i).
//
// What bounds it: every value is read once and written once, so HBM. A thread owns some neighbouring pairs of
// a token, forms their sines once (the angle in fp64: a position of 10^6 times a frequency of 1 loses 0.06
// in fp32) and applies them to one head after another; the fewer tokens, the more threads share a token's heads.
#include "attend.hpp"
#include "common.hpp"

namespace seed {

namespace {

constexpr int kThreads = 256;

// The pairs of VEC neighbouring angles: values [0, VEC) and [VEC, 2 VEC) of an item. In halves they are two
// accesses rot / 2 apart; interleaved they are one run of 2 VEC values.
template <int DT, int VEC>
struct Pairs {
  float c[VEC], s[VEC];
  __device__ __forceinline__ void angles(const double* __restrict__ turns, int i, int64_t position, float amplitude) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      double t = turns[i + e] * static_cast<double>(position);
      t -= rint(t);
      float sn, cs;
      sincospif(2.f * static_cast<float>(t), &sn, &cs);
      c[e] = amplitude * cs;
      s[e] = amplitude * sn;
    }
  }
  __device__ __forceinline__ void turn(const stor_t<DT>* __restrict__ x, stor_t<DT>* __restrict__ y, int i, int rot,
                                       int interleaved) const {
    float a[VEC], b[VEC], p[VEC], q[VEC];
    const int at = interleaved ? 2 * i : i, to = interleaved ? 2 * i + VEC : i + rot / 2;
    load_f32<DT, VEC>(x + at, a);
    load_f32<DT, VEC>(x + to, b);
    if (interleaved) {
      if constexpr (VEC == 1) {
        p[0] = a[0] * c[0] - b[0] * s[0];
        q[0] = a[0] * s[0] + b[0] * c[0];
      } else {
#pragma unroll
        for (int e = 0; e < VEC / 2; ++e) {
          p[2 * e] = a[2 * e] * c[e] - a[2 * e + 1] * s[e];
          p[2 * e + 1] = a[2 * e] * s[e] + a[2 * e + 1] * c[e];
          q[2 * e] = b[2 * e] * c[VEC / 2 + e] - b[2 * e + 1] * s[VEC / 2 + e];
          q[2 * e + 1] = b[2 * e] * s[VEC / 2 + e] + b[2 * e + 1] * c[VEC / 2 + e];
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        p[e] = a[e] * c[e] - b[e] * s[e];
        q[e] = a[e] * s[e] + b[e] * c[e];
      }
    }
    store_f32<DT, VEC>(y + at, p);
    store_f32<DT, VEC>(y + to, q);
  }
};

template <int DT, int VEC>
__device__ __forceinline__ void copy(const stor_t<DT>* __restrict__ x, stor_t<DT>* __restrict__ y) {
  if constexpr (VEC == 1) *y = *x;
  else *reinterpret_cast<uint4*>(y) = *reinterpret_cast<const uint4*>(x);
}

}  // namespace

// Thread (token, part, item): item < rot / 2 / VEC turns VEC pairs, the ones behind copy VEC values of the rest;
// heads part, part + parts, .. of the token.
template <int DT, int VEC>
__global__ __launch_bounds__(kThreads) void k_rotate_rows(const RotateArgs A, int items, int parts) {
  using T = stor_t<DT>;
  const int64_t all = A.rows * parts * items, step = static_cast<int64_t>(gridDim.x) * kThreads;
  const int turned = A.rot / 2 / VEC;
  for (int64_t id = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; id < all; id += step) {
    const int64_t group = id / items;
    const int item = static_cast<int>(id - group * items);
    const int64_t row = group / parts;
    const int part = static_cast<int>(group - row * parts);
    const T* x = static_cast<const T*>(A.x) + row * A.x_stride;
    T* y = static_cast<T*>(A.y) + row * A.y_stride;
    if (item < turned) {
      Pairs<DT, VEC> pr;
      pr.angles(A.turns, item * VEC, A.positions[row], A.amplitude);
      for (int h = part; h < A.heads; h += parts) {
        const int64_t at = static_cast<int64_t>(h) * A.dim;
        pr.turn(x + at, y + at, item * VEC, A.rot, A.interleaved);
      }
    } else {
      const int i = A.rot + (item - turned) * VEC;
      for (int h = part; h < A.heads; h += parts) {
        const int64_t at = static_cast<int64_t>(h) * A.dim + i;
        copy<DT, VEC>(x + at, y + at);
      }
    }
  }
}

// The same for the rows of seed_cache_append: heads 0 .. heads - 1 are the queries, then the keys, then the values.
template <int DT, int VEC>
__global__ __launch_bounds__(kThreads) void k_cache_append(const AppendArgs A, int items, int parts) {
  using T = stor_t<DT>;
  const CacheArgs& C = A.c;
  const int64_t all = C.tokens * parts * items, step = static_cast<int64_t>(gridDim.x) * kThreads;
  const int turned = A.rot / 2 / VEC;
  const int queries = A.q != nullptr ? C.heads : 0;
  const int lane = threadIdx.x & (kWave - 1);
  // whole wavefronts stay in the loop together: they look for their first row's request with all lanes
  for (int64_t id0 = static_cast<int64_t>(blockIdx.x) * kThreads + (threadIdx.x - lane); id0 < all; id0 += step) {
    const int64_t id = id0 + lane;
    const int64_t group = id / items;
    const int item = static_cast<int>(id - group * items);
    const int64_t row = group / parts;
    const int part = static_cast<int>(group - row * parts);
    int b = 0;
    if (C.offsets == nullptr) {
      b = static_cast<int>(row);
    } else {  // the number of requests that end at or before the wavefront's first row, then on to this thread's
      const int64_t first = id0 / items / parts;
      for (int j = 0; j < C.batch; j += kWave)
        b += __popcll(__ballot(j + lane < C.batch && C.offsets[min(j + lane, C.batch - 1) + 1] <= first));
      while (b < C.batch && C.offsets[b + 1] <= row) ++b;
    }
    if (id >= all || b >= C.batch) continue;
    int64_t lo, hi;
    request_rows(C, b, lo, hi);
    if (row < lo || row >= hi) continue;
    const int64_t position = static_cast<int64_t>(C.lengths[b]) - (hi - row);
    const int64_t entry = position >> C.page_shift;
    int64_t number = -1;
    if (position >= 0 && entry < C.width) number = C.table[static_cast<int64_t>(b) * C.width + entry];
    const bool there = number >= 0 && number < C.pages;
    const int64_t slot = there ? number * C.page_stride + (position & ((int64_t{1} << C.page_shift) - 1)) * C.token_stride : 0;
    const T* q = static_cast<const T*>(A.q) + row * A.q_stride;
    const T* k = static_cast<const T*>(A.k) + row * A.k_stride;
    const T* v = static_cast<const T*>(A.v) + row * A.v_stride;
    T* qo = static_cast<T*>(A.q_out) + row * A.o_stride;
    T* ko = static_cast<T*>(C.k) + slot;
    T* vo = static_cast<T*>(C.v) + slot;
    const int last = queries + (there ? C.key_heads : 0);
    if (item < turned) {
      Pairs<DT, VEC> pr;
      pr.angles(A.turns, item * VEC, position, A.amplitude);
      for (int h = part; h < last; h += parts) {
        const int kh = h - queries;
        const int64_t at = static_cast<int64_t>(kh < 0 ? h : kh) * C.dim;
        pr.turn((kh < 0 ? q : k) + at, kh < 0 ? qo + at : ko + kh * C.head_stride, item * VEC, A.rot, A.interleaved);
      }
    } else {
      const int i = A.rot + (item - turned) * VEC;
      for (int h = part; h < last; h += parts) {
        const int kh = h - queries;
        const int64_t at = static_cast<int64_t>(kh < 0 ? h : kh) * C.dim + i;
        copy<DT, VEC>((kh < 0 ? q : k) + at, kh < 0 ? qo + at : ko + kh * C.head_stride + i);
      }
    }
    if (there) {
      for (int h = part; h < C.key_heads; h += parts)
        for (int i = item * VEC; i < C.dim; i += items * VEC)
          copy<DT, VEC>(v + static_cast<int64_t>(h) * C.dim + i, vo + h * C.head_stride + i);
    }
  }
}

namespace {

// Threads enough to fill the chip before a thread takes more than one head.
int parts_of(int64_t threads, int heads) {
  constexpr int64_t kFill = 256 * 1024;
  const int64_t p = threads > 0 ? (kFill + threads - 1) / threads : 1;
  return static_cast<int>(p < heads ? p : heads);
}

template <int DT, int VEC>
hipError_t rotate(const RotateArgs& a, hipStream_t s) {
  const bool in_place = a.x == a.y;
  const int items = a.rot / 2 / VEC + (in_place ? 0 : (a.dim - a.rot) / VEC);
  const int parts = parts_of(a.rows * items, a.heads);
  const int64_t blocks = (a.rows * parts * items + kThreads - 1) / kThreads;
  k_rotate_rows<DT, VEC><<<dim3(loop_blocks(blocks)), dim3(kThreads), 0, s>>>(a, items, parts);
  return hipGetLastError();
}

template <int DT, int VEC>
hipError_t append(const AppendArgs& a, hipStream_t s) {
  const int items = a.rot / 2 / VEC + (a.c.dim - a.rot) / VEC;
  const int heads = (a.q != nullptr ? a.c.heads : 0) + a.c.key_heads;
  const int parts = parts_of(a.c.tokens * items, heads);
  const int64_t blocks = (a.c.tokens * parts * items + kThreads - 1) / kThreads;
  k_cache_append<DT, VEC><<<dim3(loop_blocks(blocks)), dim3(kThreads), 0, s>>>(a, items, parts);
  return hipGetLastError();
}

// Whether heads and their rotated part divide into 16-byte accesses.
bool whole(int dim, int rot, int vec) { return dim % vec == 0 && rot % (2 * vec) == 0; }

}  // namespace

hipError_t launch_rotate_rows(int32_t io_dtype, const RotateArgs& a, hipStream_t s) {
  const int bytes = io_dtype == SEED_BF16 ? 2 : 4, vec = 16 / bytes;
  const bool v = whole(a.dim, a.rot, vec) && rows_aligned16(a.x, a.x_stride, bytes) && rows_aligned16(a.y, a.y_stride, bytes);
  if (io_dtype == SEED_BF16) return v ? rotate<1, 8>(a, s) : rotate<1, 1>(a, s);
  return v ? rotate<0, 4>(a, s) : rotate<0, 1>(a, s);
}

hipError_t launch_cache_append(int32_t io_dtype, const AppendArgs& a, hipStream_t s) {
  const int bytes = io_dtype == SEED_BF16 ? 2 : 4, vec = 16 / bytes;
  bool v = whole(a.c.dim, a.rot, vec) && rows_aligned16(a.k, a.k_stride, bytes) && rows_aligned16(a.v, a.v_stride, bytes);
  if (a.q != nullptr) v = v && rows_aligned16(a.q, a.q_stride, bytes) && rows_aligned16(a.q_out, a.o_stride, bytes);
  if (io_dtype == SEED_BF16) return v ? append<1, 8>(a, s) : append<1, 1>(a, s);
  return v ? append<0, 4>(a, s) : append<0, 1>(a, s);
}

}  // namespace seed
