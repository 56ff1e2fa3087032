// Rotary positions of packed rows, and new keys and values stored into a paged cache:
//   (a, b) <- amplitude (a cos - b sin, a sin + b cos), the angle 2 pi frac(position turns_i).
//
// What bounds it: every value is read once and written once, so HBM. A workgroup takes a token: a thread forms the
// sine and cosine of an angle (fp64: a position of 10^6 times a frequency of 1 loses 0.06 in fp32) and leaves
// them in LDS, and all run over the token's heads as they lie, twice 16 bytes each a time. Where turned parts do
// not divide so, 16 bytes, with the other values of their pairs in LDS; heads or addresses that do not divide go value by
// value.
// Measured: 32768 rows x 40 heads of 128, 671 MB: 108 us, 6.2 TB/s; 32768 prompt tokens, 16 + 2 x 4 heads of 256, into
// pages, 805 MB: 135 us, 6.0 TB/s (a large copy by torch: 5.1). A token's call: 3 us, 7 with the call's host time.
#include "attend.hpp"
#include "common.hpp"

namespace seed {

namespace {

constexpr int kThreads = 256;
using u32x4 = __attribute__((ext_vector_type(4))) uint32_t;

// The sine and cosine of a pair's angle, times the amplitude. fp32 rows: in fp64, rounded once.
template <int DT>
__device__ __forceinline__ float2 turn_of(double turns, int64_t position, float amplitude) {
  double t = turns * static_cast<double>(position);
  t -= rint(t);
  if constexpr (DT == 0) {
    double sn, cs;
    sincospi(2.0 * t, &sn, &cs);
    return make_float2(static_cast<float>(amplitude * cs), static_cast<float>(amplitude * sn));
  } else {
    float sn, cs;
    sincospif(2.f * static_cast<float>(t), &sn, &cs);
    return make_float2(amplitude * cs, amplitude * sn);
  }
}

constexpr int kMostPairs = 2048;  // angles of a token

// 16 bytes as VEC floats, and back.
template <int DT, int VEC>
__device__ __forceinline__ void unpack(const u32x4& x, float (&v)[VEC]) {
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
template <int DT, int VEC>
__device__ __forceinline__ u32x4 pack(const float (&v)[VEC]) {
  u32x4 x;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (DT == 0) x[e] = __float_as_uint(v[e]);
    else x[e] = pack2<DT>(v[2 * e], v[2 * e + 1]);
  }
  return x;
}

// n over what `per` stands for (Cut).
__device__ __forceinline__ int divide(int n, uint32_t per) { return per == 0 ? n : static_cast<int>(__umulhi(n, per)); }

// An item of a head of `dim` values whose first `rot` are turned: 16 bytes of the first half of the turned values, or of
// the rest, and the 16 bytes half of them further on, so that neighbouring threads write neighbouring bytes (32 bytes
// in a row each take twice as long). Halved pairs meet as (a[e], b[e]); interleaved ones are neighbours inside a and b.
template <int DT>
struct Item {
  static constexpr int VEC = DT == 0 ? 4 : 8;
  using T = stor_t<DT>;
  u32x4 lo, hi;
  T* y = nullptr;  // where it goes; nullptr: nowhere
  int at, half;
  bool turned;
  __device__ __forceinline__ void load(const T* x, int item, int dim, int rot) {
    const int turns = rot / (2 * VEC);
    turned = item < turns;
    half = turned ? rot / 2 : (dim - rot) / 2;
    at = turned ? item * VEC : rot + (item - turns) * VEC;
    lo = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(x + at));
    hi = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(x + at + half));
  }
  __device__ __forceinline__ void finish(const float2* cs, int interleaved) {
    if (y == nullptr) return;
    if (turned) {
      float a[VEC], b[VEC];
      unpack<DT, VEC>(lo, a);
      unpack<DT, VEC>(hi, b);
      if (interleaved) {
#pragma unroll
        for (int e = 0; e < VEC; e += 2) {
          const float2 p = cs[(at + e) / 2], q = cs[(at + half + e) / 2];
          const float a0 = a[e], a1 = a[e + 1], b0 = b[e], b1 = b[e + 1];
          a[e] = a0 * p.x - a1 * p.y;
          a[e + 1] = a0 * p.y + a1 * p.x;
          b[e] = b0 * q.x - b1 * q.y;
          b[e + 1] = b0 * q.y + b1 * q.x;
        }
      } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float2 c = cs[at + e];
          const float a0 = a[e], b0 = b[e];
          a[e] = a0 * c.x - b0 * c.y;
          b[e] = a0 * c.y + b0 * c.x;
        }
      }
      lo = pack<DT, VEC>(a);
      hi = pack<DT, VEC>(b);
    }
    __builtin_nontemporal_store(lo, reinterpret_cast<u32x4*>(y + at));
    __builtin_nontemporal_store(hi, reinterpret_cast<u32x4*>(y + at + half));
    y = nullptr;
  }
};

// 16 bytes of a head as they lie, for turned parts that do not divide into halves of 16 bytes: the other values of their
// pairs are read from LDS, where all threads of a turn leave theirs.
template <int DT>
struct AnyItem {
  static constexpr int VEC = DT == 0 ? 4 : 8;
  using T = stor_t<DT>;
  u32x4 x;
  T* y = nullptr;  // where it goes; nullptr: nowhere
  int at, rot;
  __device__ __forceinline__ void load(const T* from, int item, int, int turned) {
    at = item * VEC;
    rot = turned;
    x = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(from + at));
  }
  __device__ __forceinline__ void finish(const float2* cs, const u32x4* left, int interleaved) {
    if (y == nullptr) return;
    if (at < rot) {
      const T* head = reinterpret_cast<const T*>(left + threadIdx.x) - at;
      const int half = rot / 2;
      float v[VEC];
      unpack<DT, VEC>(x, v);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const int j = min(at + e, rot - 1);
        const bool first = interleaved ? (j & 1) == 0 : j < half;
        const int other = interleaved ? j ^ 1 : (first ? j + half : j - half), pair = interleaved ? j >> 1 : min(j, other);
        const float o = to_f32<DT>(head[other]);
        const float2 c = cs[pair];
        v[e] = v[e] * c.x + (first ? -o : o) * c.y;
      }
      const u32x4 turned = pack<DT, VEC>(v);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = at + e * (VEC / 4) < rot ? turned[e] : x[e];
    }
    __builtin_nontemporal_store(x, reinterpret_cast<u32x4*>(y + at));
    y = nullptr;
  }
};

// All items of a token: n of them, loaded by fetch() and sent on their way by aim(), by turns of the workgroup's threads
// (ANY: of whole heads, the next turn's loaded ahead); the first are loaded while angles() finds the token's place and
// forms its angles (673 tokens of 40 heads of 64 into pages 6.9 us, with the place first 7.5).
template <int DT, bool ANY, typename Fetch, typename Angles, typename Aim>
__device__ __forceinline__ void turn_token(int n, int items, int interleaved, const float2* cs, Fetch fetch, Angles angles, Aim aim) {
  __shared__ u32x4 left[ANY ? 2 : 1][ANY ? kThreads : 1];
  const int tid = threadIdx.x;
  if constexpr (ANY) {
    const int turn = kThreads / items * items;
    AnyItem<DT> it;
    if (tid < turn && tid < n) fetch(it, tid);
    if (!angles()) return;
    for (int i0 = 0, buffer = 0; i0 < n; i0 += turn, buffer ^= 1) {
      const bool mine = tid < turn && i0 + tid < n;
      if (mine) {
        aim(it, i0 + tid);
        left[buffer][tid] = it.x;
      }
      __syncthreads();  // what the turn before the last one left has been read
      AnyItem<DT> next;
      if (tid < turn && i0 + turn + tid < n) fetch(next, i0 + turn + tid);
      it.finish(cs, left[buffer], interleaved);
      it = next;
    }
  } else {
    Item<DT> it;
    if (tid < n) fetch(it, tid);
    if (!angles()) return;
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
      if (i != tid) fetch(it, i);
      aim(it, i);
      it.finish(cs, interleaved);
    }
  }
}

// Where a new token goes: its request's position, and the place of it in the cache (-1: not there).
struct Place {
  int64_t position, slot;
  bool mine;  // of a request at all
};
__device__ __forceinline__ Place place_of(const CacheArgs& C, int64_t row, int b) {
  Place p{0, -1, false};
  if (b >= C.batch) return p;
  int64_t lo, hi;
  request_rows(C, b, lo, hi);
  if (row < lo || row >= hi) return p;
  p.mine = true;
  p.position = static_cast<int64_t>(C.lengths[b]) - (hi - row);
  const int64_t entry = p.position >> C.page_shift;
  if (p.position < 0 || entry >= C.width) return p;
  const int64_t number = C.table[static_cast<int64_t>(b) * C.width + entry];
  if (number >= 0 && number < C.pages)
    p.slot = number * C.page_stride + (p.position & ((int64_t{1} << C.page_shift) - 1)) * C.token_stride;
  return p;
}
// The number of requests that end at or before row `first`, found by a whole wavefront.
__device__ __forceinline__ int requests_before(const CacheArgs& C, int64_t first) {
  const int lane = threadIdx.x & (kWave - 1);
  int b = 0;
  for (int j = 0; j < C.batch; j += kWave)
    b += __popcll(__ballot(j + lane < C.batch && C.offsets[min(j + lane, C.batch - 1) + 1] <= first));
  return b;
}
__device__ __forceinline__ int request_of(const CacheArgs& C, int64_t row, int b) {
  while (b < C.batch && C.offsets[b + 1] <= row) ++b;
  return b;
}

}  // namespace

// A workgroup per token and heads_each of its heads (blockIdx.y), `items` items each. One token: with several, whose
// sines are formed together, 32768 rows x 40 heads take 112 us (two) to 132 (sixteen) in the place of 106.
template <int DT, bool ANY>
__global__ __launch_bounds__(kThreads) void k_rotate_rows(const RotateArgs A, int heads_each, int items, uint32_t per_item) {
  using T = stor_t<DT>;
  __shared__ float2 cs[kMostPairs];
  const int64_t row = blockIdx.x;
  const int h0 = static_cast<int>(blockIdx.y) * heads_each, n = min(heads_each, A.heads - h0) * items;
  const T* x = static_cast<const T*>(A.x) + row * A.x_stride + static_cast<int64_t>(h0) * A.dim;
  T* y = static_cast<T*>(A.y) + row * A.y_stride + static_cast<int64_t>(h0) * A.dim;
  turn_token<DT, ANY>(
      n, items, A.interleaved, cs,
      [&](auto& it, int i) {
        const int h = divide(i, per_item);
        it.load(x + h * A.dim, i - h * items, A.dim, A.rot);
      },
      [&] {
        const int position = A.positions[row];
        for (int i = threadIdx.x; i < A.rot / 2; i += kThreads) cs[i] = turn_of<DT>(A.turns[i], position, A.amplitude);
        return true;
      },
      [&](auto& it, int i) { it.y = y + divide(i, per_item) * A.dim; });
}

// The same for the rows of seed_cache_append: of all heads of a token, the queries come first, then the keys, then the
// values.
template <int DT, bool ANY>
__global__ __launch_bounds__(kThreads) void k_cache_append(const AppendArgs A, int heads_each, int items, uint32_t per_item) {
  using T = stor_t<DT>;
  __shared__ float2 cs[kMostPairs];
  const CacheArgs& C = A.c;
  const int64_t row = blockIdx.x;
  const int queries = A.q != nullptr ? C.heads : 0, all = queries + 2 * C.key_heads;
  const int h0 = static_cast<int>(blockIdx.y) * heads_each, n = min(heads_each, all - h0) * items;
  const T* q = static_cast<const T*>(A.q) + row * A.q_stride;
  const T* k = static_cast<const T*>(A.k) + row * A.k_stride;
  const T* v = static_cast<const T*>(A.v) + row * A.v_stride;
  T* qo = static_cast<T*>(A.q_out) + row * A.o_stride;
  Place p;
  turn_token<DT, ANY>(
      n, items, A.interleaved, cs,
      [&](auto& it, int i) {
        const int part = divide(i, per_item), item = i - part * items, h = h0 + part, kh = h - queries, vh = kh - C.key_heads;
        if (kh < 0) it.load(q + static_cast<int64_t>(h) * C.dim, item, C.dim, A.rot);
        else if (vh < 0) it.load(k + static_cast<int64_t>(kh) * C.dim, item, C.dim, A.rot);
        else it.load(v + static_cast<int64_t>(vh) * C.dim, item, C.dim, 0);
      },
      [&] {
        // every wavefront for itself
        p = place_of(C, row, C.offsets != nullptr ? request_of(C, row, requests_before(C, row)) : static_cast<int>(row));
        if (!p.mine) return false;
        for (int i = threadIdx.x; i < A.rot / 2; i += kThreads) cs[i] = turn_of<DT>(A.turns[i], p.position, A.amplitude);
        return true;
      },
      [&](auto& it, int i) {
        const int h = h0 + divide(i, per_item), kh = h - queries, vh = kh - C.key_heads;
        if (kh < 0) it.y = qo + static_cast<int64_t>(h) * C.dim;
        else if (p.slot < 0) it.y = nullptr;
        else it.y = vh < 0 ? static_cast<T*>(C.k) + p.slot + kh * C.head_stride : static_cast<T*>(C.v) + p.slot + vh * C.head_stride;
      });
}

// Value by value: a thread has one pair of a token, or one value of the rest, for heads part, part + parts, ..
template <int DT>
__global__ __launch_bounds__(kThreads) void k_rotate_values(const RotateArgs A, int items, int parts) {
  using T = stor_t<DT>;
  const int64_t all = A.rows * parts * items, step = static_cast<int64_t>(gridDim.x) * kThreads;
  const int pairs = A.rot / 2;
  for (int64_t id = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x; id < all; id += step) {
    const int64_t group = id / items, row = group / parts;
    const int item = static_cast<int>(id - group * items), part = static_cast<int>(group - row * parts);
    const T* x = static_cast<const T*>(A.x) + row * A.x_stride;
    T* y = static_cast<T*>(A.y) + row * A.y_stride;
    if (item < pairs) {
      const float2 c = turn_of<DT>(A.turns[item], A.positions[row], A.amplitude);
      const int at = A.interleaved ? 2 * item : item, to = A.interleaved ? at + 1 : at + pairs;
      for (int h = part; h < A.heads; h += parts) {
        const int64_t head = static_cast<int64_t>(h) * A.dim;
        const float a = to_f32<DT>(x[head + at]), b = to_f32<DT>(x[head + to]);
        y[head + at] = from_f32<DT>(a * c.x - b * c.y);
        y[head + to] = from_f32<DT>(a * c.y + b * c.x);
      }
    } else {
      for (int h = part; h < A.heads; h += parts) {
        const int64_t at = static_cast<int64_t>(h) * A.dim + pairs + item;
        y[at] = x[at];
      }
    }
  }
}

template <int DT>
__global__ __launch_bounds__(kThreads) void k_append_values(const AppendArgs A, int items, int parts) {
  using T = stor_t<DT>;
  const CacheArgs& C = A.c;
  const int64_t all = C.tokens * parts * items, step = static_cast<int64_t>(gridDim.x) * kThreads;
  const int pairs = A.rot / 2, queries = A.q != nullptr ? C.heads : 0;
  const int lane = threadIdx.x & (kWave - 1);
  // whole wavefronts stay in the loop together: they look for their first row's request with all lanes
  for (int64_t id0 = static_cast<int64_t>(blockIdx.x) * kThreads + (threadIdx.x - lane); id0 < all; id0 += step) {
    const int64_t id = id0 + lane, group = id / items, row = group / parts;
    const int item = static_cast<int>(id - group * items), part = static_cast<int>(group - row * parts);
    const int first = C.offsets != nullptr ? requests_before(C, id0 / items / parts) : 0;
    if (id >= all) continue;
    const Place p = place_of(C, row, C.offsets != nullptr ? request_of(C, row, first) : static_cast<int>(row));
    if (!p.mine) continue;
    const T* q = static_cast<const T*>(A.q) + row * A.q_stride;
    const T* k = static_cast<const T*>(A.k) + row * A.k_stride;
    const T* v = static_cast<const T*>(A.v) + row * A.v_stride;
    T* qo = static_cast<T*>(A.q_out) + row * A.o_stride;
    T* ko = static_cast<T*>(C.k) + p.slot;
    T* vo = static_cast<T*>(C.v) + p.slot;
    const int last = queries + (p.slot >= 0 ? C.key_heads : 0);
    float2 c = make_float2(1.f, 0.f);
    int at = pairs + item, to = at;
    if (item < pairs) {
      c = turn_of<DT>(A.turns[item], p.position, A.amplitude);
      at = A.interleaved ? 2 * item : item;
      to = A.interleaved ? at + 1 : at + pairs;
    }
    for (int h = part; h < last; h += parts) {
      const int kh = h - queries;
      const T* x = kh < 0 ? q + static_cast<int64_t>(h) * C.dim : k + static_cast<int64_t>(kh) * C.dim;
      T* y = kh < 0 ? qo + static_cast<int64_t>(h) * C.dim : ko + kh * C.head_stride;
      if (item < pairs) {
        const float a = to_f32<DT>(x[at]), b = to_f32<DT>(x[to]);
        y[at] = from_f32<DT>(a * c.x - b * c.y);
        y[to] = from_f32<DT>(a * c.y + b * c.x);
      } else {
        y[at] = x[at];
      }
    }
    if (p.slot >= 0) {
      for (int h = part; h < C.key_heads; h += parts)
        for (int i = item; i < C.dim; i += items) vo[h * C.head_stride + i] = v[static_cast<int64_t>(h) * C.dim + i];
    }
  }
}

namespace {

// Value by value: threads enough to fill the chip before a thread takes more than one head, whose angles are one. 1024 rows
// x 40 heads 8.0 us, 15 with a thread per head, 17 with one for all; 16384 rows 94, 189 and 95; 1 row 3.1 and 11.5.
int parts_of(int64_t threads, int heads) {
  constexpr int64_t kFill = 256 * 1024;
  const int64_t p = threads > 0 ? (kFill + threads - 1) / threads : 1;
  return static_cast<int>(p < heads ? p : heads);
}

// The launch over tokens whose heads divide into items: the heads of a workgroup, all but where tokens are few. 1024 rows
// x 40 heads 5.0 us cut, 6.0 whole; 2048 and 4096 the same; 16384 rows 58 cut, 55 whole.
struct Cut {
  int heads_each;
  uint32_t per_item;  // 2^32 over items, rounded up (0 for 1): exact for indexes below 2^32 / items
  dim3 grid;
};
Cut cut(int64_t rows, int heads, int items) {
  Cut c;
  c.heads_each = heads;
  if (rows < 2048) {  // a turn of the threads each
    c.heads_each = kThreads / items > 1 ? kThreads / items : 1;
    c.heads_each = c.heads_each < heads ? c.heads_each : heads;
  }
  c.per_item = static_cast<uint32_t>((0xffffffffull + items) / items);
  c.grid = dim3(static_cast<unsigned>(rows), static_cast<unsigned>((heads + c.heads_each - 1) / c.heads_each));
  return c;
}
// How a token's heads go: as pairs of 16 bytes where heads and turned parts divide into two of them, as 16 bytes and what
// LDS holds of the others where only the heads divide, or value by value; the first two within what the launch counts.
// 16384 rows x 40 heads of 128 values, bf16: all turned 55 us as pairs, 78 by LDS, 81 value by value; 98 to 124 of them
// 78 by LDS, 166 to 171 value by value (bound by the vector unit both); fp32 8192 rows 58, 61, 86 and 61, 117. One row
// takes the same.
enum class Way { kPairs, kAny, kValues };
Way way(int64_t rows, int64_t heads, int dim, int rot, int vec, bool aligned) {
  if (!aligned || dim % vec != 0 || rot / 2 > kMostPairs || rows >= (1 << 24) || heads * dim > (1 << 20)) return Way::kValues;
  if (dim % (2 * vec) == 0 && rot % (2 * vec) == 0) return heads * (dim / (2 * vec)) * (dim / (2 * vec)) < (int64_t{1} << 32) ? Way::kPairs : Way::kValues;
  return dim / vec <= kThreads ? Way::kAny : Way::kValues;
}

template <int DT>
hipError_t rotate(const RotateArgs& a, bool aligned, hipStream_t s) {
  constexpr int VEC = DT == 0 ? 4 : 8;
  const bool in_place = a.x == a.y;
  const Way w = way(a.rows, a.heads, a.dim, a.rot, VEC, aligned);
  if (w != Way::kValues) {
    const int turned = in_place ? a.rot : a.dim, items = w == Way::kPairs ? turned / (2 * VEC) : (turned + VEC - 1) / VEC;
    const Cut c = cut(a.rows, a.heads, items);
    if (w == Way::kPairs) k_rotate_rows<DT, false><<<c.grid, dim3(kThreads), 0, s>>>(a, c.heads_each, items, c.per_item);
    else k_rotate_rows<DT, true><<<c.grid, dim3(kThreads), 0, s>>>(a, c.heads_each, items, c.per_item);
  } else {
    const int items = in_place ? a.rot / 2 : a.dim - a.rot / 2, parts = parts_of(a.rows * items, a.heads);
    k_rotate_values<DT><<<dim3(loop_blocks((a.rows * parts * items + kThreads - 1) / kThreads)), dim3(kThreads), 0, s>>>(a, items, parts);
  }
  return hipGetLastError();
}

template <int DT>
hipError_t append(const AppendArgs& a, bool aligned, hipStream_t s) {
  constexpr int VEC = DT == 0 ? 4 : 8;
  const int queries = a.q != nullptr ? a.c.heads : 0;
  const Way w = way(a.c.tokens, queries + 2 * static_cast<int64_t>(a.c.key_heads), a.c.dim, a.rot, VEC, aligned);
  if (w != Way::kValues) {
    const int items = a.c.dim / (w == Way::kPairs ? 2 * VEC : VEC);
    const Cut c = cut(a.c.tokens, queries + 2 * a.c.key_heads, items);
    if (w == Way::kPairs) k_cache_append<DT, false><<<c.grid, dim3(kThreads), 0, s>>>(a, c.heads_each, items, c.per_item);
    else k_cache_append<DT, true><<<c.grid, dim3(kThreads), 0, s>>>(a, c.heads_each, items, c.per_item);
  } else {
    const int items = a.c.dim - a.rot / 2, parts = parts_of(a.c.tokens * items, queries + a.c.key_heads);
    k_append_values<DT><<<dim3(loop_blocks((a.c.tokens * parts * items + kThreads - 1) / kThreads)), dim3(kThreads), 0, s>>>(a, items, parts);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_rotate_rows(int32_t io_dtype, const RotateArgs& a, hipStream_t s) {
  const int bytes = io_dtype == SEED_BF16 ? 2 : 4;
  const bool aligned = rows_aligned16(a.x, a.x_stride, bytes) && rows_aligned16(a.y, a.y_stride, bytes);
  return io_dtype == SEED_BF16 ? rotate<1>(a, aligned, s) : rotate<0>(a, aligned, s);
}

hipError_t launch_cache_append(int32_t io_dtype, const AppendArgs& a, hipStream_t s) {
  const int bytes = io_dtype == SEED_BF16 ? 2 : 4;
  bool aligned = rows_aligned16(a.k, a.k_stride, bytes) && rows_aligned16(a.v, a.v_stride, bytes);
  if (a.q != nullptr) aligned = aligned && rows_aligned16(a.q, a.q_stride, bytes) && rows_aligned16(a.q_out, a.o_stride, bytes);
  return io_dtype == SEED_BF16 ? append<1>(a, aligned, s) : append<0>(a, aligned, s);
}

}  // namespace seed
