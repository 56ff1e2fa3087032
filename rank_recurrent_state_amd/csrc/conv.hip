// Short causal convolution of a recurrent layer's projected channels, for packed prompts and for
// single tokens:
//   y_t = act(bias + sum_{j < W} w_j x_{t - W + 1 + j}),  act = identity or SiLU, W = 2 .. 4,
// per channel, with the W - 1 inputs before a sequence's first one taken from its window.
//
// What bounds it: every input is read once and every output written once, a few FMAs each, so HBM.
// A thread owns 8 (16-bit) or 4 (fp32) adjacent channels, one 16-byte access per row, and keeps
// its taps' weights in registers. Prompts: a thread walks kRows rows of its channels with the last
// W - 1 inputs in registers, so a row is read again only by the tile behind it (W - 1 rows in
// kRows, out of L2). Tiles are cut by row, not by sequence, so short and long sequences load the
// chip alike; a tile inside one sequence takes a loop without boundary checks whose loads are all
// issued first. Channel counts, strides or addresses that do not allow 16-byte accesses take
// the same kernels with one channel per thread. Sums are fp32 and rounded once.
// Measured: 32768 rows of 16 prompts x 8192 bf16 channels, windows carried, 194 us (5.5 TB/s); 512 tokens x
// 12288 bf16 channels 22 us (4.6 TB/s); one channel per thread, 3001 rows x 1037 fp32 channels, 11.7 us
// (2.1 TB/s, the call included).
#include "common.hpp"
#include "prompt.hpp"

namespace seed {

namespace {

constexpr int kThreads = 256;
constexpr int kRows = 16;  // rows of a prompt tile

template <int DT, int VEC>
__device__ __forceinline__ void load_row(const void* base, int64_t at, float (&out)[VEC]) {
  load_f32<DT, VEC>(static_cast<const stor_t<DT>*>(base) + at, out);
}
template <int DT, int VEC>
__device__ __forceinline__ void store_row(void* base, int64_t at, const float (&in)[VEC]) {
  store_f32<DT, VEC>(static_cast<stor_t<DT>*>(base) + at, in);
}

template <int W, int VEC>
struct Taps {
  float w[W][VEC];
  float b[VEC];
  __device__ __forceinline__ void load(const ConvArgs& A, int64_t c) {
#pragma unroll
    for (int j = 0; j < W; ++j) load_f32<0, VEC>(A.weight + j * static_cast<int64_t>(A.channels) + c, w[j]);
    if (A.bias != nullptr) {
      load_f32<0, VEC>(A.bias + c, b);
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) b[e] = 0.f;
    }
  }
  // x[0 .. W-2]: the inputs before, oldest first; x[W-1]: the row's own
  template <int DT>
  __device__ __forceinline__ void apply(const float (&x)[W][VEC], int act, float (&y)[VEC]) const {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      float s = b[e];
#pragma unroll
      for (int j = 0; j < W; ++j) s = fmaf(w[j][e], x[j][e], s);
      y[e] = s;
    }
    if (act) silu<DT>(y);
  }
};

}  // namespace

template <int W, int DT, int VEC>
__global__ __launch_bounds__(kThreads) void k_prefill_conv(const ConvArgs A, int64_t tiles, int64_t cblocks, int64_t work) {
  for (int64_t item = blockIdx.x; item < work; item += gridDim.x) {
    const int64_t cb = item % cblocks, tile = item / cblocks;
    const int64_t c = (cb * kThreads + threadIdx.x) * VEC;
    if (c >= A.channels) continue;
    if (tile >= tiles) {
      // a sequence's new window: its last W - 1 inputs, those of the old window where it is shorter
      const int b = static_cast<int>(tile - tiles);
      int64_t lo, hi;
      sequence_rows(A.offsets, b, A.tokens, lo, hi);
      const int64_t n = hi - lo;
      const int64_t wrow = static_cast<int64_t>(b) * (W - 1);
      float r[W - 1][VEC];
#pragma unroll
      for (int i = 0; i < W - 1; ++i) {
        const int64_t p = n - (W - 1) + i;
        if (p >= 0) {
          load_row<DT, VEC>(A.x, (lo + p) * A.x_stride + c, r[i]);
        } else if (A.win_in != nullptr) {
          load_row<DT, VEC>(A.win_in, (wrow + (W - 1) + p) * A.channels + c, r[i]);
        } else {
#pragma unroll
          for (int e = 0; e < VEC; ++e) r[i][e] = 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < W - 1; ++i) store_row<DT, VEC>(A.win_out, (wrow + i) * A.channels + c, r[i]);
      continue;
    }

    const int64_t r0 = tile * kRows;
    const int64_t r1 = r0 + kRows < A.tokens ? r0 + kRows : A.tokens;
    // the last sequence that starts at or before row r0
    int lo_b = 0, hi_b = A.batch;
    while (hi_b - lo_b > 1) {
      const int mid = (lo_b + hi_b) >> 1;
      if (A.offsets[mid] <= r0) lo_b = mid;
      else hi_b = mid;
    }
    int b = lo_b;
    int64_t s, e;
    sequence_rows(A.offsets, b, A.tokens, s, e);

    Taps<W, VEC> taps;
    taps.load(A, c);

    if (s + (W - 1) <= r0 && r0 + kRows <= e) {
      float x[kRows + W - 1][VEC];
#pragma unroll
      for (int i = 0; i < kRows + W - 1; ++i) load_row<DT, VEC>(A.x, (r0 - (W - 1) + i) * A.x_stride + c, x[i]);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        float y[VEC], h[W][VEC];
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
          for (int q = 0; q < VEC; ++q) h[j][q] = x[i + j][q];
        taps.template apply<DT>(h, A.silu, y);
        store_row<DT, VEC>(A.y, (r0 + i) * A.y_stride + c, y);
      }
      continue;
    }

    float h[W][VEC];
    bool fresh = true;  // the history has to be read for the next row
    for (int64_t r = r0; r < r1; ++r) {
      while (r >= e && b + 1 < A.batch) {
        ++b;
        sequence_rows(A.offsets, b, A.tokens, s, e);
        fresh = true;
      }
      if (r >= e) break;     // behind the last sequence
      if (r < s) continue;   // before the first one
      if (fresh) {
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
          const int64_t p = r - s - (W - 1) + j;  // place in the sequence, below 0 in the window
          if (p >= 0) {
            load_row<DT, VEC>(A.x, (s + p) * A.x_stride + c, h[j]);
          } else if (A.win_in != nullptr) {
            load_row<DT, VEC>(A.win_in, (static_cast<int64_t>(b) * (W - 1) + (W - 1) + p) * A.channels + c, h[j]);
          } else {
#pragma unroll
            for (int q = 0; q < VEC; ++q) h[j][q] = 0.f;
          }
        }
        fresh = false;
      }
      load_row<DT, VEC>(A.x, r * A.x_stride + c, h[W - 1]);
      float y[VEC];
      taps.template apply<DT>(h, A.silu, y);
      store_row<DT, VEC>(A.y, r * A.y_stride + c, y);
#pragma unroll
      for (int j = 0; j + 1 < W; ++j)
#pragma unroll
        for (int q = 0; q < VEC; ++q) h[j][q] = h[j + 1][q];
    }
  }
}

// One token per request: the window's rows and x give y; the window moves up by one.
template <int W, int DT, int VEC>
__global__ __launch_bounds__(kThreads) void k_decode_conv(const ConvArgs A, int64_t cblocks, int64_t work) {
  for (int64_t item = blockIdx.x; item < work; item += gridDim.x) {
    const int64_t cb = item % cblocks;
    const int64_t b = item / cblocks;
    const int64_t c = (cb * kThreads + threadIdx.x) * VEC;
    if (c >= A.channels || (A.active != nullptr && A.active[b] == 0)) continue;
    Taps<W, VEC> taps;
    taps.load(A, c);
    float h[W][VEC], y[VEC];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) load_row<DT, VEC>(A.win_in, (b * (W - 1) + j) * A.channels + c, h[j]);
    load_row<DT, VEC>(A.x, b * A.x_stride + c, h[W - 1]);
    taps.template apply<DT>(h, A.silu, y);
    store_row<DT, VEC>(A.y, b * A.y_stride + c, y);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_row<DT, VEC>(A.win_out, (b * (W - 1) + j) * A.channels + c, h[j + 1]);
  }
}

namespace {

bool vector_ok(const seed_conv& c, const ConvArgs& a) {
  const int64_t bytes = c.io_dtype == SEED_F32 ? 4 : 2;
  const int64_t vec = 16 / bytes;
  auto at16 = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; };
  return a.channels % vec == 0 && rows_aligned16(a.x, a.x_stride, bytes) && rows_aligned16(a.y, a.y_stride, bytes) &&
         at16(a.weight) && at16(a.bias) && at16(a.win_in) && at16(a.win_out);
}

template <int W, int DT, int VEC>
hipError_t prefill(const ConvArgs& a, hipStream_t s) {
  const int64_t cblocks = (a.channels + kThreads * VEC - 1) / (kThreads * VEC);
  const int64_t tiles = (a.tokens + kRows - 1) / kRows;
  const int64_t work = (tiles + a.batch) * cblocks;
  k_prefill_conv<W, DT, VEC><<<dim3(loop_blocks(work)), dim3(kThreads), 0, s>>>(a, tiles, cblocks, work);
  return hipGetLastError();
}

template <int W, int DT, int VEC>
hipError_t decode(const ConvArgs& a, hipStream_t s) {
  const int64_t cblocks = (a.channels + kThreads * VEC - 1) / (kThreads * VEC);
  const int64_t work = static_cast<int64_t>(a.batch) * cblocks;
  k_decode_conv<W, DT, VEC><<<dim3(loop_blocks(work)), dim3(kThreads), 0, s>>>(a, cblocks, work);
  return hipGetLastError();
}

template <int W>
hipError_t pick(const seed_conv& c, const ConvArgs& a, bool dec, hipStream_t s) {
  const bool v = vector_ok(c, a);
  if (c.io_dtype == SEED_BF16) {
    if (v) return dec ? decode<W, 1, 8>(a, s) : prefill<W, 1, 8>(a, s);
    return dec ? decode<W, 1, 1>(a, s) : prefill<W, 1, 1>(a, s);
  }
  if (v) return dec ? decode<W, 0, 4>(a, s) : prefill<W, 0, 4>(a, s);
  return dec ? decode<W, 0, 1>(a, s) : prefill<W, 0, 1>(a, s);
}

hipError_t pick_width(const seed_conv& c, const ConvArgs& a, bool dec, hipStream_t s) {
  switch (c.width) {
    case 2: return pick<2>(c, a, dec, s);
    case 3: return pick<3>(c, a, dec, s);
    case 4: return pick<4>(c, a, dec, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_prefill_conv(const seed_conv& c, const ConvArgs& a, hipStream_t s) { return pick_width(c, a, false, s); }
hipError_t launch_decode_conv(const seed_conv& c, const ConvArgs& a, hipStream_t s) { return pick_width(c, a, true, s); }

}  // namespace seed
