// Internal launch interface of the prompt path (prompt_api.cpp to conv.hip, scan.hip and
// norm_rows.hip), and the device helpers those kernels share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/seed.h"

namespace seed {

struct ConvArgs {
  int64_t tokens;          // prefill: rows of x and y
  int32_t batch;
  int32_t channels;
  int32_t silu;
  int64_t x_stride, y_stride;  // elements between rows
  const int32_t* offsets;  // prefill: [batch + 1]
  const uint8_t* active;   // decode: requests with active[b] == 0 are skipped (nullptr: none)
  const void* x;
  const float* weight;     // [width][channels]
  const float* bias;       // [channels] or nullptr
  const void* win_in;      // [batch][width - 1][channels] or nullptr (zeros; prefill only)
  void* win_out;
  void* y;
};

struct ScanArgs {
  int64_t tokens;
  int32_t batch, heads, key_heads;
  int64_t q_stride, k_stride, v_stride, o_stride;
  const int32_t* offsets;  // [batch + 1]
  const void* q;           // [tokens][key_heads][d_k]
  const void* k;
  const void* v;           // [tokens][heads][d_v]
  const float* beta;       // [tokens][heads]
  const float* g;          // [tokens][heads], KDA [tokens][heads][d_k]
  const float* S0;         // [batch][heads][d_k][d_v] or nullptr (zeros)
  float* S;
  void* o;                 // [tokens][heads][d_v]
  void* ws;                // of prefill_scan_workspace bytes
};

struct NormArgs {
  int64_t rows;
  int32_t heads, dim;
  int64_t x_stride, y_stride, gate_stride, skip_stride, total_stride;
  const void* x;
  const float* weight;      // [heads][dim]
  const void* gate;         // nullptr: none
  const void* skip;         // nullptr: none
  const float* skip_scale;  // [heads] or nullptr (1)
  void* total;              // nullptr: not written
  void* y;
  float eps;
  int32_t gate_first;
};

hipError_t launch_prefill_conv(const seed_conv& c, const ConvArgs& a, hipStream_t s);
hipError_t launch_decode_conv(const seed_conv& c, const ConvArgs& a, hipStream_t s);
hipError_t launch_prefill_scan(const seed_shape& sh, const ScanArgs& a, hipStream_t s);
size_t prefill_scan_workspace(const seed_shape& sh, const seed_prompt& p);
// The chunked scan on the matrix cores: bf16 io, scalar gates (GDN, Mamba-2).
hipError_t launch_scan_chunk(const seed_shape& sh, const ScanArgs& a, hipStream_t s);
size_t scan_chunk_workspace(const seed_shape& sh, int64_t tokens);
hipError_t launch_norm_rows(int32_t io_dtype, const NormArgs& a, hipStream_t s);

// Whether p and a row stride (in elements of `bytes`) let every row be accessed 16 bytes at a time.
inline bool rows_aligned16(const void* p, int64_t stride, int64_t bytes) {
  return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ((stride * bytes) & 15) == 0;
}

// Blocks of a launch that loops over `work` items: enough to fill the chip many times over, few
// enough that blocks times threads stays below the launch limit of 2^32.
inline unsigned loop_blocks(int64_t work) {
  constexpr int64_t kMost = int64_t{1} << 22;
  return static_cast<unsigned>(work < kMost ? work : kMost);
}

#ifdef __HIPCC__
// Rows [lo, hi) of sequence b. offsets lives in device memory and is not checked on the host:
// entries are clamped into [0, tokens] and a decreasing pair reads as an empty sequence, so no
// content of offsets reaches outside the row buffers.
__device__ __forceinline__ void sequence_rows(const int32_t* __restrict__ offsets, int b, int64_t tokens,
                                              int64_t& lo, int64_t& hi) {
  int64_t l = offsets[b], h = offsets[b + 1];
  l = l < 0 ? 0 : (l > tokens ? tokens : l);
  h = h < l ? l : (h > tokens ? tokens : h);
  lo = l;
  hi = h;
}

// y / (1 + e^-y) in the place of every y. 16-bit outputs take the hardware exponential and reciprocal,
// fp32 ones the library's. The rounding of the exponential's argument grows with |y|: the relative
// error is below 2^-20 for |y| <= 8 and 2^-17 for y >= -80, where a 16-bit output is rounded by 2^-9. Below
// -80 the sum is e^-y and would overflow, and its reciprocal underflow, while y e^y is a normal
// number down to -91: there y e^(y/2) e^(y/2), good to 2^-16. One branch for all N: with one for each,
// 32768 rows x 8192 bf16 channels of the convolution take 199 us instead of 194.
template <int DT, int N>
__device__ __forceinline__ void silu(float (&y)[N]) {
  float low = y[0];
#pragma unroll
  for (int e = 1; e < N; ++e) low = fminf(low, y[e]);
  float r[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    if constexpr (DT == 0) r[e] = y[e] / (1.f + expf(-y[e]));
    else r[e] = y[e] * __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-1.4426950408889634f * y[e]));
  }
  if (__builtin_expect(low < -80.f, 0)) {
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float h = DT == 0 ? expf(0.5f * y[e]) : __builtin_amdgcn_exp2f(0.7213475204444817f * y[e]);
      if (y[e] < -80.f) r[e] = y[e] * h * h;
    }
  }
#pragma unroll
  for (int e = 0; e < N; ++e) y[e] = r[e];
}
#endif

}  // namespace seed
