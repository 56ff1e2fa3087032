// Head norm of packed rows, with the residual, its scale and the gate fused in:
//   x' = x + s[h] skip;  u = x' silu(z) when gate_first, else x';
//   y = w[h] u / sqrt(mean over dim of u^2 + eps)  (times silu(z) when a gate is given and !gate_first)
// for rows x heads groups of dim values: the norm of prompt read-outs (dim = d_v, as the decode
// step's epilogue has it), or the norm before a block (heads = 1, dim = the model's width, skip the
// residual stream, the sum written back).
//
// What bounds it: each stream is read or written once, so HBM. The group's values stay in
// registers between the sum of squares and the product. Groups of up to 512 values (16-byte
// accesses: 8 bf16 or 4 fp32 per lane) take 8 .. 64 lanes of one wavefront each, summed with DPP;
// wider ones, up to 8192 bf16 or 4096 fp32 values, a 256-thread workgroup. Wider groups still, and addresses,
// strides or widths that do not allow 16-byte accesses, take one workgroup per group, one value per
// access, which reads its inputs twice.
// Measured: 32768 rows x 64 heads x 64 bf16 values with gate and residual, 182 us (5.9 TB/s).
// Every value is read by the thread that writes it, before it writes: y may be x, and total skip.
#include "common.hpp"
#include "prompt.hpp"

namespace seed {

namespace {

constexpr int kThreads = 256;

// One thread's share of a group: loads its values, forms x' and the squares' sum; finish() writes.
template <int DT, int VEC>
struct Share {
  float u[VEC], z[VEC];
  __device__ __forceinline__ float load(const NormArgs& A, int64_t row, int h, int i) {
    const int64_t col = static_cast<int64_t>(h) * A.dim + i;
    using T = stor_t<DT>;
    load_f32<DT, VEC>(static_cast<const T*>(A.x) + row * A.x_stride + col, u);
    if (A.skip != nullptr) {
      float r[VEC];
      load_f32<DT, VEC>(static_cast<const T*>(A.skip) + row * A.skip_stride + col, r);
      const float sc = A.skip_scale != nullptr ? A.skip_scale[h] : 1.f;
#pragma unroll
      for (int e = 0; e < VEC; ++e) u[e] = fmaf(sc, r[e], u[e]);
    }
    if (A.gate != nullptr) {
      load_f32<DT, VEC>(static_cast<const T*>(A.gate) + row * A.gate_stride + col, z);
      silu<DT>(z);
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float w = A.gate != nullptr && A.gate_first ? u[e] * z[e] : u[e];
      s = fmaf(w, w, s);
    }
    return s;
  }
  __device__ __forceinline__ void finish(const NormArgs& A, int64_t row, int h, int i, float inv) {
    const int64_t col = static_cast<int64_t>(h) * A.dim + i;
    using T = stor_t<DT>;
    if (A.total != nullptr) store_f32<DT, VEC>(static_cast<T*>(A.total) + row * A.total_stride + col, u);
    float w[VEC], y[VEC];
    load_f32<0, VEC>(A.weight + col, w);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      y[e] = u[e] * inv * w[e];
      if (A.gate != nullptr) y[e] *= z[e];  // before or after the norm: the same factor of the product
    }
    store_f32<DT, VEC>(static_cast<T*>(A.y) + row * A.y_stride + col, y);
  }
};

__device__ __forceinline__ float block_sum(float v, float* red) {
  v = wave_sum(v);
  __syncthreads();  // the last group's sum has been read
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  return (red[0] + red[1]) + (red[2] + red[3]);
}

}  // namespace

// Groups of at most LANES * VEC values: LANES lanes of a wavefront per group.
template <int DT, int VEC, int LANES>
__global__ __launch_bounds__(kThreads) void k_norm_wave(const NormArgs A, int64_t groups) {
  constexpr int kPer = kThreads / LANES;
  const int i = (threadIdx.x % LANES) * VEC;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kPer;
  // whole wavefronts stay in the loop together: the sum needs all 64 lanes
  for (int64_t g0 = static_cast<int64_t>(blockIdx.x) * kPer; g0 < groups; g0 += step) {
    const int64_t g = g0 + threadIdx.x / LANES;
    const bool live = g < groups && i < A.dim;
    const int64_t row = g / A.heads;
    const int h = static_cast<int>(g - row * A.heads);
    Share<DT, VEC> sh;
    float s = 0.f;
    if (live) s = sh.load(A, row, h, i);
    s = group_sum<LANES>(s);
    if (live) sh.finish(A, row, h, i, 1.f / sqrtf(s / static_cast<float>(A.dim) + A.eps));
  }
}

// Groups of at most kThreads * VEC * N values: a workgroup per group.
template <int DT, int VEC, int N>
__global__ __launch_bounds__(kThreads) void k_norm_block(const NormArgs A, int64_t groups) {
  __shared__ float red[kThreads / kWave];
  for (int64_t g = blockIdx.x; g < groups; g += gridDim.x) {
    const int64_t row = g / A.heads;
    const int h = static_cast<int>(g - row * A.heads);
    Share<DT, VEC> sh[N];
    float s = 0.f;
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int i = (n * kThreads + threadIdx.x) * VEC;
      if (i < A.dim) s += sh[n].load(A, row, h, i);
    }
    s = block_sum(s, red);
    const float inv = 1.f / sqrtf(s / static_cast<float>(A.dim) + A.eps);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int i = (n * kThreads + threadIdx.x) * VEC;
      if (i < A.dim) sh[n].finish(A, row, h, i, inv);
    }
  }
}

// Any width, any address: one value per access, read again for the second pass.
template <int DT>
__global__ __launch_bounds__(kThreads) void k_norm_scalar(const NormArgs A, int64_t groups) {
  __shared__ float red[kThreads / kWave];
  for (int64_t g = blockIdx.x; g < groups; g += gridDim.x) {
    const int64_t row = g / A.heads;
    const int h = static_cast<int>(g - row * A.heads);
    Share<DT, 1> sh;
    float s = 0.f;
    for (int i = threadIdx.x; i < A.dim; i += kThreads) s += sh.load(A, row, h, i);
    s = block_sum(s, red);
    const float inv = 1.f / sqrtf(s / static_cast<float>(A.dim) + A.eps);
    for (int i = threadIdx.x; i < A.dim; i += kThreads) {
      sh.load(A, row, h, i);
      sh.finish(A, row, h, i, inv);
    }
  }
}

namespace {

template <int DT, int VEC, int LANES>
hipError_t wave(const NormArgs& a, int64_t groups, hipStream_t s) {
  const int64_t per = kThreads / LANES;
  k_norm_wave<DT, VEC, LANES><<<dim3(loop_blocks((groups + per - 1) / per)), dim3(kThreads), 0, s>>>(a, groups);
  return hipGetLastError();
}

template <int DT, int VEC, int N>
hipError_t block(const NormArgs& a, int64_t groups, hipStream_t s) {
  k_norm_block<DT, VEC, N><<<dim3(loop_blocks(groups)), dim3(kThreads), 0, s>>>(a, groups);
  return hipGetLastError();
}

template <int DT, int VEC>
hipError_t pick(const NormArgs& a, int64_t groups, hipStream_t s) {
  constexpr int bytes = DT == 0 ? 4 : 2;
  bool v = a.dim % VEC == 0 && rows_aligned16(a.x, a.x_stride, bytes) && rows_aligned16(a.y, a.y_stride, bytes) &&
           rows_aligned16(a.weight, 0, 4);
  if (a.gate != nullptr) v = v && rows_aligned16(a.gate, a.gate_stride, bytes);
  if (a.skip != nullptr) v = v && rows_aligned16(a.skip, a.skip_stride, bytes);
  if (a.total != nullptr) v = v && rows_aligned16(a.total, a.total_stride, bytes);
  if (!v || a.dim > kThreads * VEC * 4) {
    k_norm_scalar<DT><<<dim3(loop_blocks(groups)), dim3(kThreads), 0, s>>>(a, groups);
    return hipGetLastError();
  }
  if (a.dim <= 8 * VEC) return wave<DT, VEC, 8>(a, groups, s);
  if (a.dim <= 16 * VEC) return wave<DT, VEC, 16>(a, groups, s);
  if (a.dim <= 32 * VEC) return wave<DT, VEC, 32>(a, groups, s);
  if (a.dim <= 64 * VEC) return wave<DT, VEC, 64>(a, groups, s);
  if (a.dim <= kThreads * VEC) return block<DT, VEC, 1>(a, groups, s);
  if (a.dim <= kThreads * VEC * 2) return block<DT, VEC, 2>(a, groups, s);
  return block<DT, VEC, 4>(a, groups, s);
}

}  // namespace

hipError_t launch_norm_rows(int32_t io_dtype, const NormArgs& a, hipStream_t s) {
  const int64_t groups = a.rows * a.heads;
  return io_dtype == SEED_BF16 ? pick<1, 8>(a, groups, s) : pick<0, 4>(a, groups, s);
}

}  // namespace seed
