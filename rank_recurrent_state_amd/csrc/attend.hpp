// Internal launch interface of the attention layers (attend_api.cpp to rotate.hip, attend.hip and
// verify.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/seed.h"
#include "prompt.hpp"

namespace seed {

struct RotateArgs {
  int64_t rows;
  int32_t heads, dim, rot, interleaved;
  float amplitude;
  int64_t x_stride, y_stride;
  const double* turns;
  const int32_t* positions;
  const void* x;
  void* y;
};

// A seed_cache and seed_tokens as the kernels take them; strides in elements.
struct CacheArgs {
  int32_t batch, heads, key_heads, dim;
  int32_t page_shift, width;
  int64_t pages, page_stride, token_stride, head_stride;
  void* k;
  void* v;
  const int32_t* table;
  int64_t tokens;
  const int32_t* offsets;  // nullptr: row b is request b's
  const int32_t* lengths;
};

struct AppendArgs {
  CacheArgs c;
  int32_t rot, interleaved;  // rot 0: no rotation
  float amplitude;
  const double* turns;
  int64_t q_stride, k_stride, v_stride, o_stride;
  const void* q;  // nullptr: none
  const void* k;
  const void* v;
  void* q_out;
};

struct AttendArgs {
  CacheArgs c;
  int32_t max_tokens, capacity, window;
  int32_t share;            // heads / key_heads
  float per_share;          // 1 / share
  float scale2;             // |scale| log2(e)
  uint32_t negate;          // the sign bits of a word of q, where scale is negative
  int32_t chunk, splits;    // keys of a workgroup, and workgroups along the longest cache
  bool many;                // more wavefronts in the place of more workgroups
  int64_t q_stride, o_stride;
  const void* q;
  void* o;
  float* lse;   // nullptr: not written
  float* part;  // [tokens][heads][splits][dim], then [tokens][heads][splits][2]: weights' maximum and sum
  float* stat;
};

struct VerifyArgs {
  int32_t batch, vocab, segments;
  int64_t rows, target_stride, draft_stride;
  const int32_t* offsets;
  const void* target;
  const void* draft;
  const int32_t* drafts;
  const float* uniforms;
  const float* draws;
  int32_t* out;
  int32_t* counts;
  double* sums;   // [batch][segments][2]: of the weights, and of target
  int32_t* kept;  // [batch]
};

hipError_t launch_rotate_rows(int32_t io_dtype, const RotateArgs& a, hipStream_t s);
hipError_t launch_cache_append(int32_t io_dtype, const AppendArgs& a, hipStream_t s);
// Sets chunk, splits and many from the sizes.
void plan_attend(int32_t io_dtype, AttendArgs& a);
hipError_t launch_attend(int32_t io_dtype, const AttendArgs& a, hipStream_t s);
int32_t verify_segments(int32_t vocab);
hipError_t launch_verify(int32_t io_dtype, const VerifyArgs& a, hipStream_t s);

#ifdef __HIPCC__
// Rows [lo, hi) of request b.
__device__ __forceinline__ void request_rows(const CacheArgs& c, int b, int64_t& lo, int64_t& hi) {
  if (c.offsets != nullptr) {
    sequence_rows(c.offsets, b, c.tokens, lo, hi);
  } else {
    lo = b;
    hi = b + 1;
  }
}
#endif

}  // namespace seed
