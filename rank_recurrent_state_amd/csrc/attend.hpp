// Internal launch interface of the attention layers (attend_api.cpp to attend_plan.cpp, rotate.hip, attend.hip
// and verify.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/seed.h"
#include "prompt.hpp"

namespace seed {

// Workgroups of a launch: it has fewer than 2^32 threads.
constexpr int64_t most_blocks(int64_t threads) { return ((int64_t{1} << 32) - 1) / threads; }

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
  uint32_t pages;           // of the pool, as far as table entries reach
  int32_t row_waves;        // wavefronts of a workgroup that have rows of their own
  int32_t block_rows;       // rows that a workgroup takes at a time, of max_tokens share,
  int32_t row_blocks;       // and how many times
  int32_t change;           // turns that a change of rows costs, counted with a row block's
  int32_t few;              // groups 0: as few keys as one turn of a small workgroup
  int32_t groups;           // workgroups that share a key head's turns; 0: a workgroup per request and key head
  int64_t q_stride, o_stride;
  const void* q;
  void* o;
  float* lse;      // nullptr: not written
  float* part;     // [groups][key_heads][2][block_rows][dim]: accumulators of rows that several workgroups have (groups 1: none),
  float* stat;     // and their maximum and sum [..][block_rows][2]
  int32_t* notes;  // [batch][row_blocks][2]: the first and last workgroup of each
};

// What the attention's plan and its kernels share.
namespace plan {
inline constexpr int kWaves = 4;  // of a workgroup; short caches take kMany
inline constexpr int kMany = 8;
inline constexpr int kShared = 16384;  // bytes of keys in a tile that the wavefronts share
}  // namespace plan

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
  double* sums;   // [batch][segments] of the weights
  int32_t* kept;  // [batch]
};

hipError_t launch_rotate_rows(int32_t io_dtype, const RotateArgs& a, hipStream_t s);
hipError_t launch_cache_append(int32_t io_dtype, const AppendArgs& a, hipStream_t s);
// Sets row_waves, block_rows, row_blocks, change, few and groups from the sizes; false: more turns or workgroups than are
// counted.
bool plan_attend(int32_t io_dtype, AttendArgs& a);
// Rows of partial results: two places for each workgroup, none where one has all of a key head's turns.
int64_t attend_places(const AttendArgs& a);
int64_t attend_workspace(const AttendArgs& a);
hipError_t launch_attend(int32_t io_dtype, AttendArgs a, void* ws, hipStream_t s);
int32_t verify_segments(int32_t vocab);
int32_t verify_alone();  // most segments of a request that one workgroup does without a workspace
inline constexpr int32_t kAloneThreads = 1024;  // of that workgroup
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
