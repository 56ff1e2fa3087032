// Drives the attention entry points with pseudo-random arguments out of a list of edge values, on the host: built
// with attend_api.cpp and the launchers below under sanitizers. A call that reaches a launcher must have
// rows, strides and sizes whose arithmetic the kernels' types hold; no pointer is read or written but `turns`.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdio.h>
#include <stdlib.h>

#include "../../include/seed.h"
#include "../../rank_recurrent_state_amd/csrc/attend.hpp"

namespace {
int launches = 0, accepted = 0;

void need(bool ok, const char* what) {
  if (!ok) {
    printf("accepted without: %s\n", what);
    exit(1);
  }
}
// Bytes from a buffer's first value to behind its last stay in the address range.
void holds(const void* p, int64_t rows, int64_t stride, int64_t width, int64_t bytes, const char* what) {
  if (p == nullptr || rows <= 0) return;
  const __int128 end = static_cast<__int128>(reinterpret_cast<uintptr_t>(p)) + (static_cast<__int128>(rows - 1) * stride + width) * bytes;
  need(rows <= 0x7fffffffLL && stride >= width && width > 0 && end <= static_cast<__int128>(UINTPTR_MAX), what);
}
void cache_holds(const seed::CacheArgs& c) {
  need(c.batch > 0 && c.key_heads > 0 && c.width > 0 && c.pages > 0 && c.page_shift >= 4 && c.page_shift <= 20, "cache sizes");
  need((static_cast<int64_t>(c.width) << c.page_shift) <= (int64_t{1} << 30), "positions in 32 bits");
  need(c.token_stride <= (1 << 24), "places of 16 positions in 32 bits");
  const __int128 end = (static_cast<__int128>(c.pages - 1) * c.page_stride + static_cast<__int128>((1 << c.page_shift) - 1) * c.token_stride +
                        static_cast<__int128>(c.key_heads - 1) * c.head_stride + c.dim) * 4;
  need(end < (static_cast<__int128>(1) << 60), "pool in 64 bits");
}
}  // namespace

namespace seed {
hipError_t launch_rotate_rows(int32_t t, const RotateArgs& a, hipStream_t) {
  ++launches;
  const int64_t e = t == SEED_F32 ? 4 : 2, w = static_cast<int64_t>(a.heads) * a.dim;
  holds(a.x, a.rows, a.x_stride, w, e, "x");
  holds(a.y, a.rows, a.y_stride, w, e, "y");
  need(a.rot >= 2 && a.rot <= a.dim && a.rot % 2 == 0 && a.turns && a.positions && a.rows > 0, "rotation");
  return hipSuccess;
}
hipError_t launch_cache_append(int32_t t, const AppendArgs& a, hipStream_t) {
  ++launches;
  cache_holds(a.c);
  const int64_t e = t == SEED_F32 ? 4 : 2, kw = static_cast<int64_t>(a.c.key_heads) * a.c.dim, qw = static_cast<int64_t>(a.c.heads) * a.c.dim;
  holds(a.k, a.c.tokens, a.k_stride, kw, e, "k");
  holds(a.v, a.c.tokens, a.v_stride, kw, e, "v");
  if (a.q) holds(a.q, a.c.tokens, a.q_stride, qw, e, "q");
  if (a.q) holds(a.q_out, a.c.tokens, a.o_stride, qw, e, "q_out");
  need(!a.q == !a.q_out && a.c.tokens > 0, "q and q_out");
  return hipSuccess;
}
bool plan_attend(int32_t, AttendArgs& a) {
  const int64_t rows = static_cast<int64_t>(a.max_tokens) * a.share;
  need(a.max_tokens >= 1 && a.max_tokens <= 32 && a.share >= 1 && a.share <= (1 << 14) && a.capacity >= 1, "attention sizes");
  need(rows * a.c.key_heads * a.c.batch < (1 << 24), "rows in a launch");
  need(a.scale2 > 0.f && isfinite(a.scale2), "scale");
  a.block_rows = rows < 64 ? static_cast<int32_t>(rows) : 64;
  a.row_blocks = static_cast<int32_t>((rows + 63) / 64);
  a.groups = a.capacity > 512 ? 64 : 0;
  return true;
}
int64_t attend_workspace(const AttendArgs& a) { return a.groups == 0 ? 0 : static_cast<int64_t>(a.groups) * 1000 + 8; }
hipError_t launch_attend(int32_t t, AttendArgs a, void* ws, hipStream_t) {
  ++launches;
  cache_holds(a.c);
  const int64_t e = t == SEED_F32 ? 4 : 2, w = static_cast<int64_t>(a.c.heads) * a.c.dim;
  holds(a.q, a.c.tokens, a.q_stride, w, e, "q");
  holds(a.o, a.c.tokens, a.o_stride, w, e, "o");
  holds(a.lse, a.c.tokens, a.c.heads, a.c.heads, 4, "lse");
  need(a.groups == 0 || ws != nullptr, "workspace");
  return hipSuccess;
}
int32_t verify_segments(int32_t vocab) { return static_cast<int32_t>((static_cast<int64_t>(vocab) + 1023) / 1024); }
int32_t verify_alone() { return 32; }
hipError_t launch_verify(int32_t t, const VerifyArgs& a, hipStream_t) {
  ++launches;
  const int64_t e = t == SEED_F32 ? 4 : 2;
  holds(a.target, a.rows, a.target_stride, a.vocab, e, "target");
  if (a.draft) holds(a.draft, a.rows, a.draft_stride, a.vocab, e, "draft");
  need(a.batch > 0 && a.vocab > 0 && a.vocab <= (1 << 30) && static_cast<int64_t>(a.batch) * a.segments < (1 << 24), "verification sizes");
  need(a.segments <= 32 || (a.sums && a.kept), "workspace");
  return hipSuccess;
}
}  // namespace seed

namespace {
uint64_t state = 88172645463325252ull;
uint32_t next() {
  state ^= state << 13;
  state ^= state >> 7;
  state ^= state << 17;
  return static_cast<uint32_t>(state >> 32);
}
template <typename T, size_t N>
T any(const T (&v)[N]) {
  return v[next() % N];
}
// Mostly the sensible value, sometimes an edge.
int32_t i32(int32_t good) {
  const int32_t edge[] = {0, 1, -1, 2, 3, 16, 63, 64, 65, 255, 256, 1 << 20, 1 << 24, 1 << 30, 0x7fffffff, -0x7fffffff - 1};
  return next() % 12 ? good : any(edge);
}
int64_t i64(int64_t good) {
  const int64_t edge[] = {0, 1, -1, 8, 24, 1 << 24, (1 << 24) + 8, int64_t{1} << 31, int64_t{1} << 40, (int64_t{1} << 40) + 8, int64_t{1} << 50,
                          int64_t{1} << 62, INT64_MAX, INT64_MIN};
  return next() % 12 ? good : any(edge);
}
void* at(uintptr_t good) {
  const uintptr_t edge[] = {0, 1, 16, 8, 4096, UINTPTR_MAX - 15, UINTPTR_MAX - 4095, uintptr_t{1} << 63, good + 2, good + 4};
  return reinterpret_cast<void*>(next() % 16 ? good : any(edge));
}
template <typename T>
T* to(uintptr_t good) {
  return static_cast<T*>(at(good));
}
void tally(int status, int before, const char* what) {
  const bool known = status == SEED_OK || status == SEED_ERR_ARG || status == SEED_ERR_UNSUPPORTED || status == SEED_ERR_WORKSPACE;
  need(known && launches - before <= 1 && (status == SEED_OK || launches == before), what);
  accepted += launches - before;
}
constexpr uintptr_t kFar = uintptr_t{1} << 44;  // buffers that lie apart
}  // namespace

int main() {
  for (int turn = 0; turn < 300000; ++turn) {
    const int32_t dims[] = {64, 128, 256}, pages[] = {16, 64, 1 << 20}, types[] = {SEED_F32, SEED_BF16};
    const int32_t dim = any(dims), page = any(pages), kh = 1 + next() % 4, type = i32(any(types)), batch = i32(1 + next() % 300);
    const bool by_head = next() % 2;
    seed_cache c{};
    c.batch = batch;
    c.key_heads = i32(kh);
    c.dim = i32(dim);
    c.io_dtype = type;
    c.page = i32(page);
    c.width = i32(1 + next() % 100);
    c.pages = i64(1 + next() % 1000);
    c.page_stride = i64(static_cast<int64_t>(page) * kh * dim);
    c.token_stride = i64(by_head ? dim : kh * dim);
    c.head_stride = i64(by_head ? static_cast<int64_t>(page) * dim : dim);
    c.k = at(kFar);
    c.v = at(2 * kFar);
    c.table = to<const int32_t>(3 * kFar);
    const int32_t heads = i32(kh * static_cast<int32_t>(1 + next() % 16));
    const int64_t w = static_cast<int64_t>(heads) * dim, n = i64(batch);
    seed_tokens t{};
    t.tokens = n;
    t.offsets = next() % 2 ? to<const int32_t>(4 * kFar) : nullptr;
    t.lengths = to<const int32_t>(5 * kFar);
    t.heads = heads;
    t.q_stride = i64(w);
    t.o_stride = i64(w);
    t.k_stride = i64(static_cast<int64_t>(kh) * dim);
    t.v_stride = i64(static_cast<int64_t>(kh) * dim);
    const float amplitudes[] = {1.f, 1.f, 1.2f, NAN, INFINITY};
    const seed_rotary rotary{i32(dim / 2), i32(next() % 2), any(amplitudes), to<const double>(6 * kFar)};
    const float scales[] = {0.1f, -0.5f, 0.f, 1e-45f, 3e38f, NAN, INFINITY, 1.f};
    const seed_attend how{i32(1 + next() % 32), i32(1 + next() % 600), i32(next() % 2 ? 0 : 100), any(scales)};
    int before = launches;
    tally(seed_cache_append(next() % 50 ? &c : nullptr, next() % 50 ? &t : nullptr, next() % 2 ? &rotary : nullptr, at(7 * kFar), at(8 * kFar),
                            at(9 * kFar), at(10 * kFar), nullptr),
          before, "append");
    before = launches;
    const size_t bytes = seed_attend_workspace_bytes(&c, &t, &how);
    tally(seed_decode_attend(&c, &t, next() % 50 ? &how : nullptr, at(7 * kFar), at(8 * kFar), next() % 2 ? to<float>(9 * kFar) : nullptr,
                             at(11 * kFar), next() % 8 ? bytes : bytes / 2, nullptr),
          before, "attend");
    before = launches;
    seed_rows rows{};
    rows.rows = n;
    rows.heads = heads;
    rows.dim = i32(dim);
    rows.io_dtype = type;
    rows.x_stride = i64(w);
    rows.y_stride = i64(w);
    tally(seed_rotate_rows(&rows, &rotary, at(7 * kFar), to<const int32_t>(8 * kFar), at(next() % 2 ? 7 * kFar : 9 * kFar), nullptr), before, "rotate");
    before = launches;
    const int32_t vocab = i32(1 + next() % 200000);
    const seed_drafts d{batch, vocab, type, n, to<const int32_t>(3 * kFar), i64(vocab), i64(vocab)};
    const size_t sums = seed_verify_workspace_bytes(&d);
    tally(seed_verify_drafts(&d, at(4 * kFar), next() % 2 ? at(5 * kFar) : nullptr, to<const int32_t>(6 * kFar), to<const float>(7 * kFar),
                             to<const float>(8 * kFar), to<int32_t>(next() % 2 ? 6 * kFar : 9 * kFar), to<int32_t>(10 * kFar), at(11 * kFar),
                             next() % 8 ? sums : sums / 2, nullptr),
          before, "verify");
    double turns[128];
    const double values[] = {1e4, 1.0, 0.0, -1.0, 1e-300, 1e300, NAN, INFINITY, 5e-324, 32.0, 4096.0};
    const seed_rotary_scaling s{static_cast<int32_t>(next() % 7) - 1, any(values), any(values), any(values), any(values), any(values)};
    const int32_t wide = static_cast<int32_t>(next() % 257);
    if (seed_rotary_turns(&s, wide, turns) == SEED_OK)
      for (int32_t i = 0; i < wide / 2; ++i) need(isfinite(turns[i]), "finite turns");
  }
  need(accepted > 50000, "calls that are accepted");
  printf("attend_validate ok: %d accepted\n", accepted);
  return 0;
}
