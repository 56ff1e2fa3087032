// Drives the attention's plan (attend_plan.cpp) on the host with sizes that the entry point lets through, edge values among
// them, under sanitizers: the launches, the turns that the device counts in 32 bits and the workspace hold.
#include <stdio.h>
#include <stdlib.h>

#include <algorithm>

#include "../../include/seed.h"
#include "../../rank_recurrent_state_amd/csrc/attend.hpp"

namespace {
using wide = __int128;
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
int32_t size(int32_t most) {  // spread over its logarithm, the ends more often
  if (next() % 8 == 0) return next() % 2 ? most : 1;
  const int bits = 32 - __builtin_clz(static_cast<uint32_t>(most));
  return std::min(most, static_cast<int32_t>(1 + next() % (1u << (1 + next() % bits))));
}
void need(bool ok, const char* what, const seed::AttendArgs& a, int type) {
  if (ok) return;
  printf("%s: type %d batch %d key heads %d dim %d share %d tokens %d length %d window %d: waves %d rows %d blocks %d groups %d\n", what, type, a.c.batch,
         a.c.key_heads, a.c.dim, a.share, a.max_tokens, a.capacity, a.window, a.row_waves, a.block_rows, a.row_blocks, a.groups);
  exit(1);
}
}  // namespace

int main() {
  const wide launch = wide{1} << 32;
  int whole = 0, cut = 0, refused = 0;
  for (int turn = 0; turn < 2000000; ++turn) {
    const int32_t dims[] = {64, 128, 256}, types[] = {SEED_F32, SEED_BF16};
    const int type = any(types);
    seed::AttendArgs a{};
    a.c.dim = any(dims);
    a.share = size(1 << 14);
    a.max_tokens = size(32);
    const int32_t rows = a.share * a.max_tokens, most = (1 << 24) - 1;
    if (rows > most) continue;
    a.c.key_heads = size(std::min(most / rows, 1 << 20));
    a.c.batch = size(most / rows / a.c.key_heads);
    a.c.heads = a.c.key_heads * a.share;
    a.capacity = size(1 << 30);
    a.window = next() % 2 ? 0 : size(1 << 30);
    if (a.window >= a.capacity) a.window = 0;
    if (!seed::plan_attend(type, a)) {
      ++refused;
      continue;
    }
    need(a.row_waves == 1 || a.row_waves == 2 || a.row_waves == 4, "wavefronts with rows", a, type);
    need(a.block_rows >= 1 && a.block_rows <= 16 * a.row_waves && a.row_blocks >= 1, "rows of a block", a, type);
    need(wide{a.row_blocks} * a.block_rows >= rows && wide{a.row_blocks - 1} * a.block_rows < rows, "row blocks", a, type);
    need(a.row_waves > 1 || a.row_blocks == 1, "one block of own keys", a, type);
    const wide units = wide{a.c.batch} * a.c.key_heads * a.row_blocks, need_bytes = seed::attend_workspace(a);
    if (a.groups == 0) {
      ++whole;
      need(units * (a.row_waves == 1 && !a.few ? 512 : 256) < launch, "threads of whole requests", a, type);
      need(need_bytes == 0, "no workspace", a, type);
      continue;
    }
    ++cut;
    need(a.groups >= 1 && a.groups <= 512 && wide{a.groups} * a.c.key_heads * 256 < launch, "threads of shares", a, type);
    // what the device adds up, at most: keys from a multiple of 32 on, and a row block's change
    const wide keys = a.window > 0 ? std::min<wide>(a.capacity, wide{a.window} + a.max_tokens - 1 + 31) : a.capacity;
    const int32_t row = a.c.dim * (type == SEED_F32 ? 4 : 2);
    const int32_t step = a.row_waves == 1 ? (type == SEED_F32 ? 64 : 128) : 16384 / row;
    const wide turns = wide{a.c.batch} * a.row_blocks * ((keys + step - 1) / step + a.change), share = std::max<wide>((turns + a.groups - 1) / a.groups, 1);
    need(turns < (wide{1} << 30) && (share + 1) * a.groups < (wide{1} << 31), "turns in 32 bits", a, type);
    const wide places = a.groups > 1 ? wide{a.groups} * a.c.key_heads * 2 * a.block_rows : 0;
    need(seed::attend_places(a) == places && places <= 2 * wide{511 + a.c.key_heads} * 64, "places", a, type);
    need(need_bytes == places * (a.c.dim + 2) * 4 + wide{a.c.batch} * a.row_blocks * 8 && need_bytes > 0, "workspace", a, type);
  }
  if (whole < 100000 || cut < 100000 || refused < 1000) {
    printf("too few: %d whole, %d cut, %d refused\n", whole, cut, refused);
    return 1;
  }
  printf("attend_plan_validate ok: %d whole, %d cut, %d refused\n", whole, cut, refused);
  return 0;
}
