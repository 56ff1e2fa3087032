// How an attention call is cut into workgroups: sizes of the launches and of the workspace, from the call's sizes alone.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "attend.hpp"

namespace seed {

namespace {

using plan::kMany;
using plan::kShared;
using plan::kWaves;

// Workgroups of a call that share its keys: two for each compute unit, as many as their registers and LDS admit. 6 tokens
// of 48 requests 78 us, 85 with half as many and 91 with twice (before changes of rows were counted, now 67); 16 requests
// of 4096 keys 31, 33 and 33; one of 131072 keys 93, 92 and 94; each more part of a row is another one to write and to
// join.
constexpr int64_t kGroups = 512;

}  // namespace

bool plan_attend(int32_t io_dtype, AttendArgs& a) {
  const int64_t rows = static_cast<int64_t>(a.max_tokens) * a.share, tile = io_dtype == SEED_BF16 ? 32 : 16;
  const int64_t row_bytes = static_cast<int64_t>(a.c.dim) * (io_dtype == SEED_BF16 ? 2 : 4);
  // Up to 16 rows are one matrix tile's, and the wavefronts take keys of their own: against shared tiles, 16 requests
  // of 4096 keys of 128 values 31 us from 34, 64 of 3000 keys of 64 values 23 from 33, 32 of 5000 in fp32 97 from 121. Not
  // fp32 of 256 values, which a wavefront has no registers for: 8 requests of 20000 keys 75 from 96 with shared
  // tiles; nor are those faster in one launch (120 keys: 13 us from 17). Up to 32 rows: two wavefronts for each half of
  // a tile that has two products' keys (48 requests, 32 rows: fp32 240 from 353, 64 values 136 from 177; 128 values
  // the same within 4 %).
  const bool wide = row_bytes > 512;
  const int64_t shared = kShared / row_bytes;  // keys of a tile that wavefronts share
  a.row_waves = rows <= 16 && !wide ? 1 : rows <= 32 && shared >= 2 * tile ? 2 : kWaves;
  a.block_rows = static_cast<int32_t>(std::min(rows, int64_t{16} * a.row_waves));
  a.row_blocks = static_cast<int32_t>((rows + a.block_rows - 1) / a.block_rows);
  const int64_t step = a.row_waves == 1 ? tile * kWaves : shared;  // keys of one turn of a workgroup
  int64_t span = a.capacity;
  if (a.window > 0) span = std::min(span, static_cast<int64_t>(a.window) + a.max_tokens - 1 + 31);
  // A change of rows (results written, the next queries, pages and first tile) counts as turns too, or the workgroups that
  // have one end last: 6 tokens of 48 requests 69 us from 73 (1: 72, 2: 70, 4: 69), 32 rows of fp32 116 from 118 (4:
  // 120). Own keys, whose turns are longer: 200 requests of 1500 keys 96.5 from 98 (3: 101), 64 of 16384 the same.
  a.change = a.row_waves == 1 ? 1 : 3;
  const int64_t turns = static_cast<int64_t>(a.c.batch) * a.row_blocks * ((span + step - 1) / step + a.change);  // at most, of a key head
  if (turns >= int64_t{1} << 30) return false;
  // Short spans in one launch, a workgroup each, of 4 wavefronts where those hold them in one turn (256 requests of 100
  // keys 18 us, of 8 wavefronts 34; one request the same). One request of 300 keys: 7.4 us from 11.4 with shares and a join;
  // 64 requests of 1000 keys: 30 both; of 2000: 56 from 49 the other way. Wavefronts that share a tile take the keys one tile
  // after another: few are as fast where the units leave compute units idle, and more the more units there are, whose
  // requests the shares cut and join. 6 tokens of one request, 8 key heads: 250 keys (4 turns) 10.3 us, cut 12.1, 500 keys
  // 15.6 and 12.4; of 64 requests: 1000 keys 31, cut 39, 2000 keys (31 turns) 64 and 60; of 256: 2000 keys 175, cut
  // 198. fp32, whose products take longer: of 64 requests 500 keys (16 turns) 47, cut 52, 1000 keys 77 and 71.
  const int64_t units = static_cast<int64_t>(a.c.batch) * a.c.key_heads * a.row_blocks, per_turn = io_dtype == SEED_BF16 ? 16 : 32;
  const int64_t few = wide               ? 0
                      : a.row_waves == 1 ? std::min(4 * tile * kMany, (int64_t{256} << 10) / row_bytes)
                                         : std::min(std::max(units / per_turn, int64_t{4}), int64_t{64}) * step;
  a.groups = 0;
  a.few = span <= kWaves * tile;  // one turn of 4 wavefronts
  if (span <= few) return units <= most_blocks(64 * (a.row_waves == 1 && !a.few ? kMany : kWaves));
  a.groups = static_cast<int32_t>(std::max(std::min((kGroups + a.c.key_heads - 1) / a.c.key_heads, turns), int64_t{1}));
  return true;
}

int64_t attend_places(const AttendArgs& a) { return a.groups > 1 ? static_cast<int64_t>(a.groups) * a.c.key_heads * 2 * a.block_rows : 0; }

int64_t attend_workspace(const AttendArgs& a) {
  if (a.groups == 0) return 0;
  const int64_t places = attend_places(a);
  return places * (a.c.dim + 2) * 4 + static_cast<int64_t>(a.c.batch) * a.row_blocks * 8;
}

}  // namespace seed
