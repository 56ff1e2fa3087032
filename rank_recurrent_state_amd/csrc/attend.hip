// Attention of a request's newest tokens over its paged cache:
//   o = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q . k_j),
// in one pass over the keys with a running maximum m and sum l: weights are 2^(scale log2(e) q.k - m), and where
// m grows, what was summed so far is multiplied by 2^(m_old - m_new).
//
// What bounds it: every key and value is read once for all rows that share it, so HBM. The rows, queries of one key
// head of all the request's new tokens, are taken 16 at a time by a wavefront, over 32 keys (fp32: 16):
//   S^T = K Q^T   a lane has row lane % 16 and keys 4 (lane / 16) + r of each 16,
//   O^T = V^T P^T takes the weights as they lie: the order of keys inside a product is free, so V's rows are
//                 read in the order in which the lanes hold the weights, whole rows of V by 16 lanes, and its
//                 16-bit values are paired by key with byte permutes.
// Keys are loaded as whole rows and pass through LDS to where the product takes them. Up to 16 rows: every wavefront
// has keys of its own, and its values go straight to registers; the wavefronts are joined at the end. More: 4
// wavefronts share tiles of 16 KB of keys and as many of values, each loading a quarter of the next, for 4 row blocks or
// for 2 by halves of the tile. The keys of all requests are cut into equal shares for two workgroups per compute
// unit, whose partial results a second launch joins; short ones stay whole and need no second launch.
// Measured: 64 requests of up to 16384 tokens, 8 key heads of 128, 1.75 GB: 286 us, 6.1 TB/s (the kernel alone 6.2; a
// kernel that only reads such pages 6.5 - 6.7); one request of 131072 tokens 92 us, 5.8 TB/s; 6 tokens of 48 requests
// (48 rows of a key head of 256), 298 MB: 66 us, 4.5 TB/s, of which the join takes 8 and the first tiles' way 6; the loop
// between reads 7.
// bf16 weights enter as two pieces (p and p - bf16(p)), so that o is off by its own rounding only: with one
// piece the weights' rounding, 2^-9 each, is as large as o's. The products are far from the matrix unit's rate.
// m is only moved when a score passes it by 8 (weights up to 2^8): most tiles then need no exchange between
// lanes and no rescaling, and every weight keeps its relative precision.
#include <algorithm>
#include <type_traits>

#include "attend.hpp"
#include "common.hpp"

namespace seed {

namespace {

using plan::kMany;
using plan::kShared;
using plan::kWaves;

// Turns of a workgroup: equal shares of them all.
__device__ __forceinline__ int share_of(int turns, int groups) {
  return max((turns + groups - 1) / groups, 1);
}
constexpr float kNegInf = -__builtin_inff();

using f32x4 = __attribute__((ext_vector_type(4))) float;
using u32x4 = __attribute__((ext_vector_type(4))) uint32_t;
using u32x2 = __attribute__((ext_vector_type(2))) uint32_t;
using bf16x8 = __attribute__((ext_vector_type(8))) __bf16;
using global_char = __attribute__((address_space(1))) char;
using scalar_int = __attribute__((address_space(4))) int32_t;  // read by scalar loads, which vector loads do not wait for

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// Keeps an address that is the same for the whole wavefront in scalar registers.
__device__ __forceinline__ const global_char* scalar(const char* p) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a)), hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(a >> 32));
  return reinterpret_cast<const global_char*>(static_cast<uint64_t>(hi) << 32 | lo);
}
template <typename T>
__device__ __forceinline__ T load(const global_char* p) {
  return __builtin_nontemporal_load(reinterpret_cast<const __attribute__((address_space(1))) T*>(p));
}

// Maximum / sum over the four lanes that share lane % 16.
__device__ __forceinline__ float max4(float v) {
  float x = v, y = v;
  lane_swap16(x, y);
  v = fmaxf(x, y);
  x = v;
  y = v;
  lane_swap32(x, y);
  return fmaxf(x, y);
}
__device__ __forceinline__ float sum4(float v) {
  float x = v, y = v;
  lane_swap16(x, y);
  v = x + y;
  x = v;
  y = v;
  lane_swap32(x, y);
  return x + y;
}

// The largest magnitudes of two words' values (of both halves side by side for 16-bit values), whether one is
// an infinity or NaN, and a word with those set to 0.
template <int DT>
__device__ __forceinline__ uint32_t largest(uint32_t a, uint32_t b) {
  using u16x2 = __attribute__((ext_vector_type(2))) uint16_t;
  if constexpr (DT == 0) return max(a, b & 0x7fffffffu);
  else
    return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b & 0x7fff7fffu)));
}
template <int DT>
__device__ __forceinline__ bool not_finite(uint32_t w) {
  if constexpr (DT == 0) return (w & 0x7f800000u) == 0x7f800000u;
  else return (w & 0x7f800000u) == 0x7f800000u || (w & 0x7f80u) == 0x7f80u;
}
template <int DT>
__device__ __forceinline__ uint32_t finite_only(uint32_t w) {
  if constexpr (DT == 0) return (w & 0x7f800000u) == 0x7f800000u ? 0u : w;
  else return ((w & 0x7f800000u) == 0x7f800000u ? 0u : w & 0xffff0000u) | ((w & 0x7f80u) == 0x7f80u ? 0u : w & 0xffffu);
}

// log of sum 2^max.
__device__ __forceinline__ float natural_log_sum(float max, float sum) {
  constexpr float kLn2 = 0.693147181f;
  return sum == 0.f ? kNegInf : fmaf(max, kLn2, __builtin_amdgcn_logf(sum) * kLn2);
}

// The token of row r: r / share, exact for the shares that the host admits (up to 2^14, r below 32 share).
__device__ __forceinline__ int token_of(const AttendArgs& A, int r) { return static_cast<int>((static_cast<float>(r) + 0.5f) * A.per_share); }

// The positions that the rows of a request see between them: keys [k0, k1), row i at first + i.
struct Span {
  int64_t lo;
  int n, first, k0, k1, base;  // base: k0 at a tile's start
  // turns of `step` keys; a request with rows has one, if only to write their zeros
  __device__ __forceinline__ int turns(int step) const { return n == 0 ? 0 : k1 > k0 ? (k1 - base + step - 1) / step : 1; }
};
__device__ __forceinline__ Span span_of(const AttendArgs& A, int b) {
  Span s;
  int64_t hi;
  request_rows(A.c, b, s.lo, hi);
  const int64_t n = hi - s.lo;
  s.n = static_cast<int>(n < A.max_tokens ? n : A.max_tokens);
  const int64_t length = min(max(A.c.lengths[b], 0), A.capacity), first = length - n;
  const int64_t k1 = max(first + s.n, int64_t{0});
  const int64_t k0 = A.window > 0 ? max(first - A.window + 1, int64_t{0}) : 0;
  s.first = static_cast<int>(max(first, int64_t{-64}));  // a row below position 0 sees nothing: how far does not matter
  s.k1 = static_cast<int>(k1);
  s.k0 = static_cast<int>(min(k0, k1));
  s.base = s.k0 & ~31;
  return s;
}

// Sum of the lanes up to each, and of all.
__device__ __forceinline__ int scan(int v, int lane, int& total) {
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const int up = __shfl_up(v, d, kWave);
    if (lane >= d) v += up;
  }
  total = __builtin_amdgcn_readlane(v, kWave - 1);
  return v;
}

// Keys and values of a turn: a wavefront's own ones (RW = 1), or a tile of RW row blocks.
template <int DT, int D, int RW>
struct Tile {
  static constexpr int kBytes = DT == 0 ? 4 : 2;
  static constexpr int kVec = 16 / kBytes;            // values of a 16-byte access
  static constexpr int kGroup = DT == 0 ? 1 : 2;      // 16-key parts whose values enter a product together
  static constexpr int kSub = RW == 1 ? kGroup : kShared / (16 * D * kBytes);  // 16-key parts of a tile
  static constexpr int kKeys = 16 * kSub;
  static constexpr int kQ = D / (4 * kVec);           // 16-byte pieces of a row per lane
  static constexpr int VE = D / 16 < kVec ? D / 16 : kVec;  // values of V per lane and access
  static constexpr int VC = D / (16 * VE);
  static constexpr int kOut = D / 16;                 // accumulators of 16 rows: value 16 VE c + VE m + j in number VE c + j
  static constexpr int kWords = VE * kBytes / 4;
  static constexpr int kRow = D * kBytes;             // bytes of a key
  static constexpr int kLine = kRow / 16;             // lanes that load a row of 16 bytes each,
  static constexpr int kAtOnce = kWave / kLine;       // and rows of one load
  static constexpr int kTile = kKeys * kRow;
  // LDS holds 16-byte piece c of key r at r kRow + 16 (c ^ swap(r)): pieces trade places so that 16 rows' pieces of one
  // number lie in different banks. swap(r + s) = swap(r) ^ swap(s) where r is a multiple of kAtOnce and s below it,
  // or r of 16: a place is one exclusive or away from a lane's first.
  static __device__ __forceinline__ constexpr uint32_t swap(int r) { return kLine == 8 ? (r >> 1) & 7 : r & 15; }
};

}  // namespace

// A workgroup's shared memory.
template <int DT, int D, int RW, int NW>
struct Shared {
  using L = Tile<DT, D, RW>;
  static constexpr int GT = L::kOut < 8 ? L::kOut : 8;  // accumulators joined at a time
  // A wavefront's keys (RW = 1), or all wavefronts' keys and values, twice; at the end the accumulators.
  static constexpr int kJoin = NW * GT * kWave * 16, kTiles = RW == 1 ? NW * L::kTile : 4 * L::kTile;
  __attribute__((aligned(16))) char tiles[kJoin > kTiles ? kJoin : kTiles];
  // 16-bit queries of 256 values (RW = 1): in registers they leave too few for the loads
  static constexpr bool kQueries = DT != 0 && D == 256 && RW == 1;
  u32x4 q[kQueries ? L::kQ : 1][kQueries ? kWave : 1];
  // RW > 1: what a wavefront found in its rows of a tile: 1: a value that is an infinity or NaN, 2: a page that is not there
  __attribute__((aligned(16))) int found[2][NW];
  float weights[RW == 1 ? 1 : NW][RW == 1 ? 1 : L::kGroup * 256];  // RW = 1: in the place of a wavefront's keys
  float stat[NW][16][2];
};

// Rows [16 RW rb, ..) of request b and key head kh over the keys [from, to): written to o, or as maximum, sum and
// accumulators of each row to stat and part (nullptr: o). NW wavefronts: RW = 1: of the same 16 rows and keys of
// their own each; else RW of 16 rows each by NW / RW parts of the tiles that they share.
template <int DT, int D, int RW, int NW>
__device__ __forceinline__ void attend_keys(const AttendArgs& A, Shared<DT, D, RW, NW>& sm, const Span& sp, int b, int kh, int rb, int from,
                                            int to, float* part, float* part_stat) {
  using L = Tile<DT, D, RW>;
  using T = stor_t<DT>;
  constexpr int KW = NW / RW, GT = Shared<DT, D, RW, NW>::GT;
  constexpr int kParts = RW == 1 ? L::kSub : L::kSub / KW;  // of 16 keys, that a wavefront takes of a tile
  static_assert(kParts % L::kGroup == 0 && (RW == 1 || KW <= 2), "whole products; a part of a tile is one of two");
  const CacheArgs& C = A.c;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const int share = A.share;
  const int rows = sp.n * share, block0 = rb * RW * 16;

  // this lane's row of the wavefront's 16: a query of key head kh
  const int row0 = block0 + 16 * (wave % RW), half = RW == 1 || KW == 1 ? 0 : wave / RW;
  const int r = row0 + l16, token = token_of(A, r);
  const int pos = r < rows ? sp.first + token : -1;
  u32x4 Q[L::kQ];
#pragma unroll
  for (int c = 0; c < L::kQ; ++c) Q[c] = u32x4{0, 0, 0, 0};
  if (r < rows) {
    const T* q = static_cast<const T*>(A.q) + (sp.lo + token) * A.q_stride + static_cast<int64_t>(kh * share + r - token * share) * D;
#pragma unroll
    for (int c = 0; c < L::kQ; ++c) Q[c] = *reinterpret_cast<const u32x4*>(q + c * 4 * L::kVec + g * L::kVec);
  }
#pragma unroll
  for (int c = 0; c < L::kQ; ++c) Q[c] ^= A.negate;
  constexpr bool kQueries = Shared<DT, D, RW, NW>::kQueries;
  if constexpr (kQueries) {
    if (wave == 0) {
#pragma unroll
      for (int c = 0; c < L::kQ; ++c) sm.q[c][lane] = Q[c];
    }
    __syncthreads();
  }

  f32x4 O[L::kOut];
  float m = kNegInf, l = 0.f;
#pragma unroll
  for (int j = 0; j < L::kOut; ++j) O[j] = f32x4{0.f, 0.f, 0.f, 0.f};

  const int last_pos = sp.first + sp.n - 1;
  const scalar_int* table = reinterpret_cast<const scalar_int*>(reinterpret_cast<uintptr_t>(C.table + static_cast<int64_t>(b) * C.width));
  // a lane's place within 16 positions, in bytes; the positions' page is the same for the whole wavefront
  const char* __restrict__ kb = reinterpret_cast<const char*>(static_cast<const T*>(C.k) + kh * C.head_stride);
  const char* __restrict__ vb = reinterpret_cast<const char*>(static_cast<const T*>(C.v) + kh * C.head_stride);
  const int64_t ts = C.token_stride * L::kBytes, page_stride = C.page_stride * L::kBytes;
  const uint32_t in_v = static_cast<uint32_t>(4 * g * ts) + l16 * L::VE * L::kBytes;
  const int in_page = (1 << C.page_shift) - 1;

  // The places of the 16-key parts of the rows that this wavefront loads, of all of its own tile (RW = 1) or some
  // of the shared one's: 16 positions lie in one page; parts behind this workgroup's last read that again.
  constexpr int kLoaders = RW == 1 ? 1 : NW, kRows = L::kKeys / kLoaders, kMine = kRows < 16 ? 1 : kRows / 16;
  const int mine = RW == 1 ? 0 : wave * kRows;  // the first of these rows
  struct Where {
    int64_t at[kMine];
    bool there[kMine];
  };
  struct Pages {
    int number[kMine];
  };
  auto part_at = [&](int key) { return min(key, (to - 1) & ~15); };
  auto page_of = [&](int key) { return table[part_at(key) >> C.page_shift]; };
  auto look_up = [&](int t0) {
    Pages p;
#pragma unroll
    for (int u = 0; u < kMine; ++u) p.number[u] = page_of(t0 + (mine & ~15) + 16 * u);
    return p;
  };
  auto find = [&](int t0, const Pages& p) {
    Where w;
#pragma unroll
    for (int u = 0; u < kMine; ++u) {
      w.there[u] = static_cast<uint32_t>(p.number[u]) < A.pages;
      w.at[u] = static_cast<int64_t>(w.there[u] ? p.number[u] : 0) * page_stride +
                ((part_at(t0 + (mine & ~15) + 16 * u) & in_page) + mine % 16) * ts;
    }
    return w;
  };
  // Whole rows per load, 16 bytes per lane: 6.6 TB/s of keys and values, 5.7 with the 64 bytes of 16 rows that the
  // products take; and past the caches, which keep nothing of a cache read once a step (5.9 with them).
  constexpr int kLoads = kRows / L::kAtOnce;
  const int my_row = lane / L::kLine, my_piece = lane % L::kLine;
  const uint32_t in_row = static_cast<uint32_t>(my_row * ts) + my_piece * 16;
  u32x4 K[kLoads], Vr[kLoads];
  auto load_rows = [&](const char* pool, const Where& w, uint32_t in_row, u32x4 (&x)[kLoads]) {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) x[i] = load<u32x4>(scalar(pool + w.at[i * L::kAtOnce / 16] + i * L::kAtOnce % 16 * ts) + in_row);
  };
  uint32_t V[RW == 1 ? L::VC : 1][4 * L::kSub][L::kWords];
  // RW = 1: values straight to where the products take them
  auto load_v = [&](const Where& w) {
#pragma unroll
    for (int i = 0; i < 4 * L::kSub; ++i) {
      const global_char* base = scalar(vb + w.at[i / 4] + i % 4 * ts);
#pragma unroll
      for (int c = 0; c < L::VC; ++c) {
        const global_char* p = base + in_v + c * 16 * L::VE * L::kBytes;
        if constexpr (L::kWords == 4) {
          const u32x4 x = load<u32x4>(p);
#pragma unroll
          for (int e = 0; e < 4; ++e) V[c][i][e] = x[e];
        } else {
          const u32x2 x = load<u32x2>(p);
          V[c][i][0] = x[0];
          V[c][i][1] = x[1];
        }
      }
    }
  };

  // Keys are loaded a tile ahead, as soon as the last ones are in LDS, values while the scores are formed (RW > 1:
  // a tile ahead too): something is always on its way.
  constexpr int kTurn = (RW == 1 ? NW : 1) * L::kKeys;
  Where here{};
  const int start = from + (RW == 1 ? wave * L::kKeys : 0);
  const bool any = RW == 1 ? start < to : from < to;  // a tile for this wavefront (256 requests of 100 keys: 18 us, with loads for all 20)
  if (any) {
    here = find(start, look_up(start));
    load_rows(kb, here, in_row, K);
    if constexpr (RW > 1) load_rows(vb, here, in_row, Vr);
  }
  const uint32_t write_at = (mine + my_row) * L::kRow + ((my_piece ^ L::swap(mine) ^ L::swap(my_row)) << 4), read_at = l16 * L::kRow + ((g ^ L::swap(l16)) << 4);
  Pages ahead{};  // of the next turn: looked up a turn ahead too
  if (any) ahead = look_up(start + kTurn);
  int turn = 0;
  for (int t0 = start; t0 < to; t0 += kTurn) {
    char* keys = sm.tiles + (RW == 1 ? wave * L::kTile : turn * 2 * L::kTile);
    if constexpr (RW == 1) load_v(here);
    __builtin_amdgcn_sched_barrier(0);
    // Values that no row sees become 0: a weight of 0 does not keep an infinity or NaN out of a product.
    bool gap = false;
#pragma unroll
    for (int u = 0; u < kMine; ++u) gap = gap || !here.there[u];
    const bool outside = t0 < sp.k0 || t0 + L::kKeys > sp.k1 || gap;
    if constexpr (RW > 1) {
      if (outside) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
          const int key = t0 + mine + i * L::kAtOnce + my_row;
          const bool seen = here.there[i * L::kAtOnce / 16] && key >= sp.k0 && key < sp.k1;
#pragma unroll
          for (int e = 0; e < 4; ++e) Vr[i][e] = seen ? Vr[i][e] : 0u;
        }
      }
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < kLoads; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) most = largest<DT>(most, Vr[i][e]);
      const int odd = __any(not_finite<DT>(most)) ? 1 : 0;
      if (lane == 0) sm.found[turn][wave] = odd | (gap ? 2 : 0);
    }
    uint32_t write = write_at, read = read_at;  // the places follow from these, and need no registers between turns
    asm volatile("" : "+v"(write), "+v"(read));
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      constexpr int kStep = L::kAtOnce * L::kRow;
      *reinterpret_cast<u32x4*>(keys + i * kStep + (write ^ (L::swap(i * L::kAtOnce) << 4))) = K[i];
      if constexpr (RW > 1) *reinterpret_cast<u32x4*>(keys + L::kTile + i * kStep + (mine + my_row) * L::kRow + my_piece * 16) = Vr[i];
    }
    const Where next = find(t0 + kTurn, ahead);
    ahead = look_up(t0 + 2 * kTurn);
    // behind the last tile one piece of its rows, for all lanes: the loads on their way are then the same in number
    // (256 requests of 700 keys 69 us, with the whole tile again 73)
    const uint32_t in_next = t0 + kTurn < to ? in_row : 0;
    load_rows(kb, next, in_next, K);
    if constexpr (RW > 1) {
      load_rows(vb, next, in_next, Vr);
      // the tile is whole; the other one is free once every wavefront is past this point in the next turn
      __syncthreads();
      turn ^= 1;
      if (row0 >= rows) {  // a wavefront that only loads
        here = next;
        continue;
      }
    } else {
      wave_lds_sync();
    }

    // this wavefront's part of the tile
    const int first = t0 + half * 16 * kParts;
    const char* my_keys = keys + half * 16 * kParts * L::kRow;
    bool odd = false;
    if constexpr (RW > 1) {
      int found = 0;
#pragma unroll
      for (int w = 0; w < NW; ++w) found |= sm.found[turn ^ 1][w];
      found = __builtin_amdgcn_readfirstlane(found);
      odd = (found & 1) != 0;
      gap = found >= 2;
    }
    f32x4 S[kParts];
#pragma unroll
    for (int u = 0; u < kParts; ++u) S[u] = f32x4{0.f, 0.f, 0.f, 0.f};
    // Pieces of the keys in runs, one read while the products take the one before, where there are registers for them (fp32
    // and 16-bit heads of 256, and a wavefront's own values, leave none: the order is the compiler's).
    constexpr bool kOrder = RW > 1 && L::kOut <= 8;
    constexpr int kMost = kOrder ? 8 : kParts, kRun = L::kQ * kParts < kMost ? L::kQ * kParts : kMost, kRuns = L::kQ * kParts / kRun;
    u32x4 piece[2][kRun];
    auto read_run = [&](int n) {
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        const int c = (n * kRun + i) / kParts, u = (n * kRun + i) % kParts;
        piece[n % 2][i] = *reinterpret_cast<const u32x4*>(my_keys + 16 * u * L::kRow + (read ^ (c << 6)));
      }
    };
    read_run(0);
#pragma unroll
    for (int n = 0; n < kRuns; ++n) {
      if (n + 1 < kRuns) read_run(n + 1);
      if constexpr (kOrder) __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < kRun; ++i) {
        const int c = (n * kRun + i) / kParts, u = (n * kRun + i) % kParts;
        const u32x4 q = kQueries ? sm.q[kQueries ? c : 0][kQueries ? lane : 0] : Q[c], k = piece[n % 2][i];
        if constexpr (DT == 0) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            S[u] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(k[e]), __uint_as_float(q[e]), S[u], 0, 0, 0);
        } else {
          S[u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, k), __builtin_bit_cast(bf16x8, q), S[u], 0, 0, 0);
        }
      }
      if constexpr (kOrder) __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (RW == 1) wave_lds_sync();  // the next tile's keys go to the same place

    // some row does not see some position of the tile
    if (gap || t0 < sp.k0 || t0 + L::kKeys > sp.first + 1 || (A.window > 0 && t0 <= last_pos - A.window)) {
#pragma unroll
      for (int u = 0; u < kParts; ++u) {
        const bool there = !gap || static_cast<uint32_t>(page_of(first + 16 * u)) < A.pages;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int key = first + 16 * u + 4 * g + i;
          const bool seen = there && key <= pos && (A.window <= 0 || key > pos - A.window);
          S[u][i] = seen ? S[u][i] : kNegInf;
        }
      }
    }
    float top = kNegInf;
#pragma unroll
    for (int i = 0; i < 4 * kParts; ++i) top = fmaxf(top, S[i / 4][i % 4]);
    top *= A.scale2;
    if (__any(top > m + 8.f)) {
      const float now = fmaxf(m, max4(top));
      // nothing summed so far, or all of it of weight 0: 2^(-inf)
      const float f = now == kNegInf ? 1.f : exp2_(m - now);
      m = now;
      l *= f;
#pragma unroll
      for (int j = 0; j < L::kOut; ++j) O[j] *= f;
    }
    const float sub = m == kNegInf ? 0.f : m;
    float P[4 * kParts];
#pragma unroll
    for (int i = 0; i < 4 * kParts; ++i) {
      P[i] = exp2_(fmaf(S[i / 4][i % 4], A.scale2, -sub));
      l += P[i];
    }
    if constexpr (RW == 1) {
      if (outside) {
#pragma unroll
        for (int i = 0; i < 4 * L::kSub; ++i) {
          const int key = t0 + 16 * (i / 4) + 4 * g + i % 4;
          const bool seen = here.there[i / 4] && key >= sp.k0 && key < sp.k1;
#pragma unroll
          for (int c = 0; c < L::VC; ++c)
#pragma unroll
            for (int e = 0; e < L::kWords; ++e) V[c][i][e] = seen ? V[c][i][e] : 0u;
        }
      }
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < 4 * L::kSub; ++i)
#pragma unroll
        for (int c = 0; c < L::VC; ++c)
#pragma unroll
          for (int e = 0; e < L::kWords; ++e) most = largest<DT>(most, V[c][i][e]);
      odd = __any(not_finite<DT>(most));
    }
    // Neither does a second piece of 0, or the weight of a row that does not see them, keep out those that
    // are left: they are added one by one, and the products get 0 in their place.
    float* weights = RW == 1 ? reinterpret_cast<float*>(keys) : sm.weights[RW == 1 ? 0 : wave];  // [key][row]
    auto values = [&](auto is_odd) {
#pragma unroll
      for (int p0 = 0; p0 < kParts; p0 += L::kGroup) {
        constexpr int N = 4 * L::kGroup;  // a lane's weights of a product
        const float(&W)[N] = *reinterpret_cast<const float(*)[N]>(P + 4 * p0);
        u32x4 hi, lo;
        if constexpr (DT != 0) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            hi[i] = pack2<1>(W[2 * i], W[2 * i + 1]);
            lo[i] = pack2<1>(W[2 * i] - lo16<1>(hi[i]), W[2 * i + 1] - hi16<1>(hi[i]));
          }
        }
        auto product = [&](const uint32_t (&v)[N][L::kWords], int j, f32x4 z) {
          if constexpr (DT == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) z = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(v[i][j]), W[i], z, 0, 0, 0);
          } else {
            u32x4 a;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              a[i] = __builtin_amdgcn_perm(v[2 * i + 1][j / 2], v[2 * i][j / 2], j % 2 == 0 ? 0x05040100u : 0x07060302u);
            z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, hi), z, 0, 0, 0);
            z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, lo), z, 0, 0, 0);
          }
          return z;
        };
        if (__builtin_expect(is_odd, 0)) {
          wave_lds_sync();
#pragma unroll
          for (int i = 0; i < N; ++i) weights[(16 * (i / 4) + 4 * g + i % 4) * 16 + l16] = W[i];
          wave_lds_sync();
        }
#pragma unroll
        for (int c = 0; c < L::VC; ++c) {
          uint32_t v[N][L::kWords];
#pragma unroll
          for (int i = 0; i < N; ++i)
#pragma unroll
            for (int e = 0; e < L::kWords; ++e) {
              if constexpr (RW == 1)
                v[i][e] = V[c][i][e];
              else
                v[i][e] = reinterpret_cast<const uint32_t*>(my_keys + L::kTile + (16 * (p0 + i / 4) + 4 * g + i % 4) * L::kRow +
                                                            (c * 16 + l16) * L::VE * L::kBytes)[e];
            }
          if (__builtin_expect(is_odd, 0)) {
#pragma unroll
            for (int i = 0; i < N; ++i)
#pragma unroll
              for (int e = 0; e < L::kWords; ++e) v[i][e] = finite_only<DT>(v[i][e]);
          }
#pragma unroll
          for (int j = 0; j < L::VE; ++j) O[c * L::VE + j] = product(v, j, O[c * L::VE + j]);
        }
        if (__builtin_expect(is_odd, 0)) {
#pragma unroll 1
          for (int k = 0; k < 16 * L::kGroup; ++k) {
            const int key = first + 16 * p0 + k;
            // the page looked up again: a run-time index into here would take it out of the registers
            const int at = min(key, ((to - 1) & ~15) + (key & 15)), number = table[at >> C.page_shift];
            const bool seen = static_cast<uint32_t>(number) < A.pages && key <= pos && (A.window <= 0 || key > pos - A.window);
            if (!seen) continue;
            const float p = weights[k * 16 + l16];
            const char* base = vb + static_cast<int64_t>(number) * page_stride + (at & in_page) * ts;
#pragma unroll
            for (int c = 0; c < L::VC; ++c)
#pragma unroll
              for (int e = 0; e < 4; ++e) {  // this lane's values of the row: 4 runs of VE
                const T* v = reinterpret_cast<const T*>(base) + c * 16 * L::VE + (4 * g + e) * L::VE;
#pragma unroll
                for (int j = 0; j < L::VE; ++j) {
                  const float x = to_f32<DT>(v[j]);
                  if (!(fabsf(x) < __builtin_inff())) O[c * L::VE + j][e] += p * x;
                }
                __builtin_amdgcn_sched_barrier(0);
              }
          }
        }
      }
    };
    if constexpr (!kOrder) values(odd);
    else if (__builtin_expect(odd, 0)) values(std::true_type{});
    else values(std::false_type{});
    here = next;
  }

  constexpr bool kOwn = RW == 1 && L::kTile == GT * kWave * 16;  // a wavefront's accumulators take the place of its own tile
  // Join the wavefronts of the same rows: sums and accumulators brought to the largest maximum. The tiles' place
  // takes the accumulators, a few at a time.
  f32x4(*red)[GT][kWave] = reinterpret_cast<f32x4(*)[GT][kWave]>(sm.tiles);
  l = sum4(l);
  if (g == 0) {
    sm.stat[wave][l16][0] = m;
    sm.stat[wave][l16][1] = l;
  }
  const int tid = threadIdx.x & 255, orow = tid & 15, om = tid >> 4;  // the row of each 16 and the 16th of its values that this thread writes
  const int part_of = threadIdx.x >> 8;                               // NW = 8: which of the accumulators
#pragma unroll
  for (int j0 = 0; j0 < L::kOut; j0 += GT) {
    if (!kOwn || j0 > 0) __syncthreads();  // the last tile, or what was joined before, has been read
#pragma unroll
    for (int j = 0; j < GT; ++j) red[wave][j][lane] = O[j0 + j];
    __syncthreads();
#pragma unroll
    for (int w = 0; w < RW; ++w) {
      const int out = block0 + 16 * w + orow;
      if (out >= rows) continue;
      float top = kNegInf, sum = 0.f, f[KW];
#pragma unroll
      for (int k = 0; k < KW; ++k) top = fmaxf(top, sm.stat[w + RW * k][orow][0]);
#pragma unroll
      for (int k = 0; k < KW; ++k) {
        const float mw = sm.stat[w + RW * k][orow][0];
        f[k] = mw == kNegInf ? 1.f : exp2_(mw - top);  // without a weight: zeros, or NaN
        sum += sm.stat[w + RW * k][orow][1] * f[k];
      }
      const int ot = token_of(A, out), head = kh * share + out - ot * share;
      const int64_t line = (sp.lo + ot) * C.heads + head;
      if (om == 0 && part_of == 0 && j0 == 0) {
        if (part != nullptr) {
          part_stat[2 * (out - block0)] = top;
          part_stat[2 * (out - block0) + 1] = sum;
        } else if (A.lse != nullptr) {
          A.lse[line] = natural_log_sum(top, sum);
        }
      }
      constexpr int kRun = L::VE, kRuns = GT / kRun;  // neighbouring values of a thread
#pragma unroll
      for (int c = 0; c < kRuns; ++c) {
        if (NW > kWaves && c % 2 != part_of && kRuns > 1) continue;
        if (NW > kWaves && kRuns == 1 && part_of != 0) continue;
        float y[kRun];
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
          y[j] = 0.f;
#pragma unroll
          for (int k = 0; k < KW; ++k)
            y[j] = fmaf(reinterpret_cast<const float*>(&red[w + RW * k][c * kRun + j][(om >> 2) * 16 + orow])[om & 3], f[k], y[j]);
        }
        const int v = (j0 / kRun + c) * 16 * kRun + om * kRun;
        if (part != nullptr) {
          store_f32<0, kRun>(part + static_cast<int64_t>(out - block0) * D + v, y);
        } else {
          const float inv = 1.f / sum;
#pragma unroll
          for (int j = 0; j < kRun; ++j) y[j] = sum == 0.f ? 0.f : y[j] * inv;
          store_f32<DT, kRun>(static_cast<T*>(A.o) + (sp.lo + ot) * A.o_stride + static_cast<int64_t>(head) * D + v, y);
        }
      }
    }
  }
}

// A workgroup per request, key head and row block.
template <int DT, int D, int RW, int NW>
__global__ __launch_bounds__(NW* kWave, 2) void k_attend_whole(const AttendArgs A) {
  __shared__ Shared<DT, D, RW, NW> sm;
  const int kh = static_cast<int>(blockIdx.x % A.c.key_heads), rest = static_cast<int>(blockIdx.x / A.c.key_heads);
  const int b = RW == 1 ? rest : rest / A.row_blocks, rb = RW == 1 ? 0 : rest - b * A.row_blocks;
  const Span sp = span_of(A, b);
  if (16 * RW * rb >= sp.n * A.share) return;
  attend_keys<DT, D, RW, NW>(A, sm, sp, b, kh, rb, sp.base, sp.k1, nullptr, nullptr);
}

// The turns of all requests (of kStep keys, row block after row block, each with `change` turns without keys before it)
// are cut into equal shares, one for each of a key head's workgroups; the requests' lengths are known here only. A
// share that ends inside a row block leaves partial results in the workgroup's second place, one that begins inside in
// its first; the workgroup that begins a row block notes which ones hold it.
template <int DT, int D, int RW>
__global__ __launch_bounds__(kWaves * kWave, 2) void k_attend(const AttendArgs A) {
  __shared__ Shared<DT, D, RW, kWaves> sm;
  constexpr int kStep = Tile<DT, D, RW>::kKeys * (RW == 1 ? kWaves : 1);
  const CacheArgs& C = A.c;
  // neighbouring heads, whose keys lie side by side, run at the same time
  const int kh = static_cast<int>(blockIdx.x % C.key_heads), me = static_cast<int>(blockIdx.x / C.key_heads);
  const int lane = threadIdx.x & 63;
  auto of_block = [&](const Span& sp) { return sp.n > 0 ? sp.turns(kStep) + A.change : 0; };
  auto turns = [&](int i) {
    const Span sp = span_of(A, min(i, C.batch - 1));
    return i < C.batch ? of_block(sp) * ((sp.n * A.share + 16 * RW - 1) / (16 * RW)) : 0;
  };
  // every wavefront for itself: the sum of all turns, then the request in which this share begins. The lengths of up to
  // 256 requests are loaded at once (64 at a time: up to 2 us more for 256 requests; at once for one: 1 us more).
  int share = 0, w0 = 0, w1 = 0, b = -1, begin = 0;  // request, and its first turn
  auto find_share = [&](auto at_once) {
    constexpr int kAt = decltype(at_once)::value;
    int mine[kAt], run[kAt], sums[kAt], loaded = 0, total = 0;
    auto read = [&](int first) {
      loaded = first;
#pragma unroll
      for (int j = 0; j < kAt; ++j) mine[j] = turns(first + j * kWave + lane);
#pragma unroll
      for (int j = 0; j < kAt; ++j) run[j] = scan(mine[j], lane, sums[j]);
    };
    for (int i = 0; i < C.batch; i += kAt * kWave) {
      read(i);
#pragma unroll
      for (int j = 0; j < kAt; ++j) total += sums[j];
    }
    share = share_of(total, A.groups);
    w0 = me * share;
    w1 = min(w0 + share, total);
    if (w0 >= total) return;
    if (loaded != 0) read(0);
    for (;;) {
#pragma unroll
      for (int j = 0; j < kAt; ++j) {
        const uint64_t past = __ballot(begin + run[j] > w0);
        if (b < 0 && past != 0) {
          const int at = __builtin_ctzll(past);
          begin += __builtin_amdgcn_readlane(run[j] - mine[j], at);
          b = loaded + j * kWave + at;
        }
        if (b < 0) begin += sums[j];
      }
      if (b >= 0) break;
      read(loaded + kAt * kWave);
    }
  };
  if (C.batch <= kWave) find_share(std::integral_constant<int, 1>{});
  else find_share(std::integral_constant<int, 4>{});
  if (w0 >= w1) return;
  Span sp = span_of(A, b);
  for (int w = w0; w < w1;) {
    const int each = of_block(sp), blocks = (sp.n * A.share + 16 * RW - 1) / (16 * RW);
    const int rb = RW == 1 ? 0 : (w - begin) / each, t0 = w - begin - rb * each, n = min(each - t0, w1 - w);
    const bool whole = n == each;
    const int64_t place = (static_cast<int64_t>(me) * C.key_heads + kh) * 2 + (t0 == 0 ? 1 : 0);
    if (t0 == 0 && kh == 0 && threadIdx.x == 0) {
      int32_t* note = A.notes + (static_cast<int64_t>(b) * A.row_blocks + rb) * 2;
      note[0] = me;
      note[1] = me + (each - n + share - 1) / share;
    }
    if (w > w0) __syncthreads();  // the last part's results have been read
    const int from = sp.base + max(t0 - A.change, 0) * kStep;
    const int to = static_cast<int>(min(sp.base + static_cast<int64_t>(max(t0 + n - A.change, 0)) * kStep, static_cast<int64_t>(sp.k1)));
    attend_keys<DT, D, RW, kWaves>(A, sm, sp, b, kh, rb, from, to, whole ? nullptr : A.part + place * A.block_rows * D,
                                   A.stat + place * A.block_rows * 2);
    w += n;
    while (w < w1 && w == begin + of_block(sp) * ((sp.n * A.share + 16 * RW - 1) / (16 * RW))) {  // on to the next request with rows
      begin = w;
      sp = span_of(A, ++b);
    }
  }
}

// Joins the parts of the rows that more than one workgroup has: a workgroup per request, row block, key head and
// `each` rows (WR > 1: one), WR wavefronts per row, a lane D / 64 of its values.
template <int DT, int D, int WR>
__global__ __launch_bounds__(WR == 1 ? kWaves * kWave : WR * kWave) void k_attend_join(const AttendArgs A, int each) {
  using T = stor_t<DT>;
  constexpr int N = D / kWave;
  using vec = __attribute__((ext_vector_type(N))) float;
  __shared__ float acc[WR][D];
  __shared__ float stats[WR][2];
  const CacheArgs& C = A.c;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int chunks = (A.block_rows + each - 1) / each;
  const int chunk = static_cast<int>(blockIdx.x % chunks);
  const unsigned rest = blockIdx.x / chunks, block = rest / C.key_heads;
  const int kh = static_cast<int>(rest % C.key_heads), b = static_cast<int>(block / A.row_blocks), rb = static_cast<int>(block % A.row_blocks);
  const int32_t* note = A.notes + static_cast<int64_t>(block) * 2;
  const int first = note[0], parts = note[1] - first + 1;  // loaded beside the offsets; of a request without these rows nothing
  const Span sp = span_of(A, b);
  const int rows = min(sp.n * A.share - rb * A.block_rows, A.block_rows), end = min((chunk + 1) * each, rows);
  if (rows <= 0 || parts == 1) return;
  for (int in_block = chunk * each + (WR == 1 ? wave : 0); in_block < end; in_block += WR == 1 ? kWaves : 1) {
    const int row = rb * A.block_rows + in_block, token = token_of(A, row), head = kh * A.share + row - token * A.share;
    // part 0 in the second place of its workgroup, the others in the first of theirs
    auto place = [&](int s) { return ((static_cast<int64_t>(first + s) * C.key_heads + kh) * 2 + (s == 0 ? 1 : 0)) * A.block_rows + in_block; };
    float top = kNegInf, sum = 0.f, y[N] = {};
    // up to 64 parts at a time, a lane's maximum and sum each; several wavefronts take a run of parts each
    const int per = WR == 1 ? parts : (parts + WR - 1) / WR, s1 = WR == 1 ? parts : min((wave + 1) * per, parts);
    for (int s0 = WR == 1 ? 0 : wave * per; s0 < s1; s0 += kWave) {
      const int s = s0 + lane;
      const float* stat = A.stat + place(s) * 2;
      const float ms = s < s1 ? stat[0] : kNegInf, ls = s < s1 ? stat[1] : 0.f;
      const int n = min(s1 - s0, kWave);
      // The first 4 parts are loaded beside these, the others 16 or 4 at a time, the last one again where there are fewer.
      // Always 4: 397 parts 11.5 us from 9.2; always 16: 6 parts 9.0 from 8.3.
      constexpr int kFirst = 4, kMore = 16;
      auto part = [&](int i) { return *reinterpret_cast<const vec*>(A.part + place(s0 + min(i, n - 1)) * D + lane * N); };
      vec x[kMore];
#pragma unroll
      for (int i = 0; i < kFirst; ++i) x[i] = part(i);
      float now = ms;
#pragma unroll
      for (int d = 1; d < 16; d *= 2) now = fmaxf(now, __shfl_xor(now, d, kWave));
      now = fmaxf(top, max4(now));
      const float old = now == kNegInf ? 1.f : exp2_(top - now);
      top = now;
      const float f = ms == kNegInf ? 1.f : exp2_(ms - now);  // a part without a weight holds zeros, or NaN
      sum = sum * old + wave_sum(ls * f);
#pragma unroll
      for (int e = 0; e < N; ++e) y[e] *= old;
      auto add = [&](int i, const vec& xi) {
        const float fi = i < n ? __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, f), min(i, n - 1))) : 0.f;
#pragma unroll
        for (int e = 0; e < N; ++e) y[e] = i < n ? fmaf(xi[e], fi, y[e]) : y[e];
      };
#pragma unroll
      for (int i = 0; i < kFirst; ++i) add(i, x[i]);
      int i0 = kFirst;
      for (; i0 + kMore / 2 < n; i0 += kMore) {
#pragma unroll
        for (int i = 0; i < kMore; ++i) x[i] = part(i0 + i);
#pragma unroll
        for (int i = 0; i < kMore; ++i) add(i0 + i, x[i]);
      }
      for (; i0 < n; i0 += kFirst) {
#pragma unroll
        for (int i = 0; i < kFirst; ++i) x[i] = part(i0 + i);
#pragma unroll
        for (int i = 0; i < kFirst; ++i) add(i0 + i, x[i]);
      }
    }
    if constexpr (WR > 1) {
#pragma unroll
      for (int e = 0; e < N; ++e) acc[wave][lane * N + e] = y[e];
      if (lane == 0) {
        stats[wave][0] = top;
        stats[wave][1] = sum;
      }
      __syncthreads();
      if (wave != 0) return;  // one row
      float most = kNegInf;
#pragma unroll
      for (int w = 0; w < WR; ++w) most = fmaxf(most, stats[w][0]);
      sum = 0.f;
#pragma unroll
      for (int e = 0; e < N; ++e) y[e] = 0.f;
#pragma unroll
      for (int w = 0; w < WR; ++w) {
        const float f = stats[w][0] == kNegInf ? 1.f : exp2_(stats[w][0] - most);
        sum += stats[w][1] * f;
#pragma unroll
        for (int e = 0; e < N; ++e) y[e] = fmaf(acc[w][lane * N + e], f, y[e]);
      }
      top = most;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) y[e] = sum == 0.f ? 0.f : y[e] / sum;
    store_f32<DT, N>(static_cast<T*>(A.o) + (sp.lo + token) * A.o_stride + static_cast<int64_t>(head) * D + lane * N, y);
    if (lane == 0 && A.lse != nullptr) A.lse[(sp.lo + token) * C.heads + head] = natural_log_sum(top, sum);
  }
}

namespace {

template <int DT, int D>
hipError_t attend(const AttendArgs& a, hipStream_t s) {
  constexpr bool kWide = Tile<DT, D, 1>::kRow > 512;                            // as in plan_attend:
  constexpr int kTwo = Tile<DT, D, 2>::kSub >= 2 * Tile<DT, D, 2>::kGroup ? 2 : kWaves;  // row blocks of up to 32 rows
  const int64_t heads = a.c.key_heads;
  const dim3 threads(kWaves * kWave);
  if constexpr (!kWide) {
    if (a.groups == 0) {
      const dim3 grid(static_cast<unsigned>(a.c.batch * heads * a.row_blocks));
      if (a.row_waves == 1 && a.few) k_attend_whole<DT, D, 1, kWaves><<<grid, threads, 0, s>>>(a);
      else if (a.row_waves == 1) k_attend_whole<DT, D, 1, kMany><<<grid, dim3(kMany * kWave), 0, s>>>(a);
      else if (a.row_waves == 2) k_attend_whole<DT, D, kTwo, kWaves><<<grid, threads, 0, s>>>(a);
      else k_attend_whole<DT, D, kWaves, kWaves><<<grid, threads, 0, s>>>(a);
      return hipGetLastError();
    }
  }
  const dim3 grid(static_cast<unsigned>(a.groups * heads));
  if (kWide || a.row_waves == kWaves) k_attend<DT, D, kWaves><<<grid, threads, 0, s>>>(a);
  else if (a.row_waves == 2) k_attend<DT, D, kTwo><<<grid, threads, 0, s>>>(a);
  else k_attend<DT, D, kWide ? kWaves : 1><<<grid, threads, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // Few rows: 8 wavefronts each (one request of 100000 keys, 32 rows: 73 us from 76 with one), many: one (64 requests,
  // 2048 rows: 146 us from 150; 512 rows are the same), and more rows a workgroup where there are more than 2048 workgroups
  // of 4, most of whose rows then have one part (256 requests of 6 tokens, 120 keys: 52 us from 57).
  const int64_t blocks = static_cast<int64_t>(a.c.batch) * a.row_blocks * heads, items = blocks * a.block_rows;
  if (items > 512) {
    const int each = static_cast<int>(std::max((items / 2048 + kWaves - 1) / kWaves, int64_t{1})) * kWaves;
    k_attend_join<DT, D, 1><<<dim3(static_cast<unsigned>(blocks * ((a.block_rows + each - 1) / each))), threads, 0, s>>>(a, each);
  } else {
    k_attend_join<DT, D, 8><<<dim3(static_cast<unsigned>(items)), dim3(8 * kWave), 0, s>>>(a, 1);
  }
  return hipGetLastError();
}

template <int DT>
hipError_t pick(const AttendArgs& a, hipStream_t s) {
  return a.c.dim == 64 ? attend<DT, 64>(a, s) : a.c.dim == 128 ? attend<DT, 128>(a, s) : attend<DT, 256>(a, s);
}

}  // namespace

hipError_t launch_attend(int32_t io_dtype, AttendArgs a, void* ws, hipStream_t s) {
  if (a.groups > 0) {
    const int64_t places = attend_places(a);
    a.part = static_cast<float*>(ws);
    a.stat = a.part + places * a.c.dim;
    a.notes = reinterpret_cast<int32_t*>(a.stat + places * 2);
  }
  return io_dtype == SEED_BF16 ? pick<1>(a, s) : pick<0>(a, s);
}

}  // namespace seed
