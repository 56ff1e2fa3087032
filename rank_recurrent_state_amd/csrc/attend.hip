// Attention of a request's newest tokens over its paged cache:
//   o = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale q . k_j),
// in one pass over the keys with a running maximum m and sum l: weights are 2^(scale log2(e) q.k - m), and where
// m grows, what was summed so far is multiplied by 2^(m_old - m_new).
//
// What bounds it: every key and value is read once for all rows that share it, so HBM. A wavefront takes 32 keys
// at a time (fp32: 16), for 16 rows (queries of one key head, of all the request's new tokens) per matrix
// tile, and holds everything in registers:
//   S^T = K Q^T   a lane has row lane % 16 and keys 4 (lane / 16) + r of each 16,
//   O^T = V^T P^T takes the weights as they lie: the order of keys inside a product is free, so V's rows are
//                 loaded in the order in which the lanes hold the weights, whole rows of V by 16 lanes, and its
//                 16-bit values are paired by key with byte permutes. No LDS until the wavefronts are joined.
// bf16 weights enter as two pieces (p and p - bf16(p)), so that o is off by its own rounding only: with one
// piece the weights' rounding, 2^-9 each, is as large as o's. The products are far from the matrix unit's rate.
// m is only moved when a score passes it by 8 (weights up to 2^8): most tiles then need no exchange between
// lanes and no rescaling, and every weight keeps its relative precision.
#include "attend.hpp"
#include "common.hpp"

namespace seed {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr float kNegInf = -__builtin_inff();

using f32x4 = __attribute__((ext_vector_type(4))) float;
using u32x4 = __attribute__((ext_vector_type(4))) uint32_t;
using u32x2 = __attribute__((ext_vector_type(2))) uint32_t;
using bf16x8 = __attribute__((ext_vector_type(8))) __bf16;

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

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

// The positions that the rows of a request see between them: keys [k0, k1), row i at first + i.
struct Span {
  int64_t lo;
  int n, first, k0, k1, base, used;  // base: k0 at a tile's start; used: workgroups that have keys
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
  s.used = s.k1 > s.k0 ? static_cast<int>((static_cast<int64_t>(s.k1) - s.base + A.chunk - 1) / A.chunk) : 0;
  return s;
}

template <int DT, int D>
struct Tile {
  static constexpr int kBytes = DT == 0 ? 4 : 2;
  static constexpr int kVec = 16 / kBytes;            // values of a 16-byte access
  static constexpr int kSub = DT == 0 ? 1 : 2;        // 16-key parts of a tile
  static constexpr int kKeys = 16 * kSub;
  static constexpr int kQ = D / (4 * kVec);           // 16-byte pieces of a row per lane
  static constexpr int VE = D / 16 < kVec ? D / 16 : kVec;  // values of V per lane and access
  static constexpr int VC = D / (16 * VE);
  static constexpr int kOut = D / 16;                 // accumulators of 16 rows: value 16 VE c + VE m + j in number VE c + j
  static constexpr int kWords = VE * kBytes / 4;
};

}  // namespace

template <int DT, int D, int MT>
__global__ __launch_bounds__(kThreads) void k_attend(const AttendArgs A, int row_blocks, int64_t units) {
  using L = Tile<DT, D>;
  using T = stor_t<DT>;
  constexpr int GT = L::kOut < 8 ? L::kOut : 8;  // accumulators joined at a time
  __shared__ float stat[kWaves][MT * 16][2];
  __shared__ f32x4 red[kWaves][GT][kWave];

  // row blocks of one unit read the same keys: on the same XCD, one after the other
  const int64_t id = blockIdx.x;
  const int64_t group = id / (8 * row_blocks);
  const int within = static_cast<int>(id - group * 8 * row_blocks);
  const int rb = within / 8;
  const int64_t unit = group * 8 + within % 8;
  if (unit >= units) return;
  const CacheArgs& C = A.c;
  const int kh = static_cast<int>(unit % C.key_heads);
  const int64_t rest = unit / C.key_heads;
  const int b = static_cast<int>(rest % C.batch), split = static_cast<int>(rest / C.batch);

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l16 = lane & 15, g = lane >> 4;
  const Span sp = span_of(A, b);
  const int share = C.heads / C.key_heads;
  const int rows = sp.n * share, row0 = rb * MT * 16;
  if (row0 >= rows || split >= max(sp.used, 1)) return;

  // this lane's row of each 16: a query of key head kh
  int pos[MT];
  u32x4 Q[MT][L::kQ];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    const int r = row0 + 16 * t + l16;
    const int token = r / share;
    pos[t] = r < rows ? sp.first + token : -1;
    const T* q = static_cast<const T*>(A.q) + (sp.lo + token) * A.q_stride + static_cast<int64_t>(kh * share + r - token * share) * D;
#pragma unroll
    for (int c = 0; c < L::kQ; ++c) {
      Q[t][c] = u32x4{0, 0, 0, 0};
      if (r < rows) Q[t][c] = *reinterpret_cast<const u32x4*>(q + c * 4 * L::kVec + g * L::kVec);
    }
  }

  f32x4 O[MT][L::kOut];
  float m[MT], l[MT];
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    m[t] = kNegInf;
    l[t] = 0.f;
#pragma unroll
    for (int j = 0; j < L::kOut; ++j) O[t][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  }

  const int from = sp.base + split * A.chunk;
  const int to = static_cast<int>(min(static_cast<int64_t>(from) + A.chunk, static_cast<int64_t>(sp.k1)));
  const int last_pos = sp.first + sp.n - 1;
  const int32_t* __restrict__ table = C.table + static_cast<int64_t>(b) * C.width;
  const T* __restrict__ kb = static_cast<const T*>(C.k) + kh * C.head_stride;
  const T* __restrict__ vb = static_cast<const T*>(C.v) + kh * C.head_stride;
  const int64_t ts = C.token_stride;
  const int in_page = (1 << C.page_shift) - 1;

  for (int t0 = from + wave * L::kKeys; t0 < to; t0 += kWaves * L::kKeys) {
    // the 16 positions of a part lie in one page; parts behind the last key read the last one's
    bool there[L::kSub];
    int64_t at[L::kSub];
#pragma unroll
    for (int u = 0; u < L::kSub; ++u) {
      const int p = min(t0 + 16 * u, (sp.k1 - 1) & ~15);
      const int64_t number = table[p >> C.page_shift];
      there[u] = number >= 0 && number < C.pages;
      at[u] = (there[u] ? number : 0) * C.page_stride + (p & in_page) * ts;
    }
    u32x4 K[L::kSub][L::kQ];
#pragma unroll
    for (int u = 0; u < L::kSub; ++u)
#pragma unroll
      for (int c = 0; c < L::kQ; ++c)
        K[u][c] = *reinterpret_cast<const u32x4*>(kb + at[u] + l16 * ts + c * 4 * L::kVec + g * L::kVec);
    uint32_t V[4 * L::kSub][L::VC][L::kWords];
    auto load_v = [&]() {
#pragma unroll
      for (int i = 0; i < 4 * L::kSub; ++i)
#pragma unroll
        for (int c = 0; c < L::VC; ++c) {
          const T* p = vb + at[i / 4] + (4 * g + i % 4) * ts + c * 16 * L::VE + l16 * L::VE;
          if constexpr (L::kWords == 4) {
            const u32x4 w = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
            for (int e = 0; e < 4; ++e) V[i][c][e] = w[e];
          } else {
            const u32x2 w = *reinterpret_cast<const u32x2*>(p);
            V[i][c][0] = w[0];
            V[i][c][1] = w[1];
          }
        }
    };
    load_v();

    f32x4 S[MT][L::kSub];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int u = 0; u < L::kSub; ++u) {
        S[t][u] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < L::kQ; ++c) {
          if constexpr (DT == 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              S[t][u] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(K[u][c][e]), __uint_as_float(Q[t][c][e]), S[t][u], 0, 0, 0);
          } else {
            S[t][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, K[u][c]), __builtin_bit_cast(bf16x8, Q[t][c]),
                                                              S[t][u], 0, 0, 0);
          }
        }
      }

    // some row does not see some position of the tile
    bool edge = t0 < sp.k0 || t0 + L::kKeys > sp.first + 1 || (A.window > 0 && t0 <= last_pos - A.window);
#pragma unroll
    for (int u = 0; u < L::kSub; ++u) edge = edge || !there[u];
    auto sees = [&](int p, int i) {  // position p, key i of this lane
      const int key = t0 + 16 * (i / 4) + 4 * g + i % 4;
      return there[i / 4] && key <= p && (A.window <= 0 || key > p - A.window);
    };

    float P[MT][4 * L::kSub];
#pragma unroll
    for (int t = 0; t < MT; ++t) {
      float top = kNegInf;
#pragma unroll
      for (int i = 0; i < 4 * L::kSub; ++i) {
        float x = S[t][i / 4][i % 4] * A.scale2;
        if (edge && !sees(pos[t], i)) x = kNegInf;
        top = fmaxf(top, x);
      }
      if (__any(top > m[t] + 8.f)) {
        const float now = fmaxf(m[t], max4(top));
        // nothing summed so far, or all of it of weight 0: 2^(-inf)
        const float f = now == kNegInf ? 1.f : exp2_(m[t] - now);
        m[t] = now;
        l[t] *= f;
#pragma unroll
        for (int j = 0; j < L::kOut; ++j) O[t][j] *= f;
      }
      const float sub = m[t] == kNegInf ? 0.f : m[t];
#pragma unroll
      for (int i = 0; i < 4 * L::kSub; ++i) {
        float p = exp2_(fmaf(S[t][i / 4][i % 4], A.scale2, -sub));
        if (edge && !sees(pos[t], i)) p = 0.f;
        P[t][i] = p;
        l[t] += p;
      }
    }

    auto values = [&](int t, f32x4 (&acc)[L::kOut], int only) {  // only >= 0: of this row alone
      if constexpr (DT == 0) {
#pragma unroll
        for (int c = 0; c < L::VC; ++c)
#pragma unroll
          for (int j = 0; j < L::VE; ++j) {
            f32x4 z = acc[c * L::VE + j];
#pragma unroll
            for (int i = 0; i < 4; ++i) z = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(V[i][c][j]), P[t][i], z, 0, 0, 0);
            if (only < 0 || l16 == only) acc[c * L::VE + j] = z;
          }
      } else {
        u32x4 hi, lo;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          hi[i] = pack2<1>(P[t][2 * i], P[t][2 * i + 1]);
          lo[i] = pack2<1>(P[t][2 * i] - lo16<1>(hi[i]), P[t][2 * i + 1] - hi16<1>(hi[i]));
        }
#pragma unroll
        for (int c = 0; c < L::VC; ++c)
#pragma unroll
          for (int j = 0; j < L::VE; ++j) {
            u32x4 a;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              a[i] = __builtin_amdgcn_perm(V[2 * i + 1][c][j / 2], V[2 * i][c][j / 2], j % 2 == 0 ? 0x05040100u : 0x07060302u);
            f32x4 z = acc[c * L::VE + j];
            z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, hi), z, 0, 0, 0);
            z = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, lo), z, 0, 0, 0);
            if (only < 0 || l16 == only) acc[c * L::VE + j] = z;
          }
      }
    };
    auto clear_v = [&](int i) {
#pragma unroll
      for (int c = 0; c < L::VC; ++c)
#pragma unroll
        for (int e = 0; e < L::kWords; ++e) V[i][c][e] = 0;
    };

    bool apart = false;
    if (edge) {
      // A weight of 0 does not keep an infinity or NaN out of a product. Values that no row sees become 0; where
      // those that some rows see are not all finite, the rows are taken one at a time.
      uint32_t bad = 0;
#pragma unroll
      for (int i = 0; i < 4 * L::kSub; ++i) {
        const int key = t0 + 16 * (i / 4) + 4 * g + i % 4;
        if (!there[i / 4] || key < sp.k0 || key >= sp.k1) clear_v(i);
#pragma unroll
        for (int c = 0; c < L::VC; ++c)
#pragma unroll
          for (int e = 0; e < L::kWords; ++e) {
            const uint32_t w = V[i][c][e];
            if constexpr (DT == 0) bad |= (w & 0x7f800000u) == 0x7f800000u;
            else bad |= (w & 0x7f800000u) == 0x7f800000u || (w & 0x7f80u) == 0x7f80u;
          }
      }
      apart = __any(bad != 0);
    }
    if (!apart) {
#pragma unroll
      for (int t = 0; t < MT; ++t) values(t, O[t], -1);
    } else {
#pragma unroll
      for (int t = 0; t < MT; ++t)
        for (int r = 0; r < 16; ++r) {
          load_v();
          const int row = row0 + 16 * t + r;
          const int p = row < rows ? sp.first + row / share : -1;
#pragma unroll
          for (int i = 0; i < 4 * L::kSub; ++i)
            if (!sees(p, i)) clear_v(i);
          values(t, O[t], r);
        }
    }
  }

  // join the wavefronts: the largest maximum, sums and accumulators brought to it
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    l[t] = sum4(l[t]);
    if (g == 0) {
      stat[wave][16 * t + l16][0] = m[t];
      stat[wave][16 * t + l16][1] = l[t];
    }
  }
  __syncthreads();
  const bool whole = sp.used <= 1;
  const int orow = threadIdx.x & 15, om = threadIdx.x >> 4;  // the row and 16th of its values that this thread writes
#pragma unroll
  for (int t = 0; t < MT; ++t) {
    float top = kNegInf;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) top = fmaxf(top, stat[w][16 * t + l16][0]);
    const float f = m[t] == kNegInf ? 0.f : exp2_(m[t] - top);
    // the same for the row this thread writes
    float wtop = kNegInf, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) wtop = fmaxf(wtop, stat[w][16 * t + orow][0]);
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const float mw = stat[w][16 * t + orow][0], lw = stat[w][16 * t + orow][1];
      sum += mw == kNegInf ? lw : lw * exp2_(mw - wtop);  // lw: 0, or NaN
    }
    const int r = row0 + 16 * t + orow;
    const int token = r / share, head = kh * share + r - token * share;
    const int64_t line = (sp.lo + token) * C.heads + head;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    if (r < rows && om == 0) {
      if (!whole) {
        float* st = A.stat + (line * A.splits + split) * 2;
        st[0] = wtop;
        st[1] = sum;
      } else if (A.lse != nullptr) {
        A.lse[line] = sum == 0.f ? kNegInf : static_cast<float>((static_cast<double>(wtop) + log2(static_cast<double>(sum))) * 0.6931471805599453);
      }
    }
#pragma unroll
    for (int j0 = 0; j0 < L::kOut; j0 += GT) {
      __syncthreads();  // what was joined before has been read
#pragma unroll
      for (int j = 0; j < GT; ++j) red[wave][j][lane] = O[t][j0 + j] * f;
      __syncthreads();
      constexpr int kRun = L::VE;  // neighbouring values of a thread
#pragma unroll
      for (int c = 0; c < GT / kRun; ++c) {
        float y[kRun];
#pragma unroll
        for (int j = 0; j < kRun; ++j) {
          const int src = (om >> 2) * 16 + orow;
          y[j] = 0.f;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) y[j] += reinterpret_cast<const float*>(&red[w][c * kRun + j][src])[om & 3];
        }
        const int v = (j0 / kRun + c) * 16 * kRun + om * kRun;
        if (r < rows) {
          if (!whole) {
            store_f32<0, kRun>(A.part + (line * A.splits + split) * D + v, y);
          } else {
#pragma unroll
            for (int j = 0; j < kRun; ++j) y[j] = sum == 0.f ? 0.f : y[j] * inv;
            store_f32<DT, kRun>(static_cast<T*>(A.o) + (sp.lo + token) * A.o_stride + static_cast<int64_t>(head) * D + v, y);
          }
        }
      }
    }
  }
}

// Joins the workgroups along a cache: a workgroup per row and head, D / 4 threads per part.
template <int DT, int D>
__global__ __launch_bounds__(kThreads) void k_attend_join(const AttendArgs A) {
  using T = stor_t<DT>;
  constexpr int kLine = D / 4, kPer = kThreads / kLine;
  __shared__ f32x4 acc[kPer][kLine];
  __shared__ float sums[kPer];
  const int head = static_cast<int>(blockIdx.x % A.c.heads);
  const int64_t rest = blockIdx.x / A.c.heads;
  const int token = static_cast<int>(rest % A.max_tokens), b = static_cast<int>(rest / A.max_tokens);
  const Span sp = span_of(A, b);
  if (token >= sp.n || sp.used <= 1) return;
  const int64_t line = (sp.lo + token) * A.c.heads + head;
  const float* stat = A.stat + line * A.splits * 2;
  const float* part = A.part + line * A.splits * D;
  const int lane = threadIdx.x & 63;
  float top = kNegInf;
  for (int s = lane; s < sp.used; s += kWave) top = fmaxf(top, stat[2 * s]);
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) top = fmaxf(top, __shfl_xor(top, d, kWave));
  const int p = threadIdx.x / kLine, v = threadIdx.x % kLine;
  f32x4 y = {0.f, 0.f, 0.f, 0.f};
  float sum = 0.f;
#pragma unroll 4
  for (int s = p; s < sp.used; s += kPer) {
    const float mw = stat[2 * s], lw = stat[2 * s + 1];
    const f32x4 x = *reinterpret_cast<const f32x4*>(part + static_cast<int64_t>(s) * D + 4 * v);
    const float f = mw == kNegInf ? 1.f : exp2_(mw - top);  // a part of no weight holds zeros, or NaN
    y += x * f;
    sum += lw * f;
  }
  acc[p][v] = y;
  if (v == 0) sums[p] = sum;
  __syncthreads();
  if (p != 0) return;
  sum = 0.f;
  y = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < kPer; ++i) {
    y += acc[i][v];
    sum += sums[i];
  }
  float out[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) out[e] = sum == 0.f ? 0.f : y[e] / sum;
  store_f32<DT, 4>(static_cast<T*>(A.o) + (sp.lo + token) * A.o_stride + static_cast<int64_t>(head) * D + 4 * v, out);
  if (v == 0 && A.lse != nullptr)
    A.lse[line] = sum == 0.f ? kNegInf : static_cast<float>((static_cast<double>(top) + log2(static_cast<double>(sum))) * 0.6931471805599453);
}

namespace {

// 16-row tiles of a wavefront: as many as the rows need and the registers hold (accumulators and
// queries grow with both the tiles and the head).
int tiles_of(int32_t max_tokens, int32_t share, int dim) {
  const int64_t rows = static_cast<int64_t>(max_tokens) * share;
  const int most = 256 / dim;
  int t = 1;
  while (t < most && 16 * t < rows) t *= 2;
  return t;
}

template <int DT, int D, int MT>
hipError_t attend(const AttendArgs& a, hipStream_t s) {
  const int64_t rows = static_cast<int64_t>(a.max_tokens) * (a.c.heads / a.c.key_heads);
  const int64_t row_blocks = (rows + 16 * MT - 1) / (16 * MT);
  const int64_t units = static_cast<int64_t>(a.c.batch) * a.c.key_heads * a.splits;
  const int64_t blocks = (units + 7) / 8 * 8 * row_blocks;
  k_attend<DT, D, MT><<<dim3(static_cast<unsigned>(blocks)), dim3(kThreads), 0, s>>>(a, static_cast<int>(row_blocks), units);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  k_attend_join<DT, D><<<dim3(static_cast<unsigned>(static_cast<int64_t>(a.c.batch) * a.max_tokens * a.c.heads)), dim3(kThreads), 0, s>>>(a);
  return hipGetLastError();
}

template <int DT>
hipError_t pick(const AttendArgs& a, hipStream_t s) {
  const int t = tiles_of(a.max_tokens, a.c.heads / a.c.key_heads, a.c.dim);
  if (a.c.dim == 64) return t == 1 ? attend<DT, 64, 1>(a, s) : t == 2 ? attend<DT, 64, 2>(a, s) : attend<DT, 64, 4>(a, s);
  if (a.c.dim == 128) return t == 1 ? attend<DT, 128, 1>(a, s) : attend<DT, 128, 2>(a, s);
  return attend<DT, 256, 1>(a, s);
}

}  // namespace

void plan_attend(int32_t io_dtype, AttendArgs& a) {
  constexpr int kStep = 128;  // keys of one turn of a workgroup
  constexpr int64_t kGroups = 2048;
  const int share = a.c.heads / a.c.key_heads;
  const int64_t rows = static_cast<int64_t>(a.max_tokens) * share, mt = tiles_of(a.max_tokens, share, a.c.dim);
  const int64_t units = static_cast<int64_t>(a.c.batch) * a.c.key_heads * ((rows + 16 * mt - 1) / (16 * mt));
  int64_t span = a.capacity;
  if (a.window > 0) {
    const int64_t near = static_cast<int64_t>(a.window) + a.max_tokens - 1 + 31;
    span = near < span ? near : span;
  }
  int64_t splits = (kGroups + units - 1) / units;
  const int64_t most = (span + kStep - 1) / kStep;
  splits = splits < most ? splits : most;
  const int64_t chunk = ((span + splits - 1) / splits + kStep - 1) / kStep * kStep;
  a.chunk = static_cast<int32_t>(chunk < (int64_t{1} << 31) - kStep ? chunk : (int64_t{1} << 31) - kStep);
  a.splits = static_cast<int32_t>((span + a.chunk - 1) / a.chunk);
}

hipError_t launch_attend(int32_t io_dtype, const AttendArgs& a, hipStream_t s) {
  return io_dtype == SEED_BF16 ? pick<1>(a, s) : pick<0>(a, s);
}

}  // namespace seed
