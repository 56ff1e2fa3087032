// Gated scan of packed prompts over dense fp32 states, one token after another:
//   S_t = G_t S_{t-1} + beta_t k_t (v_t - [delta] (G_t S_{t-1})^T k_t)^T,   o_t = S_t^T q_t
// (the dense recurrences of GDN, KDA and Mamba-2; picx.dev summary, "Introduction and Theoretical
// Foundation" and "Exact Update (Lemma 2)").
//
// Every column of S follows its own recurrence given q, k, g and beta, so the d_v columns split
// freely. A wavefront holds its columns of one unit's state in registers: kLanes lanes share a column's
// rows and hold kCols columns each, and the two column sums S^T k and S^T q of a token are reduced over
// the kLanes lanes with DPP adds. The next kAhead tokens' rows are in flight while one block of them
// runs. The state is read and written once, whatever the prompt's length.
//
// What bounds it: with many units the vector unit (4 instructions per state element and token) and for
// prompts of a few tokens the states' bytes; with few units the latency of a token's chain. Three
// layouts, chosen by how many wavefronts 16 columns each would make (1024 fill the chip once).
// Times for 128 x 128 KDA states, 256 tokens (first row: 32 units, then 256, then 2048):
//     2 columns, 16 lanes    4 columns, 16 lanes    4 columns, 8 lanes
//            102 us                 142 us                215 us
//            269 us                 218 us                218 us
//           2025 us                1545 us               1246 us
// and 2048 one-token prompts take 99, 57 and 50 us (5.4 TB/s). With prompts shorter than 16 tokens
// the narrow layout gains nothing and is not used.
#include "common.hpp"
#include "prompt.hpp"

namespace seed {

// Wavefronts of a workgroup: up to 4, of one unit.
constexpr int scan_waves(int dv, int cols, int lanes) {
  const int n = dv * lanes / (64 * cols);
  return n < 4 ? n : 4;
}

template <int KIND, int DK, int DV, int IDT, int kCols, int kLanes, int kAhead>
__global__ __launch_bounds__(64 * scan_waves(DV, kCols, kLanes)) void k_scan_tokens(const ScanArgs A, int64_t units) {
  using IT = stor_t<IDT>;
  constexpr int R = DK / kLanes;   // rows per lane
  constexpr int WC = 64 / kLanes * kCols;  // columns per wavefront
  constexpr int NW = scan_waves(DV, kCols, kLanes);
  constexpr int SPLIT = DV / (NW * WC);    // workgroups per unit
  constexpr bool DELTA = KIND != SEED_MAMBA2;
  constexpr bool DIAG = KIND == SEED_KDA;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int row0 = (lane % kLanes) * R;
  for (int64_t item = blockIdx.x; item < units * SPLIT; item += gridDim.x) {
    const int64_t unit = item / SPLIT;
    const int col0 = static_cast<int>(item % SPLIT) * (NW * WC) + wave * WC + lane / kLanes * kCols;
    const int b = static_cast<int>(unit / A.heads), h = static_cast<int>(unit % A.heads);
    const int kh = h / (A.heads / A.key_heads);
    int64_t lo, hi;
    sequence_rows(A.offsets, b, A.tokens, lo, hi);

    float S[R][kCols];
    const int64_t sbase = unit * DK * DV + static_cast<int64_t>(row0) * DV + col0;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (A.S0 != nullptr) {
        load_f32<0, kCols>(A.S0 + sbase + i * DV, S[i]);
      } else {
#pragma unroll
        for (int c = 0; c < kCols; ++c) S[i][c] = 0.f;
      }
    }

    const IT* __restrict__ qp = static_cast<const IT*>(A.q) + static_cast<int64_t>(kh) * DK + row0;
    const IT* __restrict__ kp = static_cast<const IT*>(A.k) + static_cast<int64_t>(kh) * DK + row0;
    const IT* __restrict__ vp = static_cast<const IT*>(A.v) + static_cast<int64_t>(h) * DV + col0;
    IT* __restrict__ op = static_cast<IT*>(A.o) + static_cast<int64_t>(h) * DV + col0;

    struct Token {
      float q[R], k[R], v[kCols], g[DIAG ? R : 1], beta;
    };
    Token next[kAhead];
    // rows past the end load the last row again: never used, always inside the sequence
    auto fetch = [&](Token& t, int64_t r) {
      r = r < hi ? r : hi - 1;
      load_f32<IDT, R>(qp + r * A.q_stride, t.q);
      load_f32<IDT, R>(kp + r * A.k_stride, t.k);
      load_f32<IDT, kCols>(vp + r * A.v_stride, t.v);
      const int64_t at = r * A.heads + h;
      t.beta = A.beta[at];
      if constexpr (DIAG) load_f32<0, R>(A.g + at * DK + row0, t.g);
      else t.g[0] = A.g[at];
    };

    if (hi > lo) {
#pragma unroll
      for (int a = 0; a < kAhead; ++a) fetch(next[a], lo + a);
    }
    for (int64_t r0 = lo; r0 < hi; r0 += kAhead) {
      Token now[kAhead];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) now[a] = next[a];
#pragma unroll
      for (int a = 0; a < kAhead; ++a) fetch(next[a], r0 + kAhead + a);
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        if (r0 + a >= hi) break;  // the same for the whole wavefront
        const Token& t = now[a];
        float sk[kCols] = {}, sq[kCols] = {}, kq = 0.f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const float gi = DIAG ? t.g[i] : t.g[0];
          kq = fmaf(t.k[i], t.q[i], kq);
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            S[i][c] *= gi;
            if constexpr (DELTA) sk[c] = fmaf(t.k[i], S[i][c], sk[c]);
            sq[c] = fmaf(t.q[i], S[i][c], sq[c]);
          }
        }
        kq = group_sum<kLanes>(kq);
        float w[kCols], o[kCols];
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          sq[c] = group_sum<kLanes>(sq[c]);
          w[c] = t.v[c];
          if constexpr (DELTA) w[c] -= group_sum<kLanes>(sk[c]);
          w[c] *= t.beta;
          o[c] = fmaf(kq, w[c], sq[c]);
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int c = 0; c < kCols; ++c) S[i][c] = fmaf(t.k[i], w[c], S[i][c]);
        if (lane % kLanes == 0) store_f32<IDT, kCols>(op + (r0 + a) * A.o_stride, o);
      }
    }

#pragma unroll
    for (int i = 0; i < R; ++i) store_f32<0, kCols>(A.S + sbase + i * DV, S[i]);
  }
}

namespace {

using ScanFn = void (*)(const ScanArgs, int64_t);

struct Layout {
  int cols, lanes;
};

Layout pick_layout(const seed_shape& sh, int64_t tokens) {
  const int64_t waves = static_cast<int64_t>(sh.batch) * sh.heads * (sh.d_v / 16);
  if (waves <= 512 && tokens >= 16 * static_cast<int64_t>(sh.batch)) return {2, 16};
  if (waves <= 4096) return {4, 16};
  return {4, 8};
}

template <int KIND, int DK, int DV, int IDT>
ScanFn pick_layout_fn(Layout l) {
  if (l.cols == 2) return k_scan_tokens<KIND, DK, DV, IDT, 2, 16, 4>;
  if (l.lanes == 16) return k_scan_tokens<KIND, DK, DV, IDT, 4, 16, 4>;
  return k_scan_tokens<KIND, DK, DV, IDT, 4, 8, 1>;
}

template <int KIND, int DK, int DV>
ScanFn pick_io(int io, Layout l) {
  return io == SEED_BF16 ? pick_layout_fn<KIND, DK, DV, 1>(l) : pick_layout_fn<KIND, DK, DV, 0>(l);
}

template <int KIND>
ScanFn pick_dims(int dk, int dv, int io, Layout l) {
  if (dk == 128) return dv == 128 ? pick_io<KIND, 128, 128>(io, l) : pick_io<KIND, 128, 64>(io, l);
  return dv == 128 ? pick_io<KIND, 64, 128>(io, l) : pick_io<KIND, 64, 64>(io, l);
}

ScanFn pick_scan(const seed_shape& sh, Layout l) {
  switch (sh.kind) {
    case SEED_GDN: return pick_dims<SEED_GDN>(sh.d_k, sh.d_v, sh.io_dtype, l);
    case SEED_KDA: return pick_dims<SEED_KDA>(sh.d_k, sh.d_v, sh.io_dtype, l);
    default: return pick_dims<SEED_MAMBA2>(sh.d_k, sh.d_v, sh.io_dtype, l);
  }
}

}  // namespace

namespace {
// Whether the chunked kernel takes the call: bf16 rows and a gate per head, rows near enough for 32 of
// them to lie within a 31-bit offset, and prompts of 16 tokens or more on average. Chunked and token
// after token, from zeros, us:        8 tokens     12          16          24          32
//   GDN 128 x 128,   1024 units       49, 33       49, 42      48, 49      48, 65      48, 81
//                     256             17, 14       17, 17      17, 20      17, 26      17, 33
//                      32             13, 10       14, 11      13, 11      14, 14      14, 17
//   Mamba-2 128 x 64, 1024            22, 22       22, 26      22, 31      22, 40      22, 49
// The lengths themselves are on the device: one long prompt among many short ones goes by the average too.
bool takes_chunks(const seed_shape& sh, int64_t tokens, int64_t longest_stride) {
  return sh.io_dtype == SEED_BF16 && sh.kind != SEED_KDA && tokens >= 16 * static_cast<int64_t>(sh.batch) &&
         longest_stride < (int64_t{1} << 24);
}
int64_t longest(int64_t a, int64_t b, int64_t c, int64_t d) {
  const int64_t x = a > b ? a : b, y = c > d ? c : d;
  return x > y ? x : y;
}
}  // namespace

size_t prefill_scan_workspace(const seed_shape& sh, const seed_prompt& p) {
  if (!takes_chunks(sh, p.tokens, longest(p.q_stride, p.k_stride, p.v_stride, p.o_stride))) return 0;
  return scan_chunk_workspace(sh, p.tokens);
}

hipError_t launch_prefill_scan(const seed_shape& sh, const ScanArgs& a, hipStream_t s) {
  if (takes_chunks(sh, a.tokens, longest(a.q_stride, a.k_stride, a.v_stride, a.o_stride))) return launch_scan_chunk(sh, a, s);
  const int64_t units = static_cast<int64_t>(a.batch) * a.heads;
  const Layout l = pick_layout(sh, a.tokens);
  const int waves = scan_waves(sh.d_v, l.cols, l.lanes), split = sh.d_v * l.lanes / (64 * l.cols * waves);
  hipLaunchKernelGGL(pick_scan(sh, l), dim3(loop_blocks(units * split)), dim3(64 * waves), 0, s, a, units);
  return hipGetLastError();
}

}  // namespace seed
