// Gated scan of packed bf16 prompts in chunks of 32 tokens on the matrix cores (GDN, Mamba-2).
//
// With c_t the sum of log2 g over the chunk's tokens up to t, S0 the state before the chunk and
// s <= t throughout, the recurrence of scan.hip over a chunk is
//   (I + L) W = B (V - H K S0),  L[t][s] = beta_t 2^(c_t - c_s) k_t . k_s  (s < t)     (GDN)
//   W = B V                                                                              (Mamba-2)
//   O = H Q S0 + P W,   P[t][s] = 2^(c_t - c_s) q_t . k_s,   H = diag 2^(c_t)
//   S1 = 2^(c_end) S0 + K^T diag(2^(c_end - c_s)) W.
// T = (I + L)^-1 is formed explicitly, by forward substitution in 16 x 16 blocks (products of powers
// of L would cancel badly when keys repeat), and multiplies the right-hand side.
//
// Precision. q, k and v are bf16 and enter the matrix instructions exactly. fp32 operands enter
// as sums of bf16 pieces, each the rounding of what the ones before left: three pieces hold all 24
// bits (the state where it meets k, T and its right-hand side, W where it enters the state), two hold
// 16 (the state where it meets q, P and W in P W), enough for a read-out that is rounded to 8 bits
// and does not feed back. Sums are fp32. The running c is summed in fp64 and kept as two floats,
// so that differences of large sums keep their bits.
//
// Layout. A workgroup has one unit and one wavefront per 32 columns of d_v; a wavefront holds its
// columns of the state, d_k x 32 fp32, in accumulator layout. Rows of the operand tiles are
// permuted so that a lane's 8 consecutive accumulator registers are 8 consecutive rows: the
// accumulators of one product are then the right operand of the next, and S, W and O never leave
// the registers. K, Q, T and P are left operands in LDS; K^T and V come out of row-major tiles
// with the transposing LDS read. One wavefront forms T while another forms P and the rest already
// multiply K and Q with the state.
#include "common.hpp"
#include "prompt.hpp"

namespace seed {

namespace {

using bf16x8 = __attribute__((ext_vector_type(8))) __bf16;
using bf16x2 = __attribute__((ext_vector_type(2))) __bf16;
using f32x2 = __attribute__((ext_vector_type(2))) float;
using f32x4 = __attribute__((ext_vector_type(4))) float;
using f32x16 = __attribute__((ext_vector_type(16))) float;
using s16x4 = __attribute__((ext_vector_type(4))) short;

constexpr int C = 32;       // tokens per chunk
constexpr int kPad = 8;     // bf16 row padding: rows 16 bytes apart in the banks
constexpr int LT = C + 8;   // row length of the T and P pieces
constexpr int LF = C + 4;   // row length of the fp32 L and T

// Row m of a 32-row operand tile holds token or channel perm(m), which puts 8 consecutive ones into
// a lane's accumulator registers 0..7 and 8..15: register i of lane half h is 16 (i / 8) + 8 h + i % 8.
__device__ __forceinline__ int perm(int m) { return (m & 19) | ((m & 4) << 1) | ((m & 8) >> 1); }

__device__ __forceinline__ f32x16 mma(const bf16x8& a, const bf16x8& b, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// x[0..7] as N bf16 pieces, largest first.
template <int N>
__device__ __forceinline__ void split(const float (&x)[8], bf16x8 (&p)[N]) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    f32x2 r = {x[e], x[e + 1]};
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const bf16x2 h = __builtin_convertvector(r, bf16x2);
      p[n][e] = h[0];
      p[n][e + 1] = h[1];
      if (n + 1 < N) {
        const uint32_t w = __builtin_bit_cast(uint32_t, h);
        r[0] -= __uint_as_float(w << 16);
        r[1] -= __uint_as_float(w & 0xffff0000u);
      }
    }
  }
}

__device__ __forceinline__ bf16x8 frag(const uint16_t* p) { return *reinterpret_cast<const bf16x8*>(p); }

// Four rows of a row-major 16-bit tile, transposed: lane i of 16 passes the address of row i / 4,
// columns 4 (i % 4) .. + 3 and receives column i, rows 0 .. 3.
__device__ __forceinline__ s16x4 read_tr(const uint16_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(
      (__attribute__((address_space(3))) s16x4*)(const_cast<uint16_t*>(p)));
}

template <int KIND, int DK, int DV>
struct Tiles {
  static constexpr bool DELTA = KIND != SEED_MAMBA2;
  static constexpr int LK = DK + kPad, LV = DV + kPad;
  uint16_t K[C * LK];
  uint16_t Q[C * LK];
  uint16_t V[C * LV];             // v, then o
  uint16_t P[2][C * LT];
  uint16_t T[DELTA ? 3 : 1][DELTA ? C * LT : 8];
  float L[DELTA ? C * LF : 4];
  float Tf[DELTA ? C * LF : 4];
  float ch[C], cl[C];             // c as a sum of two floats
  float head[C], tail[C];         // 2^c_t, 2^(c_end - c_t)
  float beta[C], g[C];
};

}  // namespace

template <int KIND, int DK, int DV>
__global__ __launch_bounds__(DV * 2, 2) void k_scan_chunk(const ScanArgs A, int64_t units) {
  using TL = Tiles<KIND, DK, DV>;
  constexpr bool DELTA = TL::DELTA;
  constexpr int NW = DV / 32, NT = NW * 64;
  constexpr int LK = TL::LK, LV = TL::LV;
  constexpr int RT = DK / 32;                 // row tiles of the state
  constexpr int KP = C * DK / 8 / NT;         // 16-byte pieces of K (and Q) per thread
  constexpr int VP = C * DV / 8 / NT;
  __shared__ TL sh;

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l32 = lane & 31, half = lane >> 5;
  const int prow = perm(l32);

  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int b = static_cast<int>(unit / A.heads), h = static_cast<int>(unit % A.heads);
    const int kh = h / (A.heads / A.key_heads);
    int64_t lo, hi;
    sequence_rows(A.offsets, b, A.tokens, lo, hi);

    const uint16_t* __restrict__ qp = static_cast<const uint16_t*>(A.q) + static_cast<int64_t>(kh) * DK;
    const uint16_t* __restrict__ kp = static_cast<const uint16_t*>(A.k) + static_cast<int64_t>(kh) * DK;
    const uint16_t* __restrict__ vp = static_cast<const uint16_t*>(A.v) + static_cast<int64_t>(h) * DV;
    uint16_t* __restrict__ op = static_cast<uint16_t*>(A.o) + static_cast<int64_t>(h) * DV;

    // the state: register i of row tile r is row 32 r + 16 (i / 8) + 8 half + i % 8, column 32 wave + l32
    f32x16 S[RT];
    const int64_t sbase = unit * DK * DV + static_cast<int64_t>(8 * half) * DV + 32 * wave + l32;
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        S[r][i] = A.S0 != nullptr ? A.S0[sbase + (32 * r + 16 * (i / 8) + i % 8) * DV] : 0.f;

    // the next chunk's rows, on their way from memory; rows past the end read as zeros, g as 1
    uint4 nk[KP], nq[KP], nv[VP];
    float ng = 1.f, nb = 0.f;
    auto fetch = [&](int64_t c0) {
      const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int p = 0; p < KP; ++p) {
        const int at = p * NT + threadIdx.x, row = at / (DK / 8), col = at % (DK / 8) * 8;
        const bool in = c0 + row < hi;
        const int64_t rr = in ? c0 + row : hi - 1;
        const uint4 x = *reinterpret_cast<const uint4*>(kp + rr * A.k_stride + col);
        const uint4 y = *reinterpret_cast<const uint4*>(qp + rr * A.q_stride + col);
        nk[p] = in ? x : zero;
        nq[p] = in ? y : zero;
      }
#pragma unroll
      for (int p = 0; p < VP; ++p) {
        const int at = p * NT + threadIdx.x, row = at / (DV / 8), col = at % (DV / 8) * 8;
        const bool in = c0 + row < hi;
        const int64_t rr = in ? c0 + row : hi - 1;
        const uint4 x = *reinterpret_cast<const uint4*>(vp + rr * A.v_stride + col);
        nv[p] = in ? x : zero;
      }
      if (wave == NW - 1) {
        const bool in = c0 + l32 < hi;
        const int64_t at = (in ? c0 + l32 : hi - 1) * A.heads + h;
        ng = in ? A.g[at] : 1.f;
        nb = in ? A.beta[at] : 0.f;
      }
    };
    if (lo < hi) fetch(lo);

    for (int64_t c0 = lo; c0 < hi; c0 += C) {
      // ---- the chunk into LDS, and its gates -------------------------------------------------------
#pragma unroll
      for (int p = 0; p < KP; ++p) {
        const int at = p * NT + threadIdx.x, row = at / (DK / 8), col = at % (DK / 8) * 8;
        *reinterpret_cast<uint4*>(sh.K + row * LK + col) = nk[p];
        *reinterpret_cast<uint4*>(sh.Q + row * LK + col) = nq[p];
      }
#pragma unroll
      for (int p = 0; p < VP; ++p) {
        const int at = p * NT + threadIdx.x, row = at / (DV / 8), col = at % (DV / 8) * 8;
        *reinterpret_cast<uint4*>(sh.V + row * LV + col) = nv[p];
      }
      if (wave == NW - 1) {
        // g = 0 counts as 2^-200: across it every weight underflows to 0, as it should
        const float lg = log2f(ng);
        double c = lg < -200.f ? -200.0 : static_cast<double>(lg);
#pragma unroll
        for (int d = 1; d < C; d <<= 1) {
          const double up = __shfl_up(c, d, C);
          if (l32 >= d) c += up;
        }
        const float hi32 = static_cast<float>(c), lo32 = static_cast<float>(c - static_cast<double>(hi32));
        const double rest = __shfl(c, C - 1, C) - c;
        const float rh = static_cast<float>(rest), rl = static_cast<float>(rest - static_cast<double>(rh));
        const float eh = exp2f(hi32), et = exp2f(rh);
        if (lane < C) {
          sh.ch[lane] = hi32;
          sh.cl[lane] = lo32;
          sh.head[lane] = fmaf(eh, 0.693147181f * lo32, eh);
          sh.tail[lane] = fmaf(et, 0.693147181f * rl, et);
          sh.beta[lane] = nb;
          sh.g[lane] = ng;
        }
      }
      __syncthreads();
      if (c0 + C < hi) fetch(c0 + C);

      // ---- P, and T by another wavefront ------------------------------------------------------------
      // 2^(c_t - c_s) for t = l32 and the 16 s of the lane's accumulator registers
      auto weights = [&](float (&e)[16]) {
        const float th = sh.ch[l32], tl = sh.cl[l32];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int s = 16 * (i / 8) + 8 * half + i % 8;
          e[i] = __builtin_amdgcn_exp2f((th - sh.ch[s]) + (tl - sh.cl[s]));
        }
      };
      if (wave == NW - 1) {
        f32x16 acc = {};
#pragma unroll
        for (int ks = 0; ks < DK / 16; ++ks)
          acc = mma(frag(sh.K + prow * LK + 16 * ks + 8 * half), frag(sh.Q + l32 * LK + 16 * ks + 8 * half), acc);
        float e[16];
        weights(e);
#pragma unroll
        for (int s8 = 0; s8 < 2; ++s8) {
          float x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int s = 16 * s8 + 8 * half + j;
            float w = acc[8 * s8 + j] * e[8 * s8 + j];
            if constexpr (!DELTA) w *= sh.beta[s];
            x[j] = s <= l32 ? w : 0.f;
          }
          bf16x8 pc[2];
          split<2>(x, pc);
#pragma unroll
          for (int n = 0; n < 2; ++n) *reinterpret_cast<bf16x8*>(sh.P[n] + l32 * LT + 16 * s8 + 8 * half) = pc[n];
        }
      }
      if constexpr (DELTA) {
        if (wave == 0) {
          f32x16 acc = {};
#pragma unroll
          for (int ks = 0; ks < DK / 16; ++ks)
            acc = mma(frag(sh.K + prow * LK + 16 * ks + 8 * half), frag(sh.K + l32 * LK + 16 * ks + 8 * half), acc);
          float e[16];
          weights(e);
          const float bt = sh.beta[l32];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const int s = 16 * (i / 8) + 8 * half + i % 8;
            e[i] = s < l32 ? bt * (acc[i] * e[i]) : 0.f;
          }
#pragma unroll
          for (int i = 0; i < 16; i += 4)
            *reinterpret_cast<float4*>(sh.L + l32 * LF + 16 * (i / 8) + 8 * half + i % 8) =
                make_float4(e[i], e[i + 1], e[i + 2], e[i + 3]);
          wave_lds_sync();
          // the two diagonal blocks: lane l32 solves for column l32 % 16 of block l32 / 16
          const int blk = l32 & 16, jj = l32 & 15;
          float x[16];
#pragma unroll
          for (int t = 0; t < 16; ++t) {
            float a0 = t == jj ? 1.f : 0.f;
#pragma unroll
            for (int s = 0; s < t; ++s) a0 = fmaf(-sh.L[(blk + t) * LF + blk + s], x[s], a0);
            x[t] = a0;
          }
          if (lane < C) {
#pragma unroll
            for (int t = 0; t < 16; ++t) {
              sh.Tf[(blk + t) * LF + blk + jj] = x[t];
              if (blk) sh.Tf[t * LF + 16 + jj] = 0.f;
            }
          }
          wave_lds_sync();
          // the block below: -T11 (L10 T00), fp32 matrix instructions (k slot lane / 16 of step i is 4 (lane / 16) + i)
          const int r16 = lane & 15, g4 = lane >> 4;
          f32x4 m1 = {}, m2 = {};
          const f32x4 a1 = *reinterpret_cast<const f32x4*>(sh.L + (16 + r16) * LF + 4 * g4);
          const f32x4 a2 = *reinterpret_cast<const f32x4*>(sh.Tf + (16 + r16) * LF + 16 + 4 * g4);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            m1 = __builtin_amdgcn_mfma_f32_16x16x4f32(a1[i], sh.Tf[(4 * g4 + i) * LF + r16], m1, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) m2 = __builtin_amdgcn_mfma_f32_16x16x4f32(a2[i], m1[i], m2, 0, 0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) sh.Tf[(16 + 4 * g4 + i) * LF + r16] = -m2[i];
          wave_lds_sync();
          // T diag(beta) in pieces
#pragma unroll
          for (int s8 = 0; s8 < 2; ++s8) {
            const int col = 16 * s8 + 8 * half;
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = col + j <= l32 ? sh.Tf[l32 * LF + col + j] * sh.beta[col + j] : 0.f;
            bf16x8 pc[3];
            split<3>(y, pc);
#pragma unroll
            for (int n = 0; n < 3; ++n) *reinterpret_cast<bf16x8*>(sh.T[n] + l32 * LT + col) = pc[n];
          }
        }
      }

      // ---- K S and Q S ------------------------------------------------------------------------------
      f32x16 ks = {}, qs = {};
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          float x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = S[r][8 * s + j];
          const int col = 32 * r + 16 * s + 8 * half;
          const bf16x8 aq = frag(sh.Q + prow * LK + col);
          if constexpr (DELTA) {
            bf16x8 pc[3];
            split<3>(x, pc);
            const bf16x8 ak = frag(sh.K + prow * LK + col);
            ks = mma(ak, pc[2], ks);
            qs = mma(aq, pc[1], qs);
            ks = mma(ak, pc[1], ks);
            qs = mma(aq, pc[0], qs);
            ks = mma(ak, pc[0], ks);
          } else {
            bf16x8 pc[2];
            split<2>(x, pc);
            qs = mma(aq, pc[1], qs);
            qs = mma(aq, pc[0], qs);
          }
        }
      // v in accumulator layout, and as the bf16 right operand it already is
      bf16x8 vb[2];
      const uint16_t* vt = sh.V + (8 * half + (lane & 15) / 4) * LV + 32 * wave + (lane & 16) + 4 * (lane & 3);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const s16x4 x0 = read_tr(vt + 16 * s * LV), x1 = read_tr(vt + (16 * s + 4) * LV);
        const __attribute__((ext_vector_type(8))) short x = {x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
        vb[s] = __builtin_bit_cast(bf16x8, x);
      }
      __syncthreads();

      // ---- W ----------------------------------------------------------------------------------------
      f32x16 w;
      float hd[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) hd[i] = sh.head[16 * (i / 8) + 8 * half + i % 8];
      if constexpr (DELTA) {
        w = f32x16{};
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          float x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = fmaf(-hd[8 * s + j], ks[8 * s + j], static_cast<float>(vb[s][j]));
          bf16x8 rp[3], tp[3];
          split<3>(x, rp);
#pragma unroll
          for (int n = 0; n < 3; ++n) tp[n] = frag(sh.T[n] + prow * LT + 16 * s + 8 * half);
          w = mma(tp[2], rp[0], w);
          w = mma(tp[1], rp[1], w);
          w = mma(tp[0], rp[2], w);
          w = mma(tp[1], rp[0], w);
          w = mma(tp[0], rp[1], w);
          w = mma(tp[0], rp[0], w);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = static_cast<float>(vb[i / 8][i % 8]) * sh.beta[16 * (i / 8) + 8 * half + i % 8];
      }

      // A value that is not finite would reach the tokens before its own through the zeros of T and P:
      // such a chunk runs token after token instead.
      float fin = 0.f;
#pragma unroll
      for (int i = 0; i < 16; ++i) fin = fmaf(w[i], 0.f, fin);
      if (__builtin_expect(__any(!(fin == 0.f)), 0)) {
        const int n = static_cast<int>(hi - c0 < C ? hi - c0 : C);
#pragma unroll 1
        for (int t = 0; t < n; ++t) {
          const float gt = sh.g[t];
          float sk = 0.f, sq = 0.f, kq = 0.f;
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int col = 32 * r + 16 * (i / 8) + 8 * half + i % 8;
              const float kv = bf16_to_f32(sh.K[t * LK + col]), qv = bf16_to_f32(sh.Q[t * LK + col]);
              S[r][i] *= gt;
              sk = fmaf(kv, S[r][i], sk);
              sq = fmaf(qv, S[r][i], sq);
              kq = fmaf(kv, qv, kq);
            }
          sk += __shfl_xor(sk, 32, 64);
          sq += __shfl_xor(sq, 32, 64);
          kq += __shfl_xor(kq, 32, 64);
          float x = bf16_to_f32(sh.V[t * LV + 32 * wave + l32]);
          if constexpr (DELTA) x -= sk;
          x *= sh.beta[t];
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int i = 0; i < 16; ++i)
              S[r][i] = fmaf(bf16_to_f32(sh.K[t * LK + 32 * r + 16 * (i / 8) + 8 * half + i % 8]), x, S[r][i]);
          wave_lds_sync();  // both halves have read v
          if (half == 0) sh.V[t * LV + 32 * wave + l32] = f32_to_bf16(fmaf(kq, x, sq));
        }
      } else {
        // ---- O = H Q S + P W --------------------------------------------------------------------------
        f32x16 o;
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = hd[i] * qs[i];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const bf16x8 p0 = frag(sh.P[0] + prow * LT + 16 * s + 8 * half), p1 = frag(sh.P[1] + prow * LT + 16 * s + 8 * half);
          if constexpr (DELTA) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = w[8 * s + j];
            bf16x8 wp[2];
            split<2>(x, wp);
            o = mma(p1, wp[0], o);
            o = mma(p0, wp[1], o);
            o = mma(p0, wp[0], o);
          } else {
            o = mma(p1, vb[s], o);
            o = mma(p0, vb[s], o);
          }
        }
        // ---- S = 2^(c_end) S + K^T diag(tail) W ----------------------------------------------------------
        const float ge = sh.head[C - 1];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int i = 0; i < 16; ++i) S[r][i] *= ge;
        // lane i of 16 passes row i / 4 of 4 tokens and the channels that perm puts at 4 (i % 4)
        const uint16_t* kt = sh.K + (8 * half + (lane & 15) / 4) * LK + perm(4 * (lane & 3)) + (lane & 16);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          float x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = w[8 * s + j] * sh.tail[16 * s + 8 * half + j];
          bf16x8 wp[3];
          split<3>(x, wp);
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const s16x4 x0 = read_tr(kt + 16 * s * LK + 32 * r), x1 = read_tr(kt + (16 * s + 4) * LK + 32 * r);
            const __attribute__((ext_vector_type(8))) short y = {x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
            const bf16x8 a = __builtin_bit_cast(bf16x8, y);
            S[r] = mma(a, wp[2], S[r]);
            S[r] = mma(a, wp[1], S[r]);
            S[r] = mma(a, wp[0], S[r]);
          }
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
          sh.V[(16 * (i / 8) + 8 * half + i % 8) * LV + 32 * wave + l32] = f32_to_bf16(o[i]);
      }
      // ---- the read-outs: a wavefront's 32 columns of a row are 64 bytes, 16 per lane ----------------
      wave_lds_sync();
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int row = 16 * p + lane / 4, col = 32 * wave + 8 * (lane & 3);
        if (c0 + row < hi)
          *reinterpret_cast<uint4*>(op + (c0 + row) * A.o_stride + col) = *reinterpret_cast<const uint4*>(sh.V + row * LV + col);
      }
      __syncthreads();
    }

#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int i = 0; i < 16; ++i) A.S[sbase + (32 * r + 16 * (i / 8) + i % 8) * DV] = S[r][i];
  }
}

namespace {

using ChunkFn = void (*)(const ScanArgs, int64_t);

template <int KIND>
ChunkFn pick(int dk, int dv) {
  if (dk == 128) return dv == 128 ? k_scan_chunk<KIND, 128, 128> : k_scan_chunk<KIND, 128, 64>;
  return dv == 128 ? k_scan_chunk<KIND, 64, 128> : k_scan_chunk<KIND, 64, 64>;
}

}  // namespace

hipError_t launch_scan_chunk(const seed_shape& sh, const ScanArgs& a, hipStream_t s) {
  const int64_t units = static_cast<int64_t>(a.batch) * a.heads;
  const ChunkFn fn = sh.kind == SEED_GDN ? pick<SEED_GDN>(sh.d_k, sh.d_v) : pick<SEED_MAMBA2>(sh.d_k, sh.d_v);
  hipLaunchKernelGGL(fn, dim3(loop_blocks(units)), dim3(sh.d_v * 2), 0, s, a, units);
  return hipGetLastError();
}

}  // namespace seed
