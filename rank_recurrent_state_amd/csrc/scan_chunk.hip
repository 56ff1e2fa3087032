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
// Precision. q, k and v are bf16 and enter the matrix instructions exactly. fp32 operands (the state, T
// and its right-hand side, P, W) enter as sums of three bf16 pieces, each the rounding of what the
// ones before left, which hold all 24 bits; products of two such sums leave out the terms below
// 2^-24. Sums are fp32. The running c is summed in fp64 and kept as two floats, so that differences
// of large sums keep their bits.
//
// Layout. A workgroup has one unit and one wavefront per 32 columns of d_v; a wavefront holds its
// columns of the state, d_k x 32 fp32, in accumulator layout. Rows of the operand tiles are
// permuted so that a lane's 8 consecutive accumulator registers are 8 consecutive rows: the
// accumulators of one product are then the right operand of the next, and S, W and O never leave
// the registers. K, Q, T and P are left operands in LDS; K^T and V come out of row-major tiles
// with the transposing LDS read. As many wavefronts again prepare: rows go from memory straight to LDS two
// chunks ahead, T and P are formed a chunk ahead, so that a chunk costs one barrier and the state's
// wavefronts wait for nothing else.
//
// What bounds it: waits inside a chunk. A state wavefront spends about 940 vector instructions on a GDN chunk
// (half of them on the pieces of S) next to 96 matrix ones, in a chain K S, W, O, S; with one state and one
// preparing wavefront per SIMD to cover its waits, neither unit is full: over 32768 tokens x 32 GDN heads
// the vector unit is busy 50 % of the time and the matrix unit 30 % (Mamba-2, 64 heads: 47 % and 19 %), and
// bank conflicts take 10 % of the LDS cycles. A chunk takes 3.8 us on a compute unit of its own, 32768
// GDN tokens x 32 heads 589 us (1.95 TB/s of rows and states), the same tokens x 64 Mamba-2 heads
// 513 us. 64-token chunks would split S half as often but need 64 accumulators more than the 256
// registers; two GDN workgroups per compute unit fit LDS at 64 x 64 only.
#include "common.hpp"
#include "prompt.hpp"

namespace seed {

namespace {

using bf16x8 = __attribute__((ext_vector_type(8))) __bf16;
using bf16x2 = __attribute__((ext_vector_type(2))) __bf16;
using f32x2 = __attribute__((ext_vector_type(2))) float;
using f32x4 = __attribute__((ext_vector_type(4))) float;
using f32x16 = __attribute__((ext_vector_type(16))) float;
using u32x4 = __attribute__((ext_vector_type(4))) uint32_t;
using s16x4 = __attribute__((ext_vector_type(4))) short;
using lds_s16x4 = __attribute__((address_space(3))) s16x4;

constexpr int C = 32;       // tokens per chunk
constexpr int LT = C + 8;   // row length of the T and P pieces
constexpr int LF = 16 + 4;  // row length of the fp32 block of T
constexpr int kRanked = 128;  // sequences that are put in order of length

// Long prompts of few units, cut into segments (plan_split).
struct Split {
  int32_t pass;    // 0: whole sequences; 1: every segment's A and B; 2: the read-outs
  int32_t tokens;  // of a segment, a multiple of C
  int64_t slots;   // segments at most
  float* A;        // [slots][heads][d_k][d_k]; Mamba-2: [slots][heads], the product of the segment's gates
  float* B;        // [slots][heads][d_k][d_v]
  int32_t* bad;    // [batch][heads][kParts]: whether a join's wavefront met a value that is not finite
};
constexpr int kParts = 64;  // wavefronts of the joins of a unit, at most

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

// The LDS address of a pointer into shared memory: the low half of the generic one.
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p));
}

// Four rows of a row-major 16-bit tile, transposed: lane i of 16 passes the address of row i / 4,
// columns 4 (i % 4) .. + 3 and receives column i, rows 0 .. 3.
__device__ __forceinline__ s16x4 read_tr(const uint16_t* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s16x4*>(static_cast<uintptr_t>(lds_offset(p))));
}

// Rows c0 .. hi - 1 of a row buffer as a bounds-checked buffer: loads behind the last row's `width`
// bytes return zeros. Offsets inside a chunk stay below 2^31 (kChunkStride).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t chunk_rows(const uint16_t* base, int64_t stride, int64_t c0, int64_t hi,
                                                             int width) {
  const int n = static_cast<int>(hi - c0 < C ? hi - c0 : C);
  const int bytes = n > 0 ? static_cast<int>((n - 1) * stride * 2) + width : 0;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint16_t*>(base + c0 * stride), 0, bytes, 0x00027000);
}

// 16 bytes per lane from memory straight to LDS, lane l's at lds + 16 l; lanes outside the buffer
// write zeros. lds is the same for the whole wavefront. The compiler does not see the write: it is
// waited for with wait_loads before the barrier in front of the tile's first use.
__device__ __forceinline__ void load_lds(__amdgpu_buffer_rsrc_t rows, int voffset, int soffset, const uint16_t* lds) {
  const uint32_t to = __builtin_amdgcn_readfirstlane(lds_offset(lds));
  uint32_t m0;  // M0 holds the LDS address; what it held is put back
  asm volatile(
      "s_mov_b32 %0, m0\n\t"
      "s_mov_b32 m0, %1\n\t"
      "s_nop 0\n\t"
      "buffer_load_dwordx4 %2, %3, %4 offen lds\n\t"
      "s_mov_b32 m0, %0"
      : "=&s"(m0)
      : "s"(to), "v"(voffset), "s"(rows), "s"(soffset)
      : "memory");
}
// Waits until at most N of the wavefront's memory operations, the youngest, are under way.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

// By value: a conditional between two elements of an array would put the array in memory.
__device__ __forceinline__ float pick(bool c, float a, float b) { return c ? a : b; }

// x = (I - L)^-1 e_j for a 16 x 16 strictly lower L: lane i of 16 holds row i of L and gets column i of
// the inverse. Step S takes x[S], final by then, out of the rows below: x[R] += L[R][S] x[S], where L[R][S] is
// lane R's L[S], a row broadcast inside the instruction. Outputs are numbered from x[15] down, so the
// text of a step is the first 15 - S lines. A broadcast may read a register two instructions after its
// write at the earliest, which each step's s_nop sees to.
#define SEED_FMAC(out, row) \
  "v_fmac_f32_dpp %" #out ", %[l], %[y] row_newbcast:" #row " row_mask:0xf bank_mask:0xf\n\t"
#define SEED_STEP1 SEED_FMAC(0, 15)
#define SEED_STEP2 SEED_STEP1 SEED_FMAC(1, 14)
#define SEED_STEP3 SEED_STEP2 SEED_FMAC(2, 13)
#define SEED_STEP4 SEED_STEP3 SEED_FMAC(3, 12)
#define SEED_STEP5 SEED_STEP4 SEED_FMAC(4, 11)
#define SEED_STEP6 SEED_STEP5 SEED_FMAC(5, 10)
#define SEED_STEP7 SEED_STEP6 SEED_FMAC(6, 9)
#define SEED_STEP8 SEED_STEP7 SEED_FMAC(7, 8)
#define SEED_STEP9 SEED_STEP8 SEED_FMAC(8, 7)
#define SEED_STEP10 SEED_STEP9 SEED_FMAC(9, 6)
#define SEED_STEP11 SEED_STEP10 SEED_FMAC(10, 5)
#define SEED_STEP12 SEED_STEP11 SEED_FMAC(11, 4)
#define SEED_STEP13 SEED_STEP12 SEED_FMAC(12, 3)
#define SEED_STEP14 SEED_STEP13 SEED_FMAC(13, 2)
#define SEED_STEP15 SEED_STEP14 SEED_FMAC(14, 1)
#define SEED_X(r) "+v"(x[r])
#define SEED_OUT1 SEED_X(15)
#define SEED_OUT2 SEED_OUT1, SEED_X(14)
#define SEED_OUT3 SEED_OUT2, SEED_X(13)
#define SEED_OUT4 SEED_OUT3, SEED_X(12)
#define SEED_OUT5 SEED_OUT4, SEED_X(11)
#define SEED_OUT6 SEED_OUT5, SEED_X(10)
#define SEED_OUT7 SEED_OUT6, SEED_X(9)
#define SEED_OUT8 SEED_OUT7, SEED_X(8)
#define SEED_OUT9 SEED_OUT8, SEED_X(7)
#define SEED_OUT10 SEED_OUT9, SEED_X(6)
#define SEED_OUT11 SEED_OUT10, SEED_X(5)
#define SEED_OUT12 SEED_OUT11, SEED_X(4)
#define SEED_OUT13 SEED_OUT12, SEED_X(3)
#define SEED_OUT14 SEED_OUT13, SEED_X(2)
#define SEED_OUT15 SEED_OUT14, SEED_X(1)
#define SEED_SOLVE(S, n) asm("s_nop 1\n\t" SEED_STEP##n : SEED_OUT##n : [l] "v"(L[S]), [y] "v"(x[S]))
__device__ __forceinline__ void solve16(const float (&L)[16], float (&x)[16]) {
  SEED_SOLVE(0, 15);
  SEED_SOLVE(1, 14);
  SEED_SOLVE(2, 13);
  SEED_SOLVE(3, 12);
  SEED_SOLVE(4, 11);
  SEED_SOLVE(5, 10);
  SEED_SOLVE(6, 9);
  SEED_SOLVE(7, 8);
  SEED_SOLVE(8, 7);
  SEED_SOLVE(9, 6);
  SEED_SOLVE(10, 5);
  SEED_SOLVE(11, 4);
  SEED_SOLVE(12, 3);
  SEED_SOLVE(13, 2);
  SEED_SOLVE(14, 1);
}
#undef SEED_SOLVE
#undef SEED_OUT1
#undef SEED_STEP1
#undef SEED_OUT2
#undef SEED_STEP2
#undef SEED_OUT3
#undef SEED_STEP3
#undef SEED_OUT4
#undef SEED_STEP4
#undef SEED_OUT5
#undef SEED_STEP5
#undef SEED_OUT6
#undef SEED_STEP6
#undef SEED_OUT7
#undef SEED_STEP7
#undef SEED_OUT8
#undef SEED_STEP8
#undef SEED_OUT9
#undef SEED_STEP9
#undef SEED_OUT10
#undef SEED_STEP10
#undef SEED_OUT11
#undef SEED_STEP11
#undef SEED_OUT12
#undef SEED_STEP12
#undef SEED_OUT13
#undef SEED_STEP13
#undef SEED_OUT14
#undef SEED_STEP14
#undef SEED_OUT15
#undef SEED_STEP15
#undef SEED_X
#undef SEED_FMAC

// A copy of x that the compiler takes for a new value.
__device__ __forceinline__ int fresh(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// A tile of C rows of D bf16 values as the loads to LDS lay it out: rows back to back, the 16-byte
// pieces of row r exchanged by an XOR with swz(r). 16 consecutive rows (in any order) then read one
// piece each from 16 different bank groups, and the 4 rows of a transposing read keep apart.
template <int D>
struct Tile {
  static constexpr int PIECES = D / 8;
  uint16_t x[C * D];
  static __device__ __forceinline__ int swz(int r) {
    return D == 128 ? (2 * (r & 7) + ((r >> 3) & 1)) : (2 * ((r >> 1) & 3) + ((r >> 3) & 1));
  }
  // element (r, c), and the 8 that start there when c is a multiple of 8
  __device__ __forceinline__ uint16_t* at(int r, int c) { return x + r * D + ((((c >> 3) ^ swz(r)) << 3) | (c & 7)); }
};

template <int KIND, int DK, int DV>
struct Tiles {
  static constexpr bool DELTA = KIND != SEED_MAMBA2;
  // by the chunk's number modulo 3: one in use, one that T and P are formed of, one arriving
  Tile<DK> K[3], Q[3];
  Tile<DV> V[3];                  // v, then o
  struct alignas(16) Gates {
    float ch[C], cl[C];           // c as a sum of two floats
    float head[C], tail[C];       // 2^c_t, 2^(c_end - c_t)
    float beta[C], g[C];
    float wild;                   // NaN when the chunk has to run token after token, else 0
  } gates[3];
  // by the chunk's number modulo 2
  uint16_t P[2][3][C * LT];
  uint16_t T[DELTA ? 2 : 1][DELTA ? 3 : 1][DELTA ? C * LT : 8];
  float T11[DELTA ? 16 * LF : 4]; // column-major: the lower diagonal block of T
  int32_t len[kRanked], found;    // of ranked_sequence
};

// The 32 rows of a tile at row f0 on, by one wavefront.
template <int D>
__device__ __forceinline__ void fetch_tile(const uint16_t* base, int64_t stride, int64_t f0, int64_t hi, Tile<D>& to) {
  constexpr int RPI = 512 / D;    // rows per load: 64 lanes of 16 bytes
  const auto rows = chunk_rows(base, stride, f0, hi, D * 2);
  const int st = static_cast<int>(stride) * 2;
  const int lane = fresh(threadIdx.x & 63);
#pragma unroll
  for (int j = 0; j < C / RPI; ++j) {
    const int r = lane / (D / 8), piece = (lane % (D / 8)) ^ Tile<D>::swz(j * RPI + r);
    load_lds(rows, r * st + piece * 16, j * RPI * st, to.x + j * 512);
  }
}

// The gates of the chunk at f0: log2 g summed over the chunk, and the weights that follow. sum_gates
// returns the chunk's whole sum, minus infinity where a gate is 0. Products of gates of at most 1 only fall, and
// those that underflow stay 0. Next to a gate above 1 every product has to be a normal number, below 2^100
// here: other chunks, and those with gates that are negative or not finite, are marked and run token
// after token.
__device__ __forceinline__ void load_gates(const ScanArgs& A, int h, int64_t f0, int64_t hi, float& g, float& beta) {
  const int64_t f1 = f0 + (threadIdx.x & 31);
  const int64_t at = (f1 < hi ? f1 : hi - 1) * A.heads + h;
  const float g1 = A.g[at], b1 = A.beta[at];
  g = f1 < hi ? g1 : 1.f;
  beta = f1 < hi ? b1 : 0.f;
}
template <class Gates>
__device__ __forceinline__ double sum_gates(Gates& G, float g, float beta) {
  const int l = fresh(threadIdx.x & 63), l32 = l & 31;
  // g = 0 counts as 2^-200: with no gate above 1, every weight across it underflows to 0, as it should
  const float lg = log2f(g);
  double c = lg < -200.f ? -200.0 : static_cast<double>(lg);
#pragma unroll
  for (int d = 1; d < C; d <<= 1) {
    const double up = __shfl_up(c, d, C);
    if (l32 >= d) c += up;
  }
  const float ch = static_cast<float>(c), cl = static_cast<float>(c - static_cast<double>(ch));
  const double all = __shfl(c, C - 1, C), rest = all - c;
  const float rh = static_cast<float>(rest), rl = static_cast<float>(rest - static_cast<double>(rh));
  const float eh = exp2f(ch), et = exp2f(rh);
  if (l < C) {
    G.ch[l] = ch;
    G.cl[l] = cl;
    G.head[l] = fmaf(eh, 0.693147181f * cl, eh);
    G.tail[l] = fmaf(et, 0.693147181f * rl, et);
    G.beta[l] = beta;
    G.g[l] = g;
  }
  const bool wild = __any(!(g >= 0.f && g < __builtin_inff())) || (__any(g > 1.f) && __any(c < -50.0 || c > 50.0));
  const bool none = __any(g == 0.f);
  if (l == 0) G.wild = wild ? __builtin_nanf("") : 0.f;
  return none ? -__builtin_inf() : all;
}

// 2^(c_t - c_s) for t = l32 and the 16 s of the lane's accumulator registers.
template <class Gates>
__device__ __forceinline__ void weights(const Gates& G, int l32, int half, float (&e)[16]) {
  const float th = G.ch[l32], tl = G.cl[l32];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int s = 16 * (i / 8) + 8 * half + i % 8;
    e[i] = __builtin_amdgcn_exp2f((th - G.ch[s]) + (tl - G.cl[s]));
  }
}

// P (Mamba-2: times diag(beta)) in three pieces, by one wavefront.
template <bool DELTA, int DK, class Gates>
__device__ __forceinline__ void form_P(Tile<DK>& K, Tile<DK>& Q, const Gates& G, uint16_t (&P)[3][C * LT]) {
  const int lane = fresh(threadIdx.x & 63), l32 = lane & 31, half = lane >> 5, prow = perm(l32);
  f32x16 acc = {};
#pragma unroll
  for (int ks = 0; ks < DK / 16; ++ks)
    acc = mma(frag(K.at(prow, 16 * ks + 8 * half)), frag(Q.at(l32, 16 * ks + 8 * half)), acc);
  float e[16];
  weights(G, l32, half, e);
#pragma unroll
  for (int s8 = 0; s8 < 2; ++s8) {
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int s = 16 * s8 + 8 * half + j;
      float w = acc[8 * s8 + j] * e[8 * s8 + j];
      if constexpr (!DELTA) w *= G.beta[s];
      x[j] = s <= l32 ? w : 0.f;
    }
    bf16x8 pc[3];
    split<3>(x, pc);
#pragma unroll
    for (int n = 0; n < 3; ++n) *reinterpret_cast<bf16x8*>(P[n] + l32 * LT + 16 * s8 + 8 * half) = pc[n];
  }
}

// (I + L)^-1 diag(beta) in three pieces, by one wavefront. The block above the diagonal stays zero.
template <int DK, class Gates>
__device__ __forceinline__ void form_T(Tile<DK>& K, const Gates& G, uint16_t (&T)[3][C * LT], float* T11) {
  const int lane = fresh(threadIdx.x & 63), l32 = lane & 31, half = lane >> 5, prow = perm(l32);
  f32x16 acc = {};
#pragma unroll
  for (int ks = 0; ks < DK / 16; ++ks)
    acc = mma(frag(K.at(prow, 16 * ks + 8 * half)), frag(K.at(l32, 16 * ks + 8 * half)), acc);
  float e[16];
  weights(G, l32, half, e);
  const float bt = G.beta[l32];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int s = 16 * (i / 8) + 8 * half + i % 8;
    e[i] = s < l32 ? -bt * (acc[i] * e[i]) : 0.f;  // -L
  }
  // row l32 of its diagonal block, from both halves of the wavefront
  float Lr[16], x[16];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t z = __float_as_uint(pick(l32 & 16, e[8 + j], e[j]));
    const auto r = __builtin_amdgcn_permlane32_swap(z, z, false, false);
    Lr[j] = __uint_as_float(r[0]);
    Lr[8 + j] = __uint_as_float(r[1]);
  }
#pragma unroll
  for (int t = 0; t < 16; ++t) x[t] = t == (l32 & 15) ? 1.f : 0.f;
  solve16(Lr, x);  // both halves: lane l32 has column l32 % 16 of block l32 / 16
  // the block below the diagonal: T11 (-L10 T00) in fp32 matrix instructions, whose k slot lane / 16 of
  // step i is taken as 4 (lane / 16) + i
  const int r16 = lane & 15, g4 = lane >> 4;
  if (l32 & 16) {
#pragma unroll
    for (int t = 0; t < 16; t += 4)
      *reinterpret_cast<f32x4*>(T11 + r16 * LF + t) = f32x4{x[t], x[t + 1], x[t + 2], x[t + 3]};
  }
  f32x4 m1 = {}, m2 = {};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a0 = e[i], a1 = e[4 + i];  // -L10[r16][8 half + i], [8 half + 4 + i] in the odd rows of lanes
    lane_swap16(a0, a1);             // a1: -L10[r16][4 g4 + i]
    float b0 = pick(half, x[8 + i], x[i]), b1 = pick(half, x[12 + i], x[4 + i]);
    lane_swap16(b0, b1);             // b0: T00[4 g4 + i][r16]
    m1 = __builtin_amdgcn_mfma_f32_16x16x4f32(a1, b0, m1, 0, 0, 0);
  }
  wave_lds_sync();
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m2 = __builtin_amdgcn_mfma_f32_16x16x4f32(T11[(4 * g4 + i) * LF + r16], m1[i], m2, 0, 0, 0);
  // each half writes 8 rows of the diagonal blocks' columns, then the block below
  const int blk = l32 & 16;
  float y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = pick(half, x[8 + j], x[j]) * bt;
  bf16x8 pc[3];
  split<3>(y, pc);
#pragma unroll
  for (int n = 0; n < 3; ++n)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      T[n][(blk + 8 * half + j) * LT + l32] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(pc[n][j]));
  const float b16 = G.beta[r16];
#pragma unroll
  for (int j = 0; j < 8; ++j) y[j] = j < 4 ? m2[j & 3] * b16 : 0.f;
  split<3>(y, pc);
#pragma unroll
  for (int n = 0; n < 3; ++n)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      T[n][(16 + 4 * g4 + j) * LT + r16] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(pc[n][j]));
  wave_lds_sync();  // T11 has been read
}

}  // namespace

// The sequence that is `rank`-th by length, longest first (the earlier of two equal ones first); with
// more than kRanked sequences simply sequence `rank`. Workgroups start in block order, and a long
// sequence started last would be run by a few of them alone: with read-outs in 16 bits, 16 prompts of 0
// to 3646 tokens x 64 Mamba-2 heads took 528 us in the order given and 460 us longest first. Called by the whole workgroup.
template <int NT>
__device__ __forceinline__ int ranked_sequence(const ScanArgs& A, int rank, int32_t (&len)[kRanked], int32_t& found) {
  if (A.batch > kRanked) return rank;
  __syncthreads();  // the buffers' last use
  for (int i = threadIdx.x; i < A.batch; i += NT) {
    int64_t lo, hi;
    sequence_rows(A.offsets, i, A.tokens, lo, hi);
    len[i] = static_cast<int32_t>(hi - lo);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < A.batch; i += NT) {
    const int32_t mine = len[i];
    int before = 0;
    for (int k = 0; k < A.batch; ++k) before += len[k] > mine || (len[k] == mine && k < i);
    if (before == rank) found = i;
  }
  __syncthreads();
  return found;
}

// Segments of a sequence with `rows` rows.
__device__ __forceinline__ int segments_of(const Split& W, int64_t rows) {
  return rows > W.tokens ? static_cast<int>((rows + W.tokens - 1) / W.tokens) : 1;
}
// The sequence, the segment and its rows that slot `slot` stands for, the sequences' segments counted one
// after the other; A.batch when there are fewer. The same for all threads.
__device__ __forceinline__ int find_segment(const ScanArgs& A, const Split& W, int64_t slot, int64_t& lo, int64_t& hi,
                                            int& seg, int& segs) {
  int b = 0;
  for (; b < A.batch; ++b) {
    sequence_rows(A.offsets, b, A.tokens, lo, hi);
    segs = segments_of(W, hi - lo);
    if (slot < segs) break;
    slot -= segs;
  }
  seg = static_cast<int>(slot);
  if (b < A.batch) {
    lo += seg * static_cast<int64_t>(W.tokens);
    if (hi > lo + W.tokens) hi = lo + W.tokens;
  }
  return __builtin_amdgcn_readfirstlane(b);
}
// Sequence b's first slot, number of segments and rows.
__device__ __forceinline__ int first_segment(const ScanArgs& A, const Split& W, int b, int64_t& base, int64_t& lo, int64_t& hi) {
  base = 0;
  for (int i = 0; i < b; ++i) {
    sequence_rows(A.offsets, i, A.tokens, lo, hi);
    base += segments_of(W, hi - lo);
  }
  sequence_rows(A.offsets, b, A.tokens, lo, hi);
  return segments_of(W, hi - lo);
}

// Wavefronts 0 .. NW - 1 hold 32 columns of the state each and run a chunk while the NH others prepare:
// T and P of the next chunk, and rows and gates of the one after it. Preparing in the state's own
// wavefronts instead, with two workgroups per compute unit, took 704 us where this took 673 (32768 GDN
// tokens, at the same stage) and 1436 where this took 936 (one 8192-token prompt, uncut).
//
// The launch bound is the wavefronts of a SIMD that LDS lets run together, two at most: DV = 128 brings two,
// DV = 64 one, or two where a second workgroup fits. One leaves 512 registers to a wavefront, two 256.
template <int KIND, int DK, int DV>
constexpr int kWavesPerSimd = DV == 64 && 2 * sizeof(Tiles<KIND, DK, DV>) > 160 * 1024 ? 1 : 2;
template <int KIND, int DK, int DV>
__global__ __launch_bounds__(DV * 4, (kWavesPerSimd<KIND, DK, DV>)) void k_scan_chunk(const ScanArgs A, const Split W, int64_t items) {
  using TL = Tiles<KIND, DK, DV>;
  constexpr bool DELTA = TL::DELTA;
  constexpr int NW = DV / 32, NH = NW, NT = (NW + NH) * 64;
  constexpr int RT = DK / 32;                 // row tiles of the state
  __shared__ TL sh;

  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int role = wave - NW;                 // of the helpers
  // which helper does what
  constexpr int kT = 0, kP = 1, kK = NH == 4 ? 2 : (DELTA ? 1 : 0), kQV = NH == 4 ? 3 : kK, kG = kK;

  if constexpr (DELTA) {  // the block of T above the diagonal
    for (int i = threadIdx.x; i < 2 * 3 * 16 * 16; i += NT)
      sh.T[i / 768][i / 256 % 3][(i / 16 % 16) * LT + 16 + i % 16] = 0;
  }

  for (int64_t item = blockIdx.x; item < items; item += gridDim.x) {
    // Consecutive workgroups go to the 8 XCDs in turn. Heads of one key head are kept key_heads apart, on
    // the same XCD where key_heads is a multiple of 8, so that they share the rows of q and k in its L2.
    const int place = static_cast<int>(item % A.heads), share = A.heads / A.key_heads;
    const int kh = place % A.key_heads, h = kh * share + place / A.key_heads;
    int b;                       // sequence
    int64_t lo, hi;              // its rows to run over
    const float* init = nullptr; // the state to start from (nullptr: zeros, or the identity when v counts as zero)
    float* dest;                 // where the state goes (nullptr: nowhere)
    bool out = true, has_v = true;  // without read-outs, q and P are whatever LDS holds and o is dropped
    if (W.pass == 0) {
      b = __builtin_amdgcn_readfirstlane(ranked_sequence<NT>(A, static_cast<int>(item / A.heads), sh.len, sh.found));
      sequence_rows(A.offsets, b, A.tokens, lo, hi);
      const int64_t at = (static_cast<int64_t>(b) * A.heads + h) * (DK * DV);
      if (A.S0 != nullptr) init = A.S0 + at;
      dest = A.S + at;
    } else {
      int64_t slot = item / A.heads;
      if (DELTA && W.pass == 1) {
        has_v = (slot & 1) == 0;
        slot >>= 1;
      }
      int seg, segs;
      b = find_segment(A, W, slot, lo, hi, seg, segs);
      if (b >= A.batch) continue;
      const int64_t at = (static_cast<int64_t>(b) * A.heads + h) * (DK * DV), in_ws = (slot * A.heads + h) * (DK * DV);
      const bool last = seg == segs - 1;
      if (W.pass == 1) {
        // the first segment is run for good; of the others all but the last leave their matrices
        if (seg == 0 ? !has_v : last) continue;
        if (seg == 0 && A.S0 != nullptr) init = A.S0 + at;
        out = seg == 0;
        dest = seg == 0 && last ? A.S + at : (has_v ? W.B : W.A) + in_ws;
      } else {
        if (seg == 0) continue;
        init = W.B + in_ws - static_cast<int64_t>(A.heads) * (DK * DV);
        dest = last ? A.S + at : nullptr;
        // A S + B is not the state where either is infinite or NaN (0 times infinity, a segment's A that
        // overflows next to a state of zeros): then one workgroup runs all that follows the first segment.
        constexpr int kJoins = DELTA ? (DV / 32) * (DK / 32) : DK * DV / 256;
        const int32_t* bad = W.bad + (static_cast<int64_t>(b) * A.heads + h) * kParts;
        const int lane = threadIdx.x & 63;
        if (__any(lane < kJoins && bad[lane] != 0)) {
          if (seg != 1) continue;
          int64_t first;
          sequence_rows(A.offsets, b, A.tokens, first, hi);
          dest = A.S + at;
        }
      }
    }
    lo = __builtin_amdgcn_readfirstlane(static_cast<int>(lo));  // rows are below 2^31
    hi = __builtin_amdgcn_readfirstlane(static_cast<int>(hi));
    const int n = static_cast<int>((hi - lo + C - 1) / C);  // chunks

    const uint16_t* __restrict__ qp = static_cast<const uint16_t*>(A.q) + static_cast<int64_t>(kh) * DK;
    const uint16_t* __restrict__ kp = static_cast<const uint16_t*>(A.k) + static_cast<int64_t>(kh) * DK;
    const uint16_t* __restrict__ vp = static_cast<const uint16_t*>(A.v) + static_cast<int64_t>(h) * DV;
    uint16_t* __restrict__ op = static_cast<uint16_t*>(A.o) + static_cast<int64_t>(h) * DV;

    if (role >= 0) {
      // ---- helpers ------------------------------------------------------------------------------------
      // chunk j's rows go to buffer `to`, its gates are loaded and summed
      float g = 1.f, beta = 0.f;
      double decay = 0;  // log2 of the product of all gates
      auto fetch = [&](int j, int to) {
        const int64_t f0 = lo + static_cast<int64_t>(j) * C;
        if (role == kG) load_gates(A, h, f0, hi, g, beta);
        if (role == kK) fetch_tile<DK>(kp, A.k_stride, f0, hi, sh.K[to]);
        if (role == kQV) {
          if (out) fetch_tile<DK>(qp, A.q_stride, f0, hi, sh.Q[to]);
          fetch_tile<DV>(vp, A.v_stride, f0, has_v ? hi : f0, sh.V[to]);
        }
        if (role == kG) decay += sum_gates(sh.gates[to], g, beta);
      };
      if (n > 0) fetch(0, 0);
      wait_loads<0>();
      __syncthreads();
      int next = 0, far = 1;  // buffers of chunks j + 1 and j + 2
      for (int j = -1; j < n; ++j) {
        if (j + 2 < n) fetch(j + 2, far);
        if (j + 1 < n) {
          if constexpr (DELTA) {
            if (role == kT) form_T<DK>(sh.K[next], sh.gates[next], sh.T[(j + 1) & 1], sh.T11);
          }
          if (role == kP && out) form_P<DELTA, DK>(sh.K[next], sh.Q[next], sh.gates[next], sh.P[(j + 1) & 1]);
        }
        wait_loads<0>();
        __syncthreads();
        next = far;
        far = far == 2 ? 0 : far + 1;
      }
      if (!DELTA && W.pass == 1 && role == kG && (threadIdx.x & 63) == 0)
        W.A[item / A.heads * A.heads + h] = static_cast<float>(exp2(decay));
      continue;
    }

    // ---- the state: register i of row tile r is row 32 r + 16 (i / 8) + 8 half + i % 8, column 32 wave + l32
    f32x16 S[RT];
    constexpr int SB = DK * DV * 4;
    const int s_at = (8 * ((threadIdx.x & 63) >> 5) * DV + 32 * wave + (threadIdx.x & 31)) * 4;
    {
      // without a state to start from, the loads are outside their buffer and give zeros
      const auto sr = __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(init), 0, init != nullptr ? SB : 0, 0x00027000);
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          S[r][i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(sr, s_at, (32 * r + 16 * (i / 8) + i % 8) * DV * 4, 0));
    }
    if constexpr (DELTA) {
      // the identity: the lane's column meets the diagonal in one register of one half
      const int at = has_v ? -1 : 32 * wave + (threadIdx.x & 31) - 8 * ((threadIdx.x & 63) >> 5);
#pragma unroll
      for (int r = 0; r < RT; ++r)
#pragma unroll
        for (int i = 0; i < 16; ++i) S[r][i] = at == 32 * r + 16 * (i / 8) + i % 8 ? 1.f : S[r][i];
    }
    __syncthreads();  // chunk 0's rows and gates
    __syncthreads();  // its T and P

    int now = 0;
    for (int ci = 0; ci < n; ++ci, now = now == 2 ? 0 : now + 1) {
      const int64_t c0 = lo + static_cast<int64_t>(ci) * C;
      // lane numbers that the compiler takes for new ones in every chunk, so that the addresses made
      // of them cost an instruction each instead of a register each
      const int lane = fresh(threadIdx.x & 63);
      const int l32 = lane & 31, half = lane >> 5;
      const int prow = perm(l32);
      auto& K = sh.K[now];
      auto& Q = sh.Q[now];
      auto& V = sh.V[now];
      auto& G = sh.gates[now];
      auto& P = sh.P[ci & 1];

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
          const bf16x8 aq = frag(Q.at(prow, col));
          bf16x8 pc[3], ak;
          split<3>(x, pc);
          if constexpr (DELTA) ak = frag(K.at(prow, col));
#pragma unroll
          for (int n = 2; n >= 0; --n) {
            if constexpr (DELTA) ks = mma(ak, pc[n], ks);
            qs = mma(aq, pc[n], qs);
          }
        }
      // v in accumulator layout, and as the bf16 right operand it already is
      bf16x8 vb[2];
      const int vr4 = 8 * half + (lane & 15) / 4, vc4 = 32 * wave + (lane & 16) + 4 * (lane & 3);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const s16x4 x0 = read_tr(V.at(vr4 + 16 * s, vc4)), x1 = read_tr(V.at(vr4 + 16 * s + 4, vc4));
        const __attribute__((ext_vector_type(8))) short x = {x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
        vb[s] = __builtin_bit_cast(bf16x8, x);
      }

      // ---- W ----------------------------------------------------------------------------------------
      f32x16 w;
      float hd[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) hd[i] = G.head[16 * (i / 8) + 8 * half + i % 8];
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
          for (int n = 0; n < 3; ++n) tp[n] = frag(sh.T[ci & 1][n] + prow * LT + 16 * s + 8 * half);
          w = mma(tp[2], rp[0], w);
          w = mma(tp[1], rp[1], w);
          w = mma(tp[0], rp[2], w);
          w = mma(tp[1], rp[0], w);
          w = mma(tp[0], rp[1], w);
          w = mma(tp[0], rp[0], w);
        }
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = static_cast<float>(vb[i / 8][i % 8]) * G.beta[16 * (i / 8) + 8 * half + i % 8];
      }

      // A value that is not finite would reach the tokens before its own through the zeros of T and P:
      // such a chunk runs token after token instead, as does one whose gates are marked.
      // W has met the state in GDN; in Mamba-2 any row of Q S shows a state that is not finite.
      float fin = G.wild;
      if constexpr (!DELTA) fin = out ? fmaf(qs[0], 0.f, fin) : fin;
#pragma unroll
      for (int i = 0; i < 16; ++i) fin = fmaf(w[i], 0.f, fin);
      if (__builtin_expect(__any(!(fin == 0.f)), 0)) {
        const int live = static_cast<int>(hi - c0 < C ? hi - c0 : C);
#pragma unroll 1
        for (int t = 0; t < live; ++t) {
          const float gt = G.g[t];
          float sk = 0.f, sq = 0.f, kq = 0.f;
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int s8 = 0; s8 < 2; ++s8) {
              const int col = 32 * r + 16 * s8 + 8 * half;
              const bf16x8 kv = frag(K.at(t, col)), qv = frag(Q.at(t, col));
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float kf = static_cast<float>(kv[j]), qf = static_cast<float>(qv[j]);
                S[r][8 * s8 + j] *= gt;
                sk = fmaf(kf, S[r][8 * s8 + j], sk);
                sq = fmaf(qf, S[r][8 * s8 + j], sq);
                kq = fmaf(kf, qf, kq);
              }
              __builtin_amdgcn_sched_barrier(0);  // one piece of k and q in registers at a time
            }
          sk += __shfl_xor(sk, 32, 64);
          sq += __shfl_xor(sq, 32, 64);
          kq += __shfl_xor(kq, 32, 64);
          float x = bf16_to_f32(*V.at(t, 32 * wave + l32));
          if constexpr (DELTA) x -= sk;
          x *= G.beta[t];
#pragma unroll
          for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int s8 = 0; s8 < 2; ++s8) {
              const bf16x8 kv = frag(K.at(t, 32 * r + 16 * s8 + 8 * half));
#pragma unroll
              for (int j = 0; j < 8; ++j) S[r][8 * s8 + j] = fmaf(static_cast<float>(kv[j]), x, S[r][8 * s8 + j]);
              __builtin_amdgcn_sched_barrier(0);
            }
          wave_lds_sync();  // both halves have read v
          if (half == 0) *V.at(t, 32 * wave + l32) = f32_to_bf16(fmaf(kq, x, sq));
        }
      } else {
        // ---- O = H Q S + P W --------------------------------------------------------------------------
        f32x16 o;
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = hd[i] * qs[i];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          bf16x8 pp[3];
#pragma unroll
          for (int n = 0; n < 3; ++n) pp[n] = frag(P[n] + prow * LT + 16 * s + 8 * half);
          if constexpr (DELTA) {
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = w[8 * s + j];
            bf16x8 wp[3];
            split<3>(x, wp);
            o = mma(pp[2], wp[0], o);
            o = mma(pp[1], wp[1], o);
            o = mma(pp[0], wp[2], o);
            o = mma(pp[1], wp[0], o);
            o = mma(pp[0], wp[1], o);
            o = mma(pp[0], wp[0], o);
          } else {
#pragma unroll
            for (int n = 2; n >= 0; --n) o = mma(pp[n], vb[s], o);
          }
        }
        // ---- S = 2^(c_end) S + K^T diag(tail) W ----------------------------------------------------------
        const float ge = G.head[C - 1];
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int i = 0; i < 16; ++i) S[r][i] *= ge;
        // lane i of 16 passes row i / 4 of 4 tokens and the channels that perm puts at 4 (i % 4)
        const int kr4 = 8 * half + (lane & 15) / 4, kc4 = perm(4 * (lane & 3)) + (lane & 16);
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          bf16x8 ka[RT];
#pragma unroll
          for (int r = 0; r < RT; ++r) {
            const s16x4 x0 = read_tr(K.at(kr4 + 16 * s, kc4 + 32 * r)), x1 = read_tr(K.at(kr4 + 16 * s + 4, kc4 + 32 * r));
            const __attribute__((ext_vector_type(8))) short y = {x0[0], x0[1], x0[2], x0[3], x1[0], x1[1], x1[2], x1[3]};
            ka[r] = __builtin_bit_cast(bf16x8, y);
          }
          float x[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = w[8 * s + j] * G.tail[16 * s + 8 * half + j];
          bf16x8 wp[3];
          split<3>(x, wp);
#pragma unroll
          for (int n = 2; n >= 0; --n)
#pragma unroll
            for (int r = 0; r < RT; ++r) S[r] = mma(ka[r], wp[n], S[r]);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
          *V.at(16 * (i / 8) + 8 * half + i % 8, 32 * wave + l32) = f32_to_bf16(o[i]);
      }
      // ---- the read-outs: a wavefront's 32 columns of a row are 64 bytes, 16 per lane ----------------
      wave_lds_sync();
      const auto orow = chunk_rows(op, A.o_stride, c0, out ? hi : c0, DV * 2);  // stores outside are dropped
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        const int o_at = (lane / 4 * static_cast<int>(A.o_stride) + 32 * wave + 8 * (lane & 3)) * 2;
        const u32x4 x = *reinterpret_cast<const u32x4*>(V.at(16 * p + lane / 4, 32 * wave + 8 * (lane & 3)));
        __builtin_amdgcn_raw_buffer_store_b128(x, orow, o_at, p * 16 * static_cast<int>(A.o_stride) * 2, 0);
      }
      __syncthreads();
    }

    const auto sr = __builtin_amdgcn_make_buffer_rsrc(dest, 0, dest != nullptr ? SB : 0, 0x00027000);
#pragma unroll
    for (int r = 0; r < RT; ++r)
#pragma unroll
      for (int i = 0; i < 16; ++i)
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(S[r][i]), sr, s_at, (32 * r + 16 * (i / 8) + i % 8) * DV * 4, 0);
  }
}

// Between the passes: the states before the segments. B of a sequence's first segment is the state
// after it; S_seg = A_seg S_(seg - 1) + B_seg takes the place of B_seg, up to the last segment but one.
// A workgroup has 32 columns of one unit, a wavefront 32 rows of them; fp32 matrix instructions.
template <int DK, int DV>
__global__ __launch_bounds__(DK * 2) void k_join_delta(const ScanArgs A, const Split W) {
  constexpr int LS = 32 + 1;
  __shared__ float Sh[DK * LS];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, l32 = lane & 31, half = lane >> 5;
  const int h = blockIdx.x / (DV / 32) % A.heads, b = blockIdx.x / (DV / 32) / A.heads;
  const int col = blockIdx.x % (DV / 32) * 32 + l32;
  int64_t base, lo, hi;
  const int segs = first_segment(A, W, b, base, lo, hi);
  // the next segment's matrices are on their way while one product runs
  f32x4 a[DK / 8], na[DK / 8];
  f32x16 acc, nb;  // register i is row 32 wave + 8 (i / 4) + 4 half + i % 4
  auto load = [&](int seg) {
    const int64_t slot = (base + seg) * A.heads + h;
    const float* Bs = W.B + slot * (DK * DV);
#pragma unroll
    for (int i = 0; i < 16; ++i) nb[i] = Bs[(32 * wave + 8 * (i / 4) + 4 * half + i % 4) * DV + col];
    const float* As = W.A + slot * (DK * DK) + (32 * wave + l32) * DK + 4 * half;
    if (seg > 0) {  // the first segment has no A
#pragma unroll
      for (int k = 0; k < DK / 8; ++k) na[k] = *reinterpret_cast<const f32x4*>(As + 8 * k);
    }
  };
  const int64_t room = W.slots - base;
  const int n = static_cast<int>(segs - 1 < room ? segs - 1 : room);
  if (n > 0) load(0);
  float fin = 0.f;  // NaN once a state is not finite
  for (int seg = 0; seg < n; ++seg) {
    acc = nb;
#pragma unroll
    for (int k = 0; k < DK / 8; ++k) a[k] = na[k];
    if (seg + 1 < n) load(seg + 1);
    if (seg > 0) {
#pragma unroll
      for (int k = 0; k < DK / 8; ++k)  // k slot `half` of step i is row 8 k + 4 half + i
#pragma unroll
        for (int i = 0; i < 4; ++i)
          acc = __builtin_amdgcn_mfma_f32_32x32x2f32(a[k][i], Sh[(8 * k + 4 * half + i) * LS + l32], acc, 0, 0, 0);
      __syncthreads();  // the old state has been read
    }
    float* Bs = W.B + ((base + seg) * A.heads + h) * (DK * DV);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int row = 32 * wave + 8 * (i / 4) + 4 * half + i % 4;
      Sh[row * LS + l32] = acc[i];
      if (seg > 0) Bs[row * DV + col] = acc[i];
      fin = fmaf(acc[i], 0.f, fin);
    }
    __syncthreads();
  }
  const bool bad = __any(!(fin == 0.f));
  if (lane == 0) W.bad[(static_cast<int64_t>(b) * A.heads + h) * kParts + blockIdx.x % (DV / 32) * (DK / 32) + wave] = bad;
}

// The same where A_seg is the product of the segment's gates: a thread follows 4 elements of a state.
template <int DK, int DV>
__global__ __launch_bounds__(256) void k_join_scalar(const ScanArgs A, const Split W) {
  constexpr int PARTS = DK * DV / 1024;
  const int unit = blockIdx.x / PARTS, h = unit % A.heads, b = unit / A.heads;
  const int at = blockIdx.x % PARTS * 1024 + 4 * threadIdx.x;
  int64_t base, lo, hi;
  const int segs = first_segment(A, W, b, base, lo, hi);
  f32x4 S = {};
  float fin = 0.f;  // NaN once a state is not finite
#pragma unroll 4
  for (int seg = 0; seg + 1 < segs && base + seg < W.slots; ++seg) {
    const int64_t slot = (base + seg) * A.heads + h;
    f32x4* Bs = reinterpret_cast<f32x4*>(W.B + slot * (DK * DV) + at);
    const f32x4 x = *Bs;
    const float a = W.A[slot];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      S[e] = seg > 0 ? fmaf(a, S[e], x[e]) : x[e];
      fin = fmaf(S[e], 0.f, fin);
    }
    if (seg > 0) *Bs = S;
  }
  const bool bad = __any(!(fin == 0.f));
  if ((threadIdx.x & 63) == 0) W.bad[static_cast<int64_t>(unit) * kParts + blockIdx.x % PARTS * 4 + (threadIdx.x >> 6)] = bad;
}

namespace {

using ChunkFn = void (*)(const ScanArgs, const Split, int64_t);

template <int KIND>
ChunkFn pick_dims(int dk, int dv) {
  if (dk == 128) return dv == 128 ? k_scan_chunk<KIND, 128, 128> : k_scan_chunk<KIND, 128, 64>;
  return dv == 128 ? k_scan_chunk<KIND, 64, 128> : k_scan_chunk<KIND, 64, 64>;
}

constexpr int64_t kCUs = 256;

// Few units leave most of the chip idle while each runs its chunks one after the other. Such prompts are
// cut into segments: the state after a segment is A S + B with S the state before it, so one pass forms
// A and B of all segments side by side (A: the recurrence from the identity with v = 0; a product of
// gates for Mamba-2), the states between them follow, and a second pass gives the read-outs.
// n = slots / units + 1 segments fill the chip once with the read-outs, and once (Mamba-2) or twice (GDN, whose
// A and B are two runs) with the first pass: 2 / n or 3 / n of the serial time, and about 50 us. Three
// segments of Mamba-2 with d_v = 64 gain less, since the two workgroups of a compute unit slow each other.
// Measured, cut and whole, us:           1024 tokens   2048        4096        8192
//   GDN 128 x 128,    16 units               90, 129   107, 247   173, 484   262, 958
//                     64                    133, 130   193, 250   339, 487   632, 968
//                     85 (n = 4)            145, 130   232, 251   413, 487   770, 965
//                    128 (n = 3)            166, 131   287, 251   525, 490  1004, 968
//   Mamba-2 128 x 64, 16                     58, 89     62, 171    67, 337    95, 668
//                    128                     85, 92    123, 175   222, 344   419, 680
//                    170 (n = 4)             89, 92    147, 176   268, 344   510, 680
//                    176 (n = 3)            108, 95    183, 177   344, 345   662, 679
//                    256                    107, 93    188, 178   348, 347   670, 682
//           128 x 128, 128 (n = 3)           88, 95    145, 180   265, 351   520, 692
// and 512 tokens are always faster whole (GDN 80, 69; Mamba-2 56, 48).
Split plan_split(const seed_shape& sh, int64_t tokens) {
  Split w{};
  const bool delta = sh.kind != SEED_MAMBA2;
  const int64_t units = static_cast<int64_t>(sh.batch) * sh.heads, mean = tokens / sh.batch;
  // Workgroups that fit the chip at once. Two of GDN with 64 x 64 would fit a compute unit too; its rule was
  // measured with one.
  const int64_t slots = kCUs * (!delta && sh.d_v == 64 ? 2 : 1);
  const int64_t n = slots / units + 1;
  if (delta && sh.d_k != sh.d_v) return w;  // A is run as a state of d_k x d_k
  const int64_t least = delta ? (n < 9 ? 2048 : 1024) : (n == 3 && sh.d_v == 64 ? 4096 : 1024);
  if (n < (delta ? 4 : 3) || mean < least) return w;
  int64_t seg = (mean + n - 1) / n;
  seg = (seg < 256 ? 256 : seg) + C - 1;
  w.tokens = static_cast<int32_t>(seg / C * C);
  w.slots = tokens / w.tokens + sh.batch;
  return w;
}

int64_t floats_of_B(const seed_shape& sh, const Split& w) { return w.slots * sh.heads * sh.d_k * sh.d_v; }
int64_t floats_of_A(const seed_shape& sh, const Split& w) {
  return w.slots * sh.heads * (sh.kind == SEED_MAMBA2 ? 1 : sh.d_k * sh.d_k);
}

template <int DK, int DV>
void join(const seed_shape& sh, const ScanArgs& a, const Split& w, hipStream_t s) {
  const unsigned units = static_cast<unsigned>(a.batch * a.heads);
  if (sh.kind == SEED_MAMBA2) k_join_scalar<DK, DV><<<dim3(units * (DK * DV / 1024)), dim3(256), 0, s>>>(a, w);
  else k_join_delta<DK, DV><<<dim3(units * (DV / 32)), dim3(DK * 2), 0, s>>>(a, w);
}

}  // namespace

size_t scan_chunk_workspace(const seed_shape& sh, int64_t tokens) {
  const Split w = plan_split(sh, tokens);
  if (w.slots == 0) return 0;
  return static_cast<size_t>(floats_of_B(sh, w) + floats_of_A(sh, w)) * sizeof(float) +
         static_cast<size_t>(sh.batch) * sh.heads * kParts * sizeof(int32_t);
}

hipError_t launch_scan_chunk(const seed_shape& sh, const ScanArgs& a, hipStream_t s) {
  const ChunkFn fn = sh.kind == SEED_GDN ? pick_dims<SEED_GDN>(sh.d_k, sh.d_v) : pick_dims<SEED_MAMBA2>(sh.d_k, sh.d_v);
  const dim3 threads(sh.d_v * 4);
  Split w = plan_split(sh, a.tokens);
  if (w.slots == 0) {
    const int64_t units = static_cast<int64_t>(a.batch) * a.heads;
    hipLaunchKernelGGL(fn, dim3(loop_blocks(units)), threads, 0, s, a, w, units);
    return hipGetLastError();
  }
  const bool delta = sh.kind != SEED_MAMBA2;
  w.B = static_cast<float*>(a.ws);
  w.A = w.B + floats_of_B(sh, w);
  w.bad = reinterpret_cast<int32_t*>(w.A + floats_of_A(sh, w));
  const int64_t items = w.slots * a.heads;
  w.pass = 1;
  hipLaunchKernelGGL(fn, dim3(loop_blocks(items * (delta ? 2 : 1))), threads, 0, s, a, w, items * (delta ? 2 : 1));
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (sh.d_k == 128) sh.d_v == 128 ? join<128, 128>(sh, a, w, s) : join<128, 64>(sh, a, w, s);
  else sh.d_v == 128 ? join<64, 128>(sh, a, w, s) : join<64, 64>(sh, a, w, s);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  w.pass = 2;
  hipLaunchKernelGGL(fn, dim3(loop_blocks(items)), threads, 0, s, a, w, items);
  return hipGetLastError();
}

}  // namespace seed
