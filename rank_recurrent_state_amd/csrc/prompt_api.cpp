// C ABI of the prompt path: the short convolution, the gated scan of packed prompts and the norm
// of packed rows. As in api.cpp, every entry point validates on the host before anything is
// enqueued, never synchronises and allocates nothing.
#include <hip/hip_runtime.h>

#include <initializer_list>

#include "../../include/seed.h"
#include "prompt.hpp"

namespace {

constexpr int64_t kMostRows = (int64_t{1} << 31) - 1;  // offsets are int32
constexpr int64_t kMostStride = int64_t{1} << 40;      // a row's bytes stay far inside 64 bits
constexpr int64_t kMostBytes = int64_t{1} << 56;       // of a buffer, so that its offsets and end stay inside 64 bits

bool io_ok(int32_t d) { return d == SEED_F32 || d == SEED_BF16 || d == SEED_F16; }
int64_t io_bytes(int32_t d) { return d == SEED_F32 ? 4 : 2; }
int hip_status(hipError_t e) { return e == hipSuccess ? SEED_OK : SEED_ERR_HIP; }
bool aligned(const void* p, int64_t to) { return (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(to - 1)) == 0; }
bool stride_ok(int64_t stride, int64_t width) { return stride >= width && stride <= kMostStride; }

// `rows` rows of `width` bytes, `stride` bytes apart.
struct Rows {
  const void* p;
  int64_t rows, stride, width;
  // within the address range that the kernels' and these checks' arithmetic holds
  bool fits() const { return p == nullptr || rows <= 0 || stride <= 0 || (rows <= kMostBytes / stride && lo() <= UINTPTR_MAX - kMostBytes); }
  uintptr_t lo() const { return reinterpret_cast<uintptr_t>(p); }
  uintptr_t hi() const { return lo() + static_cast<uintptr_t>((rows - 1) * stride + width); }
};

// Whether two row buffers share a byte. Rows of one stride may interleave (two column ranges of the
// same rows); buffers of different strides whose ranges meet count as sharing.
bool overlap(const Rows& a, const Rows& b) {
  if (a.p == nullptr || b.p == nullptr || a.rows <= 0 || b.rows <= 0 || a.width <= 0 || b.width <= 0) return false;
  if (a.hi() <= b.lo() || b.hi() <= a.lo()) return false;
  if (a.stride != b.stride) return true;
  const uintptr_t st = static_cast<uintptr_t>(a.stride);
  const uintptr_t d = b.lo() >= a.lo() ? (b.lo() - a.lo()) % st : (st - (a.lo() - b.lo()) % st) % st;
  // row i of b starts d behind some row position of a and ends before the next one
  return !(d >= static_cast<uintptr_t>(a.width) && d + static_cast<uintptr_t>(b.width) <= st);
}
// A buffer of `count` times `bytes` bytes.
Rows flat(const void* p, int64_t count, int64_t bytes) { return Rows{p, count, bytes, bytes}; }
bool all_fit(std::initializer_list<Rows> all) {
  for (const Rows& r : all)
    if (!r.fits()) return false;
  return true;
}
// Whether one of `outs` shares a byte with one of `ins` or with another of `outs`.
bool any_overlap(std::initializer_list<Rows> outs, std::initializer_list<Rows> ins) {
  for (const Rows* o = outs.begin(); o != outs.end(); ++o) {
    for (const Rows& i : ins)
      if (overlap(*o, i)) return true;
    for (const Rows* p = o + 1; p != outs.end(); ++p)
      if (overlap(*o, *p)) return true;
  }
  return false;
}
// The same rows exactly: reading and writing them in place.
bool same(const Rows& a, const Rows& b) { return a.p == b.p && (a.stride == b.stride || a.rows <= 1); }

int check_conv(const seed_conv* c) {
  if (!c) return SEED_ERR_ARG;
  if (c->batch <= 0 || c->channels <= 0 || c->width <= 0) return SEED_ERR_ARG;
  if (!io_ok(c->io_dtype) || (c->silu != 0 && c->silu != 1)) return SEED_ERR_ARG;
  if (c->io_dtype == SEED_F16) return SEED_ERR_UNSUPPORTED;  // fp16 is a factor format only
  if (c->width < 2 || c->width > 4) return SEED_ERR_UNSUPPORTED;
  return SEED_OK;
}

int check_scan(const seed_shape* sh, const seed_prompt* p) {
  if (!sh || !p) return SEED_ERR_ARG;
  if (sh->kind != SEED_GDN && sh->kind != SEED_KDA && sh->kind != SEED_MAMBA2) return SEED_ERR_ARG;
  if (sh->batch <= 0 || sh->heads <= 0 || sh->d_k <= 0 || sh->d_v <= 0) return SEED_ERR_ARG;
  if (!io_ok(sh->io_dtype)) return SEED_ERR_ARG;
  if (p->tokens < 0 || p->key_heads <= 0 || sh->heads % p->key_heads != 0) return SEED_ERR_ARG;
  const int64_t align = 16 / io_bytes(sh->io_dtype);  // elements of a 16-byte access
  const int64_t kw = static_cast<int64_t>(p->key_heads) * sh->d_k, vw = static_cast<int64_t>(sh->heads) * sh->d_v;
  if (!stride_ok(p->q_stride, kw) || !stride_ok(p->k_stride, kw) || !stride_ok(p->v_stride, vw) ||
      !stride_ok(p->o_stride, vw))
    return SEED_ERR_ARG;
  if (p->q_stride % align != 0 || p->k_stride % align != 0 || p->v_stride % align != 0 || p->o_stride % align != 0)
    return SEED_ERR_ARG;
  if (sh->io_dtype == SEED_F16) return SEED_ERR_UNSUPPORTED;
  if ((sh->d_k != 64 && sh->d_k != 128) || (sh->d_v != 64 && sh->d_v != 128)) return SEED_ERR_UNSUPPORTED;
  if (p->tokens > kMostRows) return SEED_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(sh->batch) * sh->heads > kMostRows) return SEED_ERR_UNSUPPORTED;
  return SEED_OK;
}

}  // namespace

extern "C" {

int seed_prefill_conv(const seed_conv* conv, int64_t tokens, const int32_t* offsets, const void* x, int64_t x_stride,
                      const float* weight, const float* bias, const void* window_in, void* window_out, void* y,
                      int64_t y_stride, void* stream) {
  const int c = check_conv(conv);
  if (c != SEED_OK) return c;
  if (tokens < 0 || !offsets || !weight || !window_out || (tokens > 0 && (!x || !y))) return SEED_ERR_ARG;
  if (!stride_ok(x_stride, conv->channels) || !stride_ok(y_stride, conv->channels)) return SEED_ERR_ARG;
  const int64_t e = io_bytes(conv->io_dtype);
  if (!aligned(offsets, 4) || !aligned(weight, 4) || !aligned(bias, 4) || !aligned(x, e) || !aligned(y, e) ||
      !aligned(window_in, e) || !aligned(window_out, e))
    return SEED_ERR_ARG;
  if (tokens > kMostRows) return SEED_ERR_UNSUPPORTED;
  const int64_t ch = conv->channels;
  const int64_t wrow = ch * (conv->width - 1) * e;
  // rows before a tile and the old window are read by other workgroups than those that write
  const Rows rx{x, tokens, x_stride * e, ch * e}, ry{y, tokens, y_stride * e, ch * e};
  const Rows wi{window_in, conv->batch, wrow, wrow}, wo{window_out, conv->batch, wrow, wrow};
  const Rows fw = flat(weight, conv->width, ch * 4), fb = flat(bias, ch, 4);
  const Rows fo = flat(offsets, static_cast<int64_t>(conv->batch) + 1, 4);
  if (!all_fit({rx, ry, wi, wo, fw, fb, fo})) return SEED_ERR_UNSUPPORTED;
  if (any_overlap({ry, wo}, {rx, wi, fw, fb, fo})) return SEED_ERR_ARG;
  seed::ConvArgs a{};
  a.tokens = tokens;
  a.batch = conv->batch;
  a.channels = conv->channels;
  a.silu = conv->silu;
  a.x_stride = x_stride;
  a.y_stride = y_stride;
  a.offsets = offsets;
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.win_in = window_in;
  a.win_out = window_out;
  a.y = y;
  return hip_status(seed::launch_prefill_conv(*conv, a, static_cast<hipStream_t>(stream)));
}

int seed_decode_conv(const seed_conv* conv, const uint8_t* active, const void* x, int64_t x_stride,
                     const float* weight, const float* bias, const void* window_in, void* window_out, void* y,
                     int64_t y_stride, void* stream) {
  const int c = check_conv(conv);
  if (c != SEED_OK) return c;
  if (!x || !weight || !window_in || !window_out || !y) return SEED_ERR_ARG;
  if (!stride_ok(x_stride, conv->channels) || !stride_ok(y_stride, conv->channels)) return SEED_ERR_ARG;
  const int64_t e = io_bytes(conv->io_dtype);
  if (!aligned(weight, 4) || !aligned(bias, 4) || !aligned(x, e) || !aligned(y, e) || !aligned(window_in, e) ||
      !aligned(window_out, e))
    return SEED_ERR_ARG;
  const int64_t ch = conv->channels;
  const int64_t wrow = ch * (conv->width - 1) * e;
  const Rows rx{x, conv->batch, x_stride * e, ch * e}, ry{y, conv->batch, y_stride * e, ch * e};
  const Rows wi{window_in, conv->batch, wrow, wrow}, wo{window_out, conv->batch, wrow, wrow};
  const Rows fw = flat(weight, conv->width, ch * 4), fb = flat(bias, ch, 4), fa = flat(active, conv->batch, 1);
  if (!all_fit({rx, ry, wi, wo, fw, fb, fa})) return SEED_ERR_UNSUPPORTED;
  if (any_overlap({ry, wo}, {fw, fb, fa}) || overlap(wo, rx) || overlap(wi, ry) || (overlap(rx, ry) && !same(rx, ry)) ||
      (overlap(wi, wo) && !same(wi, wo)))
    return SEED_ERR_ARG;
  seed::ConvArgs a{};
  a.batch = conv->batch;
  a.channels = conv->channels;
  a.silu = conv->silu;
  a.x_stride = x_stride;
  a.y_stride = y_stride;
  a.active = active;
  a.x = x;
  a.weight = weight;
  a.bias = bias;
  a.win_in = window_in;
  a.win_out = window_out;
  a.y = y;
  return hip_status(seed::launch_decode_conv(*conv, a, static_cast<hipStream_t>(stream)));
}

size_t seed_prefill_workspace_bytes(const seed_shape* sh, const seed_prompt* prompt) {
  if (check_scan(sh, prompt) != SEED_OK) return 0;
  return seed::prefill_scan_workspace(*sh, *prompt);
}

int seed_prefill_scan(const seed_shape* sh, const seed_prompt* prompt, const void* q, const void* k, const void* v,
                      const float* beta, const float* g, const float* S0, float* S, void* o, void* ws,
                      size_t ws_bytes, void* stream) {
  const int c = check_scan(sh, prompt);
  if (c != SEED_OK) return c;
  const int64_t n = prompt->tokens;
  if (!prompt->offsets || !S || (n > 0 && (!q || !k || !v || !beta || !g || !o))) return SEED_ERR_ARG;
  if (!aligned(prompt->offsets, 4) || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(o, 16) ||
      !aligned(S0, 16) || !aligned(S, 16) || !aligned(beta, 4) || !aligned(g, sh->kind == SEED_KDA ? 16 : 4))
    return SEED_ERR_ARG;
  const int64_t e = io_bytes(sh->io_dtype);
  const int64_t kw = static_cast<int64_t>(prompt->key_heads) * sh->d_k * e, vw = static_cast<int64_t>(sh->heads) * sh->d_v * e;
  const Rows rq{q, n, prompt->q_stride * e, kw}, rk{k, n, prompt->k_stride * e, kw};
  const Rows rv{v, n, prompt->v_stride * e, vw}, ro{o, n, prompt->o_stride * e, vw};
  const int64_t sw = static_cast<int64_t>(sh->d_k) * sh->d_v * 4, units = static_cast<int64_t>(sh->batch) * sh->heads;
  const Rows s0{S0, units, sw, sw}, s1{S, units, sw, sw};
  const Rows fb = flat(beta, n, static_cast<int64_t>(sh->heads) * 4), fo = flat(prompt->offsets, static_cast<int64_t>(sh->batch) + 1, 4);
  const Rows fg = flat(g, n, static_cast<int64_t>(sh->heads) * 4 * (sh->kind == SEED_KDA ? sh->d_k : 1));
  if (!all_fit({rq, rk, rv, ro, s0, s1, fb, fg, fo})) return SEED_ERR_UNSUPPORTED;
  if (any_overlap({ro, s1}, {rq, rk, rv, fb, fg, fo}) || overlap(ro, s0) || (overlap(s0, s1) && !same(s0, s1)))
    return SEED_ERR_ARG;
  const size_t need = seed_prefill_workspace_bytes(sh, prompt);
  if (need > 0) {
    if (!ws || ws_bytes < need) return SEED_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return SEED_ERR_ARG;
    if (any_overlap({flat(ws, static_cast<int64_t>(need), 1)}, {rq, rk, rv, ro, s0, s1, fb, fg, fo})) return SEED_ERR_ARG;
  }
  seed::ScanArgs a{};
  a.tokens = n;
  a.batch = sh->batch;
  a.heads = sh->heads;
  a.key_heads = prompt->key_heads;
  a.q_stride = prompt->q_stride;
  a.k_stride = prompt->k_stride;
  a.v_stride = prompt->v_stride;
  a.o_stride = prompt->o_stride;
  a.offsets = prompt->offsets;
  a.q = q;
  a.k = k;
  a.v = v;
  a.beta = beta;
  a.g = g;
  a.S0 = S0;
  a.S = S;
  a.o = o;
  a.ws = ws;
  return hip_status(seed::launch_prefill_scan(*sh, a, static_cast<hipStream_t>(stream)));
}

int seed_norm_rows(const seed_rows* rows, const void* x, const seed_head_norm* norm, const seed_residual* residual,
                   void* y, void* stream) {
  if (!rows || !norm || !norm->weight) return SEED_ERR_ARG;
  if (rows->rows < 0 || rows->heads <= 0 || rows->dim <= 0 || !io_ok(rows->io_dtype)) return SEED_ERR_ARG;
  if (!(norm->eps >= 0.f) || !(norm->eps < 3.0e38f) || (norm->gate_first != 0 && norm->gate_first != 1)) return SEED_ERR_ARG;
  const void* skip = residual ? residual->skip : nullptr;
  void* total = residual ? residual->total : nullptr;
  const float* scale = residual ? residual->scale : nullptr;
  if (rows->rows > 0 && (!x || !y)) return SEED_ERR_ARG;
  if (rows->rows > 0 && scale && !skip) return SEED_ERR_ARG;
  const int64_t e = io_bytes(rows->io_dtype);
  const int64_t w = static_cast<int64_t>(rows->heads) * rows->dim;
  if (!stride_ok(rows->x_stride, w) || !stride_ok(rows->y_stride, w) || (norm->gate && !stride_ok(rows->gate_stride, w)) ||
      (skip && !stride_ok(rows->skip_stride, w)) || (total && !stride_ok(rows->total_stride, w)))
    return SEED_ERR_ARG;
  if (!aligned(x, e) || !aligned(y, e) || !aligned(norm->gate, e) || !aligned(skip, e) || !aligned(total, e) ||
      !aligned(norm->weight, 4) || !aligned(scale, 4))
    return SEED_ERR_ARG;
  if (rows->io_dtype == SEED_F16) return SEED_ERR_UNSUPPORTED;
  if (rows->rows > kMostRows) return SEED_ERR_UNSUPPORTED;
  const Rows rx{x, rows->rows, rows->x_stride * e, w * e}, ry{y, rows->rows, rows->y_stride * e, w * e};
  const Rows none{};  // the strides of absent buffers are not looked at
  const Rows rg = norm->gate ? Rows{norm->gate, rows->rows, rows->gate_stride * e, w * e} : none;
  const Rows rs = skip ? Rows{skip, rows->rows, rows->skip_stride * e, w * e} : none;
  const Rows rt = total ? Rows{total, rows->rows, rows->total_stride * e, w * e} : none;
  const Rows fw = flat(norm->weight, w, 4), fs = flat(scale, rows->heads, 4);
  if (!all_fit({rx, ry, rg, rs, rt, fw, fs})) return SEED_ERR_UNSUPPORTED;
  for (const Rows& in : {rx, rg, rs})
    for (const Rows& out : {ry, rt})
      if (overlap(in, out) && !same(in, out)) return SEED_ERR_ARG;
  if (any_overlap({ry, rt}, {fw, fs})) return SEED_ERR_ARG;
  if (rows->rows == 0) return SEED_OK;
  seed::NormArgs a{};
  a.rows = rows->rows;
  a.heads = rows->heads;
  a.dim = rows->dim;
  a.x_stride = rows->x_stride;
  a.y_stride = rows->y_stride;
  a.gate_stride = rows->gate_stride;
  a.skip_stride = rows->skip_stride;
  a.total_stride = rows->total_stride;
  a.x = x;
  a.weight = norm->weight;
  a.gate = norm->gate;
  a.skip = skip;
  a.skip_scale = scale;
  a.total = total;
  a.y = y;
  a.eps = norm->eps;
  a.gate_first = norm->gate_first;
  return hip_status(seed::launch_norm_rows(rows->io_dtype, a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
