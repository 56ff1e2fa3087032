// C ABI of the attention layers and of drafted tokens: rotary positions, the paged cache, attention over
// it and the verification of drafts. As in api.cpp, every entry point validates on the host before
// anything is enqueued, never synchronises and allocates nothing.
#include <hip/hip_runtime.h>
#include <math.h>

#include "../../include/seed.h"
#include "attend.hpp"
#include "extents.hpp"

namespace {

using namespace seed;

constexpr int64_t kMostBlocks = most_blocks(256);
constexpr int64_t kMostTokenStride = int64_t{1} << 24;   // 16 positions' bytes are 32-bit offsets
constexpr int32_t kMostShare = 1 << 14;                  // a row's token is found in fp32
constexpr int64_t kMostPositions = int64_t{1} << 30;     // positions and their tiles' ends are int32

int check_rotary(const seed_rotary* r, int32_t dim) {
  if (r->dim < 2 || r->dim % 2 != 0 || r->dim > dim || (r->interleaved != 0 && r->interleaved != 1)) return SEED_ERR_ARG;
  if (!isfinite(r->amplitude) || !r->turns || !aligned(r->turns, 8)) return SEED_ERR_ARG;
  return SEED_OK;
}
Rows turns_of(const seed_rotary* r) { return r ? flat(r->turns, r->dim / 2, 8) : Rows{}; }

int check_cache(const seed_cache* c) {
  if (!c) return SEED_ERR_ARG;
  if (c->batch <= 0 || c->key_heads <= 0 || c->dim <= 0 || c->page <= 0 || c->width <= 0 || c->pages <= 0) return SEED_ERR_ARG;
  if (!io_ok(c->io_dtype) || !c->k || !c->v || !c->table) return SEED_ERR_ARG;
  if (c->io_dtype == SEED_F16) return SEED_ERR_UNSUPPORTED;  // fp16 is a factor format only
  if (c->dim != 64 && c->dim != 128 && c->dim != 256) return SEED_ERR_UNSUPPORTED;
  if (c->page < 16 || c->page > (1 << 20) || (c->page & (c->page - 1)) != 0) return SEED_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(c->page) * c->width > kMostPositions) return SEED_ERR_UNSUPPORTED;
  const int64_t align = 16 / io_bytes(c->io_dtype);
  for (const int64_t st : {c->page_stride, c->token_stride, c->head_stride})
    if (st <= 0 || st > kMostStride || st % align != 0) return SEED_ERR_ARG;
  // the spans below stay inside 64 bits
  if (c->key_heads > kMostBytes / 4 / c->head_stride || c->page > kMostBytes / 4 / c->token_stride) return SEED_ERR_UNSUPPORTED;
  if (c->token_stride > kMostTokenStride) return SEED_ERR_UNSUPPORTED;
  // [page][key_heads][dim] or [key_heads][page][dim], nothing overlapping; the stride of a single head or page is not looked at
  const int64_t d = c->dim, heads = c->key_heads, page = c->page;
  const bool by_token = (heads == 1 || c->head_stride >= d) && c->token_stride >= (heads - 1) * c->head_stride + d &&
                        (c->pages == 1 || c->page_stride >= (page - 1) * c->token_stride + (heads - 1) * c->head_stride + d);
  const bool by_head = c->token_stride >= d && (heads == 1 || c->head_stride >= (page - 1) * c->token_stride + d) &&
                       (c->pages == 1 || c->page_stride >= (heads - 1) * c->head_stride + (page - 1) * c->token_stride + d);
  if (!by_token && !by_head) return SEED_ERR_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->table, 4)) return SEED_ERR_ARG;
  return SEED_OK;
}

// The bytes from a pool's first value to behind its last one, and its pages as rows.
int64_t page_bytes(const seed_cache* c) {
  return ((c->page - 1) * c->token_stride + (c->key_heads - 1) * c->head_stride + c->dim) * io_bytes(c->io_dtype);
}
Rows pool(const seed_cache* c, const void* p) {
  return Rows{p, c->pages, c->page_stride * io_bytes(c->io_dtype), page_bytes(c)};
}
bool pool_fits(const seed_cache* c) { return page_bytes(c) <= kMostBytes && pool(c, c->k).fits() && pool(c, c->v).fits(); }
// Whether a buffer meets a pool: its pages' gaps count as the pool's.
bool meets(const Rows& r, const seed_cache* c, const void* p) {
  if (r.p == nullptr || r.rows <= 0 || r.width <= 0) return false;
  const Rows q = pool(c, p);
  return !(r.hi() <= q.lo() || q.hi() <= r.lo());
}
// A pool's pages, the tokens (or heads) of a page, and the heads (tokens) of those: `count` blocks of `width` bytes,
// `stride` bytes apart, which is at least the width where there is a second one.
struct Level {
  int64_t stride, count, width;
};
// Whether one of k's blocks and one of v's share a byte, v's first lying d bytes behind k's first. Blocks n of v and m of
// k are d + (n - m) stride apart: only the two distances next to 0 are below a width.
bool blocks_meet(const Level* level, int levels, int64_t d) {
  const Level& l = *level;
  if (l.count == 1) return d > -l.width && d < l.width && (levels == 1 || blocks_meet(level + 1, levels - 1, d));
  int64_t steps = d / l.stride, rest = d % l.stride;
  if (rest < 0) {
    rest += l.stride;
    --steps;
  }
  auto meet = [&](int64_t n, int64_t way) {
    return n > -l.count && n < l.count && way > -l.width && way < l.width && (levels == 1 || blocks_meet(level + 1, levels - 1, way));
  };
  return meet(steps, rest) || meet(steps + 1, rest - l.stride);
}
// Whether k and v share a byte. Of one set of strides, they may lie side by side: by pages, tokens or heads, whether or not
// one stride is a multiple of another.
bool pools_meet(const seed_cache* c) {
  const Rows a = pool(c, c->k), b = pool(c, c->v);
  if (a.hi() <= b.lo() || b.hi() <= a.lo()) return false;
  const int64_t e = io_bytes(c->io_dtype), d = static_cast<int64_t>(b.lo() - a.lo());
  const int64_t head = c->dim * e, heads = c->key_heads, page = c->page, hs = c->head_stride * e, ts = c->token_stride * e;
  const Level pages{c->page_stride * e, c->pages, page_bytes(c)};
  if (ts >= (heads - 1) * hs + head) {  // by token
    const Level levels[3] = {pages, {ts, page, (heads - 1) * hs + head}, {hs, heads, head}};
    return blocks_meet(levels, 3, d);
  }
  const Level levels[3] = {pages, {hs, heads, (page - 1) * ts + head}, {ts, page, head}};
  return blocks_meet(levels, 3, d);
}

int check_tokens(const seed_cache* c, const seed_tokens* t, bool queries) {
  if (!t || t->tokens < 0 || !t->lengths) return SEED_ERR_ARG;
  if (!t->offsets && t->tokens != c->batch) return SEED_ERR_ARG;
  if (queries && (t->heads <= 0 || t->heads % c->key_heads != 0)) return SEED_ERR_ARG;
  if (!aligned(t->offsets, 4) || !aligned(t->lengths, 4)) return SEED_ERR_ARG;
  if (t->tokens > kMostRows) return SEED_ERR_UNSUPPORTED;
  return SEED_OK;
}

CacheArgs cache_args(const seed_cache* c, const seed_tokens* t) {
  CacheArgs a{};
  a.batch = c->batch;
  a.heads = t->heads;
  a.key_heads = c->key_heads;
  a.dim = c->dim;
  for (a.page_shift = 0; (1 << a.page_shift) < c->page;) ++a.page_shift;
  a.width = c->width;
  a.pages = c->pages;
  a.page_stride = c->page_stride;
  a.token_stride = c->token_stride;
  a.head_stride = c->head_stride;
  a.k = c->k;
  a.v = c->v;
  a.table = c->table;
  a.tokens = t->tokens;
  a.offsets = t->offsets;
  a.lengths = t->lengths;
  return a;
}
Rows table_of(const seed_cache* c) { return flat(c->table, c->batch, static_cast<int64_t>(c->width) * 4); }
Rows offsets_of(const seed_cache* c, const seed_tokens* t) { return flat(t->offsets, static_cast<int64_t>(c->batch) + 1, 4); }
Rows lengths_of(const seed_cache* c, const seed_tokens* t) { return flat(t->lengths, c->batch, 4); }

// The arguments without pointers, for the workspace's size too.
int check_attend(const seed_cache* c, const seed_tokens* t, const seed_attend* w, AttendArgs& a) {
  int s = check_cache(c);
  if (s != SEED_OK) return s;
  s = check_tokens(c, t, true);
  if (s != SEED_OK) return s;
  if (!w || w->max_tokens < 1 || w->max_length < 1 || w->window < 0 || !isfinite(w->scale)) return SEED_ERR_ARG;
  if (static_cast<int64_t>(w->max_length) > static_cast<int64_t>(c->page) * c->width) return SEED_ERR_ARG;
  if (w->max_tokens > 32) return SEED_ERR_UNSUPPORTED;
  const double scale2 = fabs(static_cast<double>(w->scale)) * 1.4426950408889634;
  if (!isfinite(static_cast<float>(scale2)) || static_cast<float>(scale2) == 0.f) return SEED_ERR_ARG;
  a.c = cache_args(c, t);
  a.share = t->heads / c->key_heads;
  a.per_share = 1.f / static_cast<float>(a.share);
  a.max_tokens = w->max_tokens;
  a.capacity = w->max_length;
  a.pages = static_cast<uint32_t>(c->pages < (int64_t{1} << 31) ? c->pages : int64_t{1} << 31);
  a.window = w->window >= w->max_length ? 0 : w->window;  // a window that holds every position
  a.scale2 = static_cast<float>(scale2);
  a.negate = w->scale < 0.f ? (c->io_dtype == SEED_F32 ? 0x80000000u : 0x80008000u) : 0u;
  // the launch has to hold a workgroup for every 16 rows, and one per row to join them
  const int64_t rows = static_cast<int64_t>(w->max_tokens) * t->heads;
  if (a.share > kMostShare || rows > kMostBlocks / c->batch) return SEED_ERR_UNSUPPORTED;
  return plan_attend(c->io_dtype, a) ? SEED_OK : SEED_ERR_UNSUPPORTED;
}
int check_drafts(const seed_drafts* d) {
  if (!d || d->batch <= 0 || d->vocab <= 0 || d->rows < 0 || !io_ok(d->io_dtype)) return SEED_ERR_ARG;
  if (d->io_dtype == SEED_F16) return SEED_ERR_UNSUPPORTED;
  if (d->rows > kMostRows || d->vocab > (1 << 30)) return SEED_ERR_UNSUPPORTED;
  const int32_t segments = verify_segments(d->vocab);
  if (segments > kMostBlocks / d->batch) return SEED_ERR_UNSUPPORTED;
  if (segments <= verify_alone() && d->batch > most_blocks(kAloneThreads)) return SEED_ERR_UNSUPPORTED;
  return SEED_OK;
}
int64_t verify_workspace(const seed_drafts* d) {
  if (verify_segments(d->vocab) <= verify_alone()) return 0;
  return static_cast<int64_t>(d->batch) * verify_segments(d->vocab) * 8 + static_cast<int64_t>(d->batch) * 4;
}

}  // namespace

extern "C" {

int seed_rotary_turns(const seed_rotary_scaling* s, int32_t dim, double* turns) {
  if (!s || !turns || dim < 2 || dim % 2 != 0) return SEED_ERR_ARG;
  if (s->kind < SEED_ROTARY_PLAIN || s->kind > SEED_ROTARY_INDEX) return SEED_ERR_ARG;
  if (!(s->base > 0.0) || !isfinite(s->base) || (s->kind == SEED_ROTARY_INDEX && !(s->base > 1.0))) return SEED_ERR_ARG;
  if (s->kind != SEED_ROTARY_PLAIN && (!(s->factor > 0.0) || !isfinite(s->factor))) return SEED_ERR_ARG;
  const bool ramp = s->kind == SEED_ROTARY_PARTS || s->kind == SEED_ROTARY_INDEX;
  if (ramp && (!(s->length > 0.0) || !isfinite(s->length) || !(s->low > 0.0) || !(s->high > s->low) || !isfinite(s->high)))
    return SEED_ERR_ARG;
  const double tau = 6.283185307179586476925;
  double base = s->base;
  if (s->kind == SEED_ROTARY_BASE && dim > 2) base *= pow(s->factor, static_cast<double>(dim) / (dim - 2));
  double first = 0.0, last = 0.0;  // SEED_ROTARY_INDEX: the ramp's ends
  if (s->kind == SEED_ROTARY_INDEX) {
    // n(i) = length base^(-2 i / dim) / tau, solved for i
    first = fmax(floor(dim * log(s->length / (s->high * tau)) / (2.0 * log(s->base))), 0.0);
    last = fmin(ceil(dim * log(s->length / (s->low * tau)) / (2.0 * log(s->base))), dim - 1.0);
  }
  for (int32_t i = 0; i < dim / 2; ++i) {
    double t = pow(base, -2.0 * i / dim) / tau;
    if (s->kind == SEED_ROTARY_LINEAR) t /= s->factor;
    if (ramp) {
      double keep = s->kind == SEED_ROTARY_PARTS ? (s->length * t - s->low) / (s->high - s->low)
                    : last > first               ? 1.0 - (i - first) / (last - first)
                                                 : (i <= first ? 1.0 : 0.0);  // no room for a ramp: a step
      keep = fmin(fmax(keep, 0.0), 1.0);
      t *= keep + (1.0 - keep) / s->factor;
    }
    if (!isfinite(t)) return SEED_ERR_ARG;  // a base or factor next to 0
    turns[i] = t;
  }
  return SEED_OK;
}

int seed_rotate_rows(const seed_rows* rows, const seed_rotary* rotary, const void* x, const int32_t* positions, void* y,
                     void* stream) {
  if (!rows || !rotary) return SEED_ERR_ARG;
  if (rows->rows < 0 || rows->heads <= 0 || rows->dim <= 0 || !io_ok(rows->io_dtype)) return SEED_ERR_ARG;
  const int c = check_rotary(rotary, rows->dim);
  if (c != SEED_OK) return c;
  if (rows->rows > 0 && (!x || !y || !positions)) return SEED_ERR_ARG;
  const int64_t e = io_bytes(rows->io_dtype), w = static_cast<int64_t>(rows->heads) * rows->dim;
  if (!stride_ok(rows->x_stride, w) || !stride_ok(rows->y_stride, w)) return SEED_ERR_ARG;
  if (!aligned(x, e) || !aligned(y, e) || !aligned(positions, 4)) return SEED_ERR_ARG;
  if (rows->io_dtype == SEED_F16 || rows->rows > kMostRows) return SEED_ERR_UNSUPPORTED;
  const Rows rx{x, rows->rows, rows->x_stride * e, w * e}, ry{y, rows->rows, rows->y_stride * e, w * e};
  const Rows fp = flat(positions, rows->rows, 4), ft = turns_of(rotary);
  if (!all_fit({rx, ry, fp, ft})) return SEED_ERR_UNSUPPORTED;
  if ((overlap(rx, ry) && !same(rx, ry)) || any_overlap({ry}, {fp, ft})) return SEED_ERR_ARG;
  if (rows->rows == 0) return SEED_OK;
  RotateArgs a{};
  a.rows = rows->rows;
  a.heads = rows->heads;
  a.dim = rows->dim;
  a.rot = rotary->dim;
  a.interleaved = rotary->interleaved;
  a.amplitude = rotary->amplitude;
  a.x_stride = rows->x_stride;
  a.y_stride = rows->y_stride;
  a.turns = rotary->turns;
  a.positions = positions;
  a.x = x;
  a.y = y;
  return hip_status(launch_rotate_rows(rows->io_dtype, a, static_cast<hipStream_t>(stream)));
}

int seed_cache_append(const seed_cache* cache, const seed_tokens* tokens, const seed_rotary* rotary, const void* q,
                      const void* k, const void* v, void* q_out, void* stream) {
  int c = check_cache(cache);
  if (c != SEED_OK) return c;
  c = check_tokens(cache, tokens, q != nullptr);
  if (c != SEED_OK) return c;
  if (rotary) {
    c = check_rotary(rotary, cache->dim);
    if (c != SEED_OK) return c;
  }
  const int64_t n = tokens->tokens;
  if (n > 0 && (!k || !v || !q != !q_out)) return SEED_ERR_ARG;
  const int64_t e = io_bytes(cache->io_dtype);
  const int64_t kw = static_cast<int64_t>(cache->key_heads) * cache->dim, qw = q ? static_cast<int64_t>(tokens->heads) * cache->dim : 0;
  if (!stride_ok(tokens->k_stride, kw) || !stride_ok(tokens->v_stride, kw)) return SEED_ERR_ARG;
  if (q && (!stride_ok(tokens->q_stride, qw) || !stride_ok(tokens->o_stride, qw))) return SEED_ERR_ARG;
  if (!aligned(q, e) || !aligned(k, e) || !aligned(v, e) || !aligned(q_out, e)) return SEED_ERR_ARG;
  const Rows none{};
  const Rows rq = q ? Rows{q, n, tokens->q_stride * e, qw * e} : none, ro = q ? Rows{q_out, n, tokens->o_stride * e, qw * e} : none;
  const Rows rk{k, n, tokens->k_stride * e, kw * e}, rv{v, n, tokens->v_stride * e, kw * e};
  const Rows ft = turns_of(rotary), fb = table_of(cache), fo = offsets_of(cache, tokens), fl = lengths_of(cache, tokens);
  if (!pool_fits(cache) || !all_fit({rq, ro, rk, rv, ft, fb, fo, fl})) return SEED_ERR_UNSUPPORTED;
  if (pools_meet(cache) || any_overlap({ro}, {rk, rv, ft, fb, fo, fl}) || (overlap(rq, ro) && !same(rq, ro))) return SEED_ERR_ARG;
  for (const Rows& r : {rq, ro, rk, rv, ft, fb, fo, fl})
    if (meets(r, cache, cache->k) || meets(r, cache, cache->v)) return SEED_ERR_ARG;
  if (n == 0) return SEED_OK;
  AppendArgs a{};
  a.c = cache_args(cache, tokens);
  if (rotary) {
    a.rot = rotary->dim;
    a.interleaved = rotary->interleaved;
    a.amplitude = rotary->amplitude;
    a.turns = rotary->turns;
  }
  a.q_stride = tokens->q_stride;
  a.k_stride = tokens->k_stride;
  a.v_stride = tokens->v_stride;
  a.o_stride = tokens->o_stride;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_out = q_out;
  return hip_status(launch_cache_append(cache->io_dtype, a, static_cast<hipStream_t>(stream)));
}

size_t seed_attend_workspace_bytes(const seed_cache* cache, const seed_tokens* tokens, const seed_attend* attend) {
  AttendArgs a{};
  if (check_attend(cache, tokens, attend, a) != SEED_OK) return 0;
  return static_cast<size_t>(attend_workspace(a));
}

int seed_decode_attend(const seed_cache* cache, const seed_tokens* tokens, const seed_attend* attend, const void* q,
                       void* o, float* lse, void* ws, size_t ws_bytes, void* stream) {
  AttendArgs a{};
  const int c = check_attend(cache, tokens, attend, a);
  if (c != SEED_OK) return c;
  const int64_t n = tokens->tokens;
  if (n > 0 && (!q || !o)) return SEED_ERR_ARG;
  const int64_t e = io_bytes(cache->io_dtype), align = 16 / e, w = static_cast<int64_t>(tokens->heads) * cache->dim;
  if (!stride_ok(tokens->q_stride, w) || !stride_ok(tokens->o_stride, w) || tokens->q_stride % align != 0 || tokens->o_stride % align != 0)
    return SEED_ERR_ARG;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(lse, 4)) return SEED_ERR_ARG;
  const Rows rq{q, n, tokens->q_stride * e, w * e}, ro{o, n, tokens->o_stride * e, w * e};
  const Rows rl = flat(lse, n, static_cast<int64_t>(tokens->heads) * 4);
  const Rows fb = table_of(cache), fo = offsets_of(cache, tokens), fl = lengths_of(cache, tokens);
  const int64_t need = attend_workspace(a);
  if (!pool_fits(cache) || !all_fit({rq, ro, rl, fb, fo, fl})) return SEED_ERR_UNSUPPORTED;
  if (pools_meet(cache) || any_overlap({ro, rl}, {rq, fb, fo, fl})) return SEED_ERR_ARG;
  for (const Rows& r : {ro, rl})
    if (meets(r, cache, cache->k) || meets(r, cache, cache->v)) return SEED_ERR_ARG;
  if (n == 0) return SEED_OK;
  if (need > 0) {
    if (!ws || ws_bytes < static_cast<size_t>(need)) return SEED_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return SEED_ERR_ARG;
    const Rows fw = flat(ws, need, 1);
    if (!fw.fits()) return SEED_ERR_UNSUPPORTED;
    if (any_overlap({fw}, {rq, ro, rl, fb, fo, fl}) || meets(fw, cache, cache->k) || meets(fw, cache, cache->v)) return SEED_ERR_ARG;
  }
  a.q_stride = tokens->q_stride;
  a.o_stride = tokens->o_stride;
  a.q = q;
  a.o = o;
  a.lse = lse;
  return hip_status(launch_attend(cache->io_dtype, a, ws, static_cast<hipStream_t>(stream)));
}

size_t seed_verify_workspace_bytes(const seed_drafts* drafts) {
  return check_drafts(drafts) == SEED_OK ? static_cast<size_t>(verify_workspace(drafts)) : 0;
}

int seed_verify_drafts(const seed_drafts* d, const void* target, const void* draft, const int32_t* drafts,
                       const float* uniforms, const float* draws, int32_t* out, int32_t* counts, void* ws,
                       size_t ws_bytes, void* stream) {
  const int c = check_drafts(d);
  if (c != SEED_OK) return c;
  const int64_t n = d->rows, e = io_bytes(d->io_dtype), w = d->vocab;
  if (!d->offsets || !draws || !counts || (n > 0 && (!target || !drafts || !uniforms || !out))) return SEED_ERR_ARG;
  if (!stride_ok(d->target_stride, w) || (draft && !stride_ok(d->draft_stride, w))) return SEED_ERR_ARG;
  if (!aligned(target, e) || !aligned(draft, e) || !aligned(d->offsets, 4) || !aligned(drafts, 4) || !aligned(uniforms, 4) ||
      !aligned(draws, 4) || !aligned(out, 4) || !aligned(counts, 4))
    return SEED_ERR_ARG;
  const Rows none{};
  const Rows rt{target, n, d->target_stride * e, w * e}, rd = draft ? Rows{draft, n, d->draft_stride * e, w * e} : none;
  const Rows fo = flat(d->offsets, static_cast<int64_t>(d->batch) + 1, 4), fx = flat(drafts, n, 4), fu = flat(uniforms, n, 4);
  const Rows fr = flat(draws, d->batch, 4), out_rows = flat(out, n, 4), fc = flat(counts, d->batch, 4);
  if (!all_fit({rt, rd, fo, fx, fu, fr, out_rows, fc})) return SEED_ERR_UNSUPPORTED;
  if (any_overlap({out_rows, fc}, {rt, rd, fo, fu, fr}) || overlap(fc, fx) || (overlap(out_rows, fx) && out != drafts)) return SEED_ERR_ARG;
  const int64_t need = verify_workspace(d);
  if (need > 0) {
    if (!ws || ws_bytes < static_cast<size_t>(need)) return SEED_ERR_WORKSPACE;
    if (!aligned(ws, 16)) return SEED_ERR_ARG;
    const Rows fw = flat(ws, need, 1);
    if (!fw.fits()) return SEED_ERR_UNSUPPORTED;
    if (any_overlap({fw}, {rt, rd, fo, fx, fu, fr, out_rows, fc})) return SEED_ERR_ARG;
  }
  VerifyArgs a{};
  a.batch = d->batch;
  a.vocab = d->vocab;
  a.segments = verify_segments(d->vocab);
  a.rows = n;
  a.target_stride = d->target_stride;
  a.draft_stride = d->draft_stride;
  a.offsets = d->offsets;
  a.target = target;
  a.draft = draft;
  a.drafts = drafts;
  a.uniforms = uniforms;
  a.draws = draws;
  a.out = out;
  a.counts = counts;
  if (need > 0) {
    a.sums = static_cast<double*>(ws);
    a.kept = reinterpret_cast<int32_t*>(a.sums + static_cast<int64_t>(d->batch) * a.segments);
  }
  return hip_status(launch_verify(d->io_dtype, a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
