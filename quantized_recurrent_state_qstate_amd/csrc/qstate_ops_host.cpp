// C-ABI host side of the operators around the decode step: argument checks
// and launches.  Everything that can be refused is refused before a HIP call.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "qstate.h"
#include "qstate_ops.hpp"

namespace {

using qs::op_fail;
using qs::op_ok;

bool aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1u)) == 0u; }

int elem_bytes(int dtype) { return dtype == QS_BF16 ? 2 : 4; }

// Rows of `bytes` bytes at `p`, one every `stride` bytes.
struct Rows {
  const void* p;
  int64_t stride, bytes, rows;
};

// Whether two sets of rows share a byte, as far as strides tell: rows that
// interleave (slices of one wider tensor) do not.
bool overlap(const Rows& x, const Rows& y) {
  if (!x.p || !y.p || x.rows <= 0 || y.rows <= 0 || x.bytes <= 0 || y.bytes <= 0) return false;
  const uintptr_t x0 = (uintptr_t)x.p, y0 = (uintptr_t)y.p;
  const uintptr_t x1 = x0 + (uintptr_t)((x.rows - 1) * x.stride + x.bytes);
  const uintptr_t y1 = y0 + (uintptr_t)((y.rows - 1) * y.stride + y.bytes);
  if (x1 <= y0 || y1 <= x0) return false;
  if (x.stride == y.stride && x.stride > 0) {
    const uintptr_t st = (uintptr_t)x.stride;
    const uintptr_t d = y0 >= x0 ? (y0 - x0) % st : (st - (x0 - y0) % st) % st;   // y's column after x's
    if (d >= (uintptr_t)x.bytes && d + (uintptr_t)y.bytes <= st) return false;
  }
  return true;
}

// A row stride that keeps rows apart and addressable (one row needs none).
bool stride_ok(int64_t stride, int64_t width, int64_t rows) {
  return rows <= 1 ? stride >= 0 : stride >= width && stride <= (int64_t(1) << 62) / rows / 4;
}

qs_status check_conv(const qstate_conv* c, bool step, qs::ConvArgs* a) {
  if (!c) return op_fail(QS_EINVAL, "convolution arguments are NULL");
  if (c->dtype != QS_BF16 && c->dtype != QS_FP32)
    return op_fail(c->dtype == QS_FP16 ? QS_EUNSUPPORTED : QS_EINVAL, "dtype %d (supported: fp32, bf16)", c->dtype);
  if (c->channels < 1 || c->n < 0 || c->slots < 0 || (!step && c->tokens < 0))
    return op_fail(QS_EINVAL, "channels %d, n %d, slots %d, tokens %d", c->channels, c->n, c->slots, c->tokens);
  if (c->width < 2 || c->width > 4) return op_fail(QS_EUNSUPPORTED, "width %d (supported: 2..4)", c->width);
  if (c->silu != 0 && c->silu != 1) return op_fail(QS_EINVAL, "silu %d", c->silu);
  const int64_t rows = step ? c->n : c->tokens, C = c->channels, es = elem_bytes(c->dtype);
  if (c->n == 0 || (!step && rows == 0)) return QS_OK;
  if (!c->x || !c->out || !c->weight) return op_fail(QS_EINVAL, "x, out or weight is NULL");
  if (!aligned(c->x, es) || !aligned(c->out, es) || !aligned(c->weight, 4) || !aligned(c->bias, 4) ||
      !aligned(c->window, es) || !aligned(c->slot, 4) || !aligned(c->offsets, 4))
    return op_fail(QS_EINVAL, "a pointer is not aligned to its elements");
  if (!stride_ok(c->x_stride, C, rows) || !stride_ok(c->out_stride, C, rows))
    return op_fail(QS_EINVAL, "x_stride %lld, out_stride %lld for %lld channels", (long long)c->x_stride,
                   (long long)c->out_stride, (long long)C);
  if (step && !c->window) return op_fail(QS_EINVAL, "window is NULL");
  if (!step && !c->offsets) return op_fail(QS_EINVAL, "offsets is NULL");
  if (c->window && !c->slot && c->n > c->slots)
    return op_fail(QS_EINVAL, "%d sequences without slot numbers, %d windows", c->n, c->slots);
  const Rows x{c->x, c->x_stride * es, C * es, rows}, y{c->out, c->out_stride * es, C * es, rows};
  const int64_t wbytes = (int64_t)(c->width - 1) * C * es;
  const Rows w{c->window, wbytes, wbytes, c->slots};
  if (overlap(x, y) || overlap(x, w) || overlap(y, w)) return op_fail(QS_EINVAL, "x, out and window overlap");
  a->x = c->x;
  a->out = c->out;
  a->weight = c->weight;
  a->bias = c->bias;
  a->window = c->window;
  a->slot = c->slot;
  a->offsets = c->offsets;
  a->x_stride = c->x_stride;
  a->out_stride = c->out_stride;
  a->bf16 = c->dtype == QS_BF16;
  a->T = (int32_t)rows;
  a->C = c->channels;
  a->W = c->width;
  a->n = c->n;
  a->slots = c->slots;
  a->silu = c->silu;
  const int64_t v = 16 / es;
  a->vec = aligned(c->x, 16) && aligned(c->out, 16) && (!c->window || aligned(c->window, 16)) && C % v == 0 &&
           c->x_stride % v == 0 && c->out_stride % v == 0;
  // workgroups of the narrowest variant
  const int64_t tiles = (C + 63) / 64;
  const int64_t blocks = tiles * (step ? rows : rows / 16 + 1 + c->n);
  if (blocks > 0x7FFFFFFF || tiles > qs::max_blocks(256) / 2) return op_fail(QS_EUNSUPPORTED, "%lld rows of %lld channels in one call", (long long)rows, (long long)C);
  return QS_OK;
}

}  // namespace

extern "C" {

qs_status qstate_causal_conv(const qstate_conv* c, void* stream) {
  qs::ConvArgs a{};
  qs_status s = check_conv(c, false, &a);
  if (s != QS_OK) return s;
  if (c->n == 0 || c->tokens == 0) return op_ok();
  hipError_t e = qs::launch_conv(a, reinterpret_cast<hipStream_t>(stream));
  if (e != hipSuccess) return op_fail(QS_EHIP, "convolution launch: %s", hipGetErrorString(e));
  return op_ok();
}

qs_status qstate_causal_conv_step(const qstate_conv* c, void* stream) {
  qs::ConvArgs a{};
  qs_status s = check_conv(c, true, &a);
  if (s != QS_OK) return s;
  if (c->n == 0) return op_ok();
  hipError_t e = qs::launch_conv_step(a, reinterpret_cast<hipStream_t>(stream));
  if (e != hipSuccess) return op_fail(QS_EHIP, "convolution step launch: %s", hipGetErrorString(e));
  return op_ok();
}

qs_status qstate_qk_norm_rotate(const qstate_qk* c, void* stream) {
  if (!c) return op_fail(QS_EINVAL, "arguments are NULL");
  if (c->dtype != QS_BF16 && c->dtype != QS_FP32)
    return op_fail(c->dtype == QS_FP16 ? QS_EUNSUPPORTED : QS_EINVAL, "dtype %d (supported: fp32, bf16)", c->dtype);
  if (c->tokens < 0 || c->q_heads < 0 || c->k_heads < 0 || c->q_heads + (int64_t)c->k_heads < 1)
    return op_fail(QS_EINVAL, "tokens %d, q_heads %d, k_heads %d", c->tokens, c->q_heads, c->k_heads);
  if (c->dim < 1) return op_fail(QS_EINVAL, "dim %d", c->dim);
  if (c->dim % 8 || c->dim > 512) return op_fail(QS_EUNSUPPORTED, "dim %d (supported: multiples of 8 up to 512)", c->dim);
  if (c->rot < 0 || c->rot > c->dim) return op_fail(QS_EINVAL, "rot %d of %d channels", c->rot, c->dim);
  if (c->rot % 16) return op_fail(QS_EUNSUPPORTED, "rot %d (supported: multiples of 16)", c->rot);
  if (c->norm != QS_NORM_NONE && c->norm != QS_NORM_L2 && c->norm != QS_NORM_RMS)
    return op_fail(QS_EINVAL, "norm %d", c->norm);
  if (c->norm != QS_NORM_RMS && (c->q_weight || c->k_weight)) return op_fail(QS_EINVAL, "weights without the RMS norm");
  if (c->interleaved != 0 && c->interleaved != 1) return op_fail(QS_EINVAL, "interleaved %d", c->interleaved);
  if (!std::isfinite(c->eps) || c->eps < 0.0f) return op_fail(QS_EINVAL, "eps %g", c->eps);
  if (!std::isfinite(c->q_scale)) return op_fail(QS_EINVAL, "q_scale %g", c->q_scale);
  if (c->tokens == 0) return op_ok();
  if (c->rot && (!c->position || !c->frequency || !aligned(c->position, 4) || !aligned(c->frequency, 8)))
    return op_fail(QS_EINVAL, "position or frequency NULL or misaligned");
  const int64_t es = elem_bytes(c->dtype), T = c->tokens;
  const void* x[2] = {c->q, c->k};
  void* y[2] = {c->q_out, c->k_out};
  const int64_t xs[2] = {c->q_stride, c->k_stride}, ys[2] = {c->q_out_stride, c->k_out_stride};
  const int32_t heads[2] = {c->q_heads, c->k_heads};
  const float* w[2] = {c->q_weight, c->k_weight};
  Rows in[2], out[2];
  for (int i = 0; i < 2; ++i) {
    const int64_t width = (int64_t)heads[i] * c->dim;
    in[i] = {x[i], xs[i] * es, width * es, heads[i] ? T : 0};
    out[i] = {y[i], ys[i] * es, width * es, heads[i] ? T : 0};
    if (!heads[i]) continue;
    if (!x[i] || !y[i]) return op_fail(QS_EINVAL, "%c or its output is NULL", "qk"[i]);
    if (!stride_ok(xs[i], width, T) || !stride_ok(ys[i], width, T))
      return op_fail(QS_EINVAL, "%c: stride %lld, output stride %lld for rows of %lld", "qk"[i], (long long)xs[i],
                     (long long)ys[i], (long long)width);
    if (!aligned(x[i], 16) || !aligned(y[i], 16) || (T > 1 && (xs[i] * es % 16 || ys[i] * es % 16)))
      return op_fail(QS_EINVAL, "%c: a row is not 16-byte aligned", "qk"[i]);
    if (w[i] && !aligned(w[i], 16)) return op_fail(QS_EINVAL, "%c_weight is not 16-byte aligned", "qk"[i]);
  }
  for (int i = 0; i < 2; ++i)
    for (int j = 0; j < 2; ++j)
      if (overlap(in[i], out[j]) && !(i == j && x[i] == y[i] && xs[i] == ys[i]))
        return op_fail(QS_EINVAL, "%c overlaps the output of %c", "qk"[i], "qk"[j]);
  if (overlap(out[0], out[1])) return op_fail(QS_EINVAL, "the outputs overlap");
  qs::QkArgs a{};
  for (int i = 0; i < 2; ++i) {
    a.x[i] = x[i];
    a.y[i] = y[i];
    a.w[i] = w[i];
    a.xs[i] = xs[i];
    a.ys[i] = ys[i];
    a.heads[i] = heads[i];
  }
  a.position = c->position;
  a.frequency = c->frequency;
  a.bf16 = c->dtype == QS_BF16;
  a.T = c->tokens;
  a.dim = c->dim;
  a.rot = c->rot;
  a.norm = c->norm;
  a.interleaved = c->interleaved;
  a.eps = c->eps;
  a.scale[0] = c->q_scale;
  a.scale[1] = 1.0f;
  hipError_t e = qs::launch_qk(a, reinterpret_cast<hipStream_t>(stream));
  if (e != hipSuccess) return op_fail(QS_EHIP, "norm and rotation launch: %s", hipGetErrorString(e));
  return op_ok();
}

static qs_status check_scan(const qstate_handle* h, const qstate_scan_args* c, qs::ScanArgs* a) {
  if (!h) return op_fail(QS_EINVAL, "handle is NULL");
  if (!c) return op_fail(QS_EINVAL, "scan arguments are NULL");
  const qstate_config& f = *qs::op_view(h).cfg;
  if (c->tokens < 0 || c->n < 0) return op_fail(QS_EINVAL, "tokens %d, n %d", c->tokens, c->n);
  if (c->k_heads < 1 || f.H % c->k_heads)
    return op_fail(QS_EINVAL, "k_heads %d does not divide %d heads", c->k_heads, f.H);
  if ((int64_t)c->n * f.H * f.dv > 0x7FFFFFFF)
    return op_fail(QS_EUNSUPPORTED, "%d sequences of %d heads in one call", c->n, f.H);
  a->T = c->tokens;
  a->n = c->n;
  a->H = f.H;
  a->G = c->k_heads;
  a->dk = f.dk;
  a->dv = f.dv;
  a->bf16 = f.in_dtype == QS_BF16;
  a->delta = f.kind == QS_KIND_DELTA;
  a->key = f.decay_mode == QS_DECAY_KEY;
  a->least = 0;
  a->most = 0x7FFFFFFF;
  return QS_OK;
}

// How a scan's sequences run (a.least > 0: the long ones of them).  The chunked
// kernels take bf16 prompts but the delta rule with a decay for every key channel,
// if the sequences are long enough on the average: of 32 tokens (32 heads of
// 128 x 128: one 8.7 us, 9.9 token by token, sixteen 36, 41, 128 of them 221, 266;
// of 16 tokens 8.6, 6.9, and 23, 26, and 217, 154), by the delta rule of 48 (sixteen
// 60, 72; of 32 tokens one 15, 11, sixteen 47, 51).  Everything else runs token by
// token.
// Additive sequences are cut into segments when the heads alone would leave
// compute units idle; a segment costs a state written, read and written again,
// so it has at least 256 tokens (one decay a head; 16384 tokens of 32 heads of
// 128 x 64: 158 us with segments for 512 workgroups, 163 us for 1024, 200 us
// for 384) or 128 (a decay a channel, whose blocks are slower; 2048 tokens of
// 32 heads of 128 x 128: 107 us for 1024, 140 us with at least 256 tokens) or,
// token by token, 64 (fp32, 2048 tokens of 8 heads of 64 x 64: 45 us, 43 with
// at least 128, 285 uncut), there only if the sequences have two segments on
// the average (16 of 64 tokens: 20 us cut, 13 not) or are the long ones of a batch
// of short ones (scan_split).
struct ScanPlan {
  bool chunked;
  qs::ScanSegs segs;
  uint64_t states, total, uncut;   // workspace bytes
};
// Sequences of more than 2 cut tokens in pieces (delta rule).
static void set_pieces(const qs::ScanArgs& a, int64_t cut, ScanPlan* p) {
  p->segs.cut = (int32_t)cut;
  p->total = (uint64_t)((a.T - 1) / cut + a.n) * (uint64_t)a.H * (uint64_t)(a.dv + a.dk) * (uint64_t)a.dk * 4u;
  p->uncut = (uint64_t)a.n * (uint64_t)a.H * 4u;
}
static bool chunks(const qs::ScanArgs& a) { return a.bf16 && !(a.key && a.delta); }
// The token by token kernel is ahead.
static bool short_on_average(const qs::ScanArgs& a) { return a.T < (int64_t)a.n * (a.delta ? 48 : 32); }
static ScanPlan scan_plan(const qs::ScanArgs& a) {
  ScanPlan p{};
  p.chunked = chunks(a) && (a.least > 0 || !short_on_average(a));
  p.segs.seg = 1 << 30;
  p.segs.count = a.n;
  if (a.delta && !p.chunked) {
    const int64_t rows = (int64_t)a.H * (a.dv + a.dk);   // of one piece's L and M
    // Pieces: with up to 16384 rows at once a token costs little more than with
    // few; of 64 tokens or more (dk 256: 128), and at least four, as they go
    // twice.  fp32, one sequence: 1280 tokens of a head of 64 x 64 39 us, in one
    // piece 196 (pieces of 128: 45); 5120 of 8 heads of 128 x 128 301, 943; 1280
    // of 16 heads of 128 x 128 140, 239.  Every sequence has a place for L and M,
    // so not with many (32768 rows of 256 are 34 MB).
    const int64_t cut = std::max<int64_t>(std::max(64, a.dk / 2), (a.T * rows / 16384 + 15) / 16 * 16);
    if (4 * rows <= 16384 && a.n * rows <= 32768 && a.T > 2 * cut) set_pieces(a, cut, &p);
    return p;
  }
  if (a.delta) {
    p.segs.seg = 64;
    p.segs.count = (a.T + 63) / 64 + a.n;
    p.states = (uint64_t)p.segs.count * (uint64_t)a.H * (uint64_t)qs::kScanPrepBytes;
    // Pieces: as many as have their L and M made by 256 workgroups at once (the
    // first needs no M, the last neither), of 512 tokens or more (4 heads of 256 x
    // 256, 4096 tokens: 173 us, 217 with 1024).  One sequence of 8192 tokens of 128 x
    // 128: 2 heads 112 us, in one piece 560; 8 heads 157, 573; 32 heads 375, 610.  A
    // batch with none that is long pays for launches that do nothing (8 of 1024
    // tokens, 16 heads: 125 us, 117).
    const int64_t wide = (a.dv + 63) / 64, blocks = (int64_t)a.H * (wide + a.dk / 64);   // of one piece's L and M
    const int64_t cut = std::max<int64_t>(512, (a.T / (256 / blocks + 1) + 63) / 64 * 64);
    if (blocks <= 128 && a.n * a.H * wide <= 256 && a.T > 2 * cut) set_pieces(a, cut, &p);
    return p;
  }
  const int columns = p.chunked ? 64 : 32;     // a workgroup's
  const int64_t work = (int64_t)a.T * a.H * ((a.dv + columns - 1) / columns);
  const int64_t least = !p.chunked ? 64 : a.key ? 128 : 256, groups = p.chunked && !a.key ? 512 : 1024;
  const int64_t seg = std::max<int64_t>(least, (work / groups + 63) / 64 * 64);
  if (seg >= a.T || (!p.chunked && a.least == 0 && 2 * seg * a.n > a.T)) return p;
  p.segs.seg = (int32_t)seg;
  p.segs.count = (int32_t)((a.T + seg - 1) / seg + a.n);
  p.states = (uint64_t)p.segs.count * (uint64_t)a.H * (uint64_t)a.dv * (uint64_t)a.dk * 4u;
  p.total = ((uint64_t)p.segs.count * (uint64_t)a.H * (a.key ? (uint64_t)a.dk : 1u) * 4u + 255u) / 256u * 256u;
  p.uncut = (uint64_t)a.n * (uint64_t)a.H * 4u;
  return p;
}

// The average says nothing of a batch's longest sequence, which the host does not
// know: many single tokens with one long prompt would go token by token, uncut.
// So the sequences of this many tokens or more of a batch that is short on the
// average go in launches of their own, as the plan for long ones says, and the
// others token by token (0: no split).  Where there are none, those launches cost
// about 5 ns for each head of a sequence; a token of a chain costs 0.2 us.  The
// split is taken where one chain of all tokens would cost eight times the
// launches.  32 heads of 128 x 64: 255 single tokens with a prompt of 2000 146 us,
// 643 token by token; 256 of 8 tokens 139, 95.
static int scan_split(const qs::ScanArgs& a) {
  if (a.n < 2 || a.T < 1024 || (int64_t)a.n * a.H > (int64_t)a.T * 5) return 0;
  if (chunks(a)) return short_on_average(a) ? 64 : 0;
  if (a.delta) return 0;                       // pieces are of long sequences alone
  qs::ScanArgs some = a;
  some.least = 1;
  const ScanPlan p = scan_plan(some);
  return scan_plan(a).states || !p.states || 2 * p.segs.seg > a.T ? 0 : 2 * p.segs.seg;
}

qs_status qstate_scan_workspace(const qstate_handle* h, const qstate_scan_args* c, uint64_t* bytes) {
  if (!bytes) return op_fail(QS_EINVAL, "bytes is NULL");
  qs::ScanArgs a{};
  qs_status s = check_scan(h, c, &a);
  if (s != QS_OK) return s;
  a.least = scan_split(a);
  const ScanPlan p = scan_plan(a);
  *bytes = p.states + p.total + p.uncut;
  return op_ok();
}

qs_status qstate_scan(qstate_handle* h, const qstate_scan_args* c, void* workspace, uint64_t bytes, void* stream) {
  qs::ScanArgs a{};
  qs_status s = check_scan(h, c, &a);
  if (s != QS_OK) return s;
  if (a.n == 0) return op_ok();
  if (!c->offsets && a.n != 1) return op_fail(QS_EINVAL, "offsets is NULL with %d sequences", a.n);
  if (!c->final || !aligned(c->final, 16) || !aligned(c->initial, 16))
    return op_fail(QS_EINVAL, "final NULL or a state not 16-byte aligned");
  const int64_t es = a.bf16 ? 2 : 4, T = a.T, kw = (int64_t)a.G * a.dk, vw = (int64_t)a.H * a.dv;
  const int64_t dw = a.key ? (int64_t)a.H * a.dk : a.H;
  if (T > 0) {
    if (!c->q || !c->k || !c->v || !c->decay || !c->out) return op_fail(QS_EINVAL, "q, k, v, decay or out is NULL");
    if (!aligned(c->q, es) || !aligned(c->k, es) || !aligned(c->v, es) || !aligned(c->out, es) ||
        !aligned(c->decay, 4) || !aligned(c->beta, 4) || !aligned(c->skip, 4) || !aligned(c->offsets, 4))
      return op_fail(QS_EINVAL, "a pointer is not aligned to its elements");
    if (!stride_ok(c->q_stride, kw, T) || !stride_ok(c->k_stride, kw, T) || !stride_ok(c->v_stride, vw, T) ||
        !stride_ok(c->out_stride, vw, T) || !stride_ok(c->decay_stride, dw, T) ||
        (c->beta && !stride_ok(c->beta_stride, a.H, T)))
      return op_fail(QS_EINVAL, "a stride is smaller than its row");
  }
  const int64_t sb = (int64_t)a.n * a.H * a.dv * a.dk * 4;
  const Rows fin{c->final, sb, sb, 1}, ini{c->initial, sb, sb, 1}, out{c->out, c->out_stride * es, vw * es, T};
  const Rows ins[] = {{c->q, c->q_stride * es, kw * es, T}, {c->k, c->k_stride * es, kw * es, T},
                      {c->v, c->v_stride * es, vw * es, T}, {c->decay, c->decay_stride * 4, dw * 4, T},
                      {c->beta, c->beta_stride * 4, (int64_t)a.H * 4, T}};
  for (const Rows& r : ins)
    if (overlap(r, out) || overlap(r, fin)) return op_fail(QS_EINVAL, "an output overlaps an input");
  if (overlap(out, fin) || overlap(out, ini) || (c->initial != c->final && overlap(ini, fin)))
    return op_fail(QS_EINVAL, "an output overlaps another or the initial state");
  const int split = a.least = scan_split(a);
  ScanPlan p = scan_plan(a);
  if (const uint64_t need = p.states + p.total + p.uncut) {
    if (!workspace || !aligned(workspace, 256) || bytes < need)
      return op_fail(QS_EINVAL, "workspace of %llu bytes, %llu needed, 256-byte aligned", (unsigned long long)bytes,
                     (unsigned long long)need);
    const Rows w{workspace, (int64_t)need, (int64_t)need, 1};
    for (const Rows& r : ins)
      if (overlap(r, w)) return op_fail(QS_EINVAL, "the workspace overlaps an input");
    if (overlap(w, fin) || overlap(w, ini) || overlap(w, out))
      return op_fail(QS_EINVAL, "the workspace overlaps an output or the initial state");
    p.segs.total = (float*)workspace;
    if (p.states) p.segs.states = (float*)((char*)workspace + p.total);
    if (p.uncut) p.segs.uncut = (int32_t*)((char*)workspace + p.total + p.states);
  }
  // workgroups of 256 threads of the launches that have most: a segment's rows
  // (by the delta rule M's too), and the joins
  const int64_t blocks = (int64_t)std::max(p.segs.count, p.segs.cut ? a.n + (a.T - 1) / p.segs.cut : 0) * a.H;
  if (blocks * ((a.dv + 31) / 32 + (p.segs.cut ? a.dk / 32 : 0)) > qs::max_blocks(256) ||
      (int64_t)a.n * (((int64_t)a.H * a.dv * a.dk / 4 + 255) / 256) > qs::max_blocks(256))
    return op_fail(QS_EUNSUPPORTED, "%d tokens of %d sequences in one call", a.T, a.n);
  a.q = c->q;
  a.k = c->k;
  a.v = c->v;
  a.decay = c->decay;
  a.beta = c->beta;
  a.skip = c->skip;
  a.initial = c->initial;
  a.final = c->final;
  a.out = c->out;
  a.offsets = c->offsets;
  a.qs = c->q_stride;
  a.ks = c->k_stride;
  a.vs = c->v_stride;
  a.ds = c->decay_stride;
  a.bs = c->beta_stride;
  a.os = c->out_stride;
  const int64_t v = 16 / es;
  const int64_t far = int64_t(1) << 24;   // the kernels keep offsets within 64 rows in 32 bits
  if (p.chunked && T > 1 && (c->q_stride > far || c->k_stride > far || c->v_stride > far || c->out_stride > far)) {
    if (!split) return op_fail(QS_EUNSUPPORTED, "a stride of more than 2^24 elements");
    a.most = -1;                               // token by token, all of them
  }
  // Value rows of any width leave q and k their wide loads: 3080 tokens of 32 heads
  // of 256 x 35 by the delta rule 481 us, 1026 with none; 3000 of 128 x 63,
  // additive: 79, 152.
  const bool qk = aligned(c->q, 16) && aligned(c->k, 16) && (T <= 1 || (c->q_stride % v == 0 && c->k_stride % v == 0));
  const bool vo = aligned(c->v, 16) && aligned(c->out, 16) && a.dv % v == 0 &&
                  (T <= 1 || (c->v_stride % v == 0 && c->out_stride % v == 0));
  a.vec = !qk ? 0 : vo ? 2 : 1;
  if ((s = qs::op_check_device(h)) != QS_OK) return s;
  const hipStream_t on = reinterpret_cast<hipStream_t>(stream);
  hipError_t e = hipSuccess;
  if (split) {                                 // the short ones, in one piece each
    qs::ScanArgs b = a;
    b.least = 0;
    b.most = a.most < 0 ? 0x7FFFFFFF : split - 1;
    qs::ScanSegs whole{};
    whole.seg = 1 << 30;
    whole.count = a.n;
    e = qs::launch_scan(b, whole, on);
  }
  if (e == hipSuccess && a.most >= 0)
    e = (!p.chunked ? qs::launch_scan : a.delta ? qs::launch_scan_delta : a.key ? qs::launch_scan_key
                                                                              : qs::launch_scan_chunk)(a, p.segs, on);
  if (e != hipSuccess) return op_fail(QS_EHIP, "scan launch: %s", hipGetErrorString(e));
  return op_ok();
}

// The buffers of a slot: the state's own (bytes per slot from the plan) and
// the caller's, cut into pieces.
static qs_status slot_buffers(const qstate_handle* h, const qstate_tensors* pool, const qstate_tensors* source,
                              const qstate_slot_buffer* extra, int32_t n_extra, qs::SlotArgs* a) {
  const qs::HandleView v = qs::op_view(h);
  const qstate_sizes& z = *v.sizes;
  const uint64_t B = (uint64_t)v.cfg->B;
  const uint64_t size[6] = {z.codes, z.scales, z.hp, z.lrb_W, z.lrb_U, z.lrb_n};
  const void* src[6] = {source->codes, source->scales, source->hp, source->lrb_W, source->lrb_U, source->lrb_n};
  void* dst[6] = {pool->codes, pool->scales, pool->hp, pool->lrb_W, pool->lrb_U, pool->lrb_n};
  if (n_extra < 0 || n_extra > qs::kMaxSlotBuffers - 6)
    return op_fail(QS_EINVAL, "n_extra %d (at most %d)", n_extra, qs::kMaxSlotBuffers - 6);
  if (n_extra && !extra) return op_fail(QS_EINVAL, "extra is NULL");
  uint64_t pieces = 0;
  auto add = [&](const void* s, void* d, uint64_t bytes) {
    qs::SlotBuffer& b = a->buf[a->nbuf++];
    b.src = (const uint8_t*)s;
    b.dst = (uint8_t*)d;
    b.bytes = bytes;
    b.first = (uint32_t)pieces;
    const uint64_t all = bytes | (uint64_t)(uintptr_t)s | (uint64_t)(uintptr_t)d;
    b.unit = all % 16 == 0 ? 16 : all % 4 == 0 ? 4 : all % 2 == 0 ? 2 : 1;
    pieces += (bytes + qs::kSlotPiece - 1) / qs::kSlotPiece;
  };
  for (int i = 0; i < 6; ++i)
    if (size[i]) add(src[i], dst[i], size[i] / B);
  for (int i = 0; i < n_extra; ++i) {
    if (!extra[i].bytes) continue;
    if (!extra[i].src || !extra[i].dst) return op_fail(QS_EINVAL, "extra[%d] is NULL", i);
    if (extra[i].bytes > (1ull << 40)) return op_fail(QS_EUNSUPPORTED, "extra[%d]: %llu bytes a slot", i,
                                                      (unsigned long long)extra[i].bytes);
    add(extra[i].src, extra[i].dst, extra[i].bytes);
  }
  if (pieces > (uint64_t)qs::max_blocks(256)) return op_fail(QS_EUNSUPPORTED, "a slot of %llu pieces", (unsigned long long)pieces);
  a->pieces = (uint32_t)pieces;
  return QS_OK;
}

qs_status qstate_copy_slots(qstate_handle* h, const qstate_tensors* pool, const qstate_tensors* source,
                            int32_t src_slots, int32_t n, const int32_t* src_slot, const int32_t* dst_slot,
                            const qstate_slot_buffer* extra, int32_t n_extra, void* stream) {
  if (!h) return op_fail(QS_EINVAL, "handle is NULL");
  qs_status s = qs::op_check_tensors(h, pool);
  if (s == QS_OK) s = qs::op_check_tensors(h, source);
  if (s != QS_OK) return s;
  if (n < 0 || src_slots < 0) return op_fail(QS_EINVAL, "n %d, src_slots %d", n, src_slots);
  qs::SlotArgs a{};
  if ((s = slot_buffers(h, pool, source, extra, n_extra, &a)) != QS_OK) return s;
  if (n == 0 || a.pieces == 0) return op_ok();
  if (!src_slot || !dst_slot || !aligned(src_slot, 4) || !aligned(dst_slot, 4))
    return op_fail(QS_EINVAL, "src_slot or dst_slot NULL or misaligned");
  // The buffers of two pools are the same ones or apart: a copy between
  // overlapping ranges at different bases would read what it writes.
  const int64_t B = qs::op_view(h).cfg->B;
  for (int i = 0; i < a.nbuf; ++i) {
    const qs::SlotBuffer& b = a.buf[i];
    const Rows x{b.src, (int64_t)b.bytes, (int64_t)b.bytes, src_slots}, y{b.dst, (int64_t)b.bytes, (int64_t)b.bytes, B};
    if (b.src != b.dst && overlap(x, y)) return op_fail(QS_EINVAL, "source and pool overlap without being the same");
    if ((b.src == b.dst) != (a.buf[0].src == a.buf[0].dst))
      return op_fail(QS_EINVAL, "some of the source's buffers are the pool's and some are not");
  }
  if (a.buf[0].src == a.buf[0].dst && src_slots > B)
    return op_fail(QS_EINVAL, "%d slots of a source that is the pool, which has %d", src_slots, (int)B);
  if ((uint64_t)n * a.pieces > 0x7FFFFFFFull) return op_fail(QS_EUNSUPPORTED, "%d copies in one call", n);
  if ((s = qs::op_check_device(h)) != QS_OK) return s;
  a.src_slots = src_slots;
  a.dst_slots = (int32_t)B;
  a.n = n;
  a.src_slot = src_slot;
  a.dst_slot = dst_slot;
  hipError_t e = qs::launch_copy_slots(a, reinterpret_cast<hipStream_t>(stream));
  if (e != hipSuccess) return op_fail(QS_EHIP, "slot copy launch: %s", hipGetErrorString(e));
  return op_ok();
}

qs_status qstate_compact_slots(qstate_handle* h, const qstate_tensors* pool, const uint8_t* live, int32_t* where,
                               const qstate_slot_buffer* extra, int32_t n_extra, void* stream) {
  if (!h) return op_fail(QS_EINVAL, "handle is NULL");
  qs_status s = qs::op_check_tensors(h, pool);
  if (s != QS_OK) return s;
  qs::SlotArgs a{};
  if ((s = slot_buffers(h, pool, pool, extra, n_extra, &a)) != QS_OK) return s;
  const int32_t B = qs::op_view(h).cfg->B;
  if (B == 0) return op_ok();
  if (B > qs::kMaxCompactSlots) return op_fail(QS_EUNSUPPORTED, "%d slots (at most %d)", B, qs::kMaxCompactSlots);
  if (!live || !where || !aligned(where, 4)) return op_fail(QS_EINVAL, "live or where NULL or misaligned");
  for (int i = 0; i < a.nbuf; ++i)
    if (a.buf[i].src != a.buf[i].dst) return op_fail(QS_EINVAL, "extra buffers of a compaction have src = dst");
  if ((uint64_t)(B / 2) * a.pieces > 0x7FFFFFFFull) return op_fail(QS_EUNSUPPORTED, "%d slots of %u pieces", B, a.pieces);
  if ((s = qs::op_check_device(h)) != QS_OK) return s;
  a.dst_slots = B;
  a.live = live;
  a.where = where;
  hipError_t e = qs::launch_compact_slots(a, reinterpret_cast<hipStream_t>(stream));
  if (e != hipSuccess) return op_fail(QS_EHIP, "compaction launch: %s", hipGetErrorString(e));
  return op_ok();
}

}  // extern "C"
