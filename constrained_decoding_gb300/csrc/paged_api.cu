// extern "C" entry points of rotary positions and the 8-bit paged K/V cache
// (include/pcd_kernels.h): argument checks, then one launch each.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <climits>
#include <cstdint>
#include <cstdlib>

#include "paged.h"
#include "pcd.h"
#include "pcd_kernels.h"

// Refuses the call with a code and pcd_last_error's text.
#define PCD_REFUSE(cond, code, detail)                    \
  do {                                                    \
    if (cond) return pcd::set_error(code, detail);        \
  } while (0)

namespace {

constexpr int64_t kMaxRows = int64_t{1} << 30;  // query rows (tokens x heads) of a call
constexpr int kMaxSeqs = 1 << 24;

int elem_size(int dtype) {
  switch (dtype) {
    case PCD_DTYPE_F32: return 4;
    case PCD_DTYPE_F16:
    case PCD_DTYPE_BF16: return 2;
    default: return 0;
  }
}
bool aligned(const void* p, int64_t n) { return reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(n) == 0; }

int device_sms() {
  int dev = 0, sms = 0;
  cudaGetDevice(&dev);
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  return sms > 0 ? sms : 152;  // no GPU here: a GB300's, so sizes can be asked for
}

int launched(int r) {
  if (r == 0) return PCD_OK;
  const cudaError_t e = cudaGetLastError();
  return pcd::set_error(PCD_ERR_CUDA, e == cudaSuccess ? "kernel launch failed" : cudaGetErrorString(e));
}

// Limit of a pipeline's waits: 2 s, or PCD_WAIT_LIMIT_MS as the process's first call finds it.
uint64_t wait_limit_ns() {
  static const uint64_t ns = [] {
    const char* ms = std::getenv("PCD_WAIT_LIMIT_MS");
    return ms ? static_cast<uint64_t>(std::atof(ms) * 1e6) : uint64_t{2000000000};
  }();
  return ns;
}

int check_rope(const pcd::RopeSpec& r, int dim) {
  PCD_REFUSE(r.rot < 0 || r.rot % 2 || r.rot > dim, PCD_ERR_INVALID_ARG, "rot_dim is even and at most head_dim");
  PCD_REFUSE((r.rot > 0) != (r.freqs != nullptr), PCD_ERR_INVALID_ARG, "freqs go with rot_dim > 0");
  PCD_REFUSE(!aligned(r.freqs, 8), PCD_ERR_INVALID_ARG, "freqs: unaligned pointer");
  PCD_REFUSE(!std::isfinite(r.amp), PCD_ERR_INVALID_ARG, "amp is not finite");
  return PCD_OK;
}

int log2_page(int page) {
  for (int s = 4; s <= 7; ++s)
    if (page == 1 << s) return s;
  return -1;
}

// Rows of a view along one axis: n of them, `stride` bytes apart.
struct Axis {
  int64_t stride, n;
};
// Do two rows of `width` bytes meet, whose places differ by delta + sum d_i stride_i, |d_i| < n_i, one row being another
// than itself (`other`: it is another view's) ?  Axes by falling stride: where each stride holds all that the axes
// after it span, at most two d_i of an axis come near.
bool rows_meet(__int128 delta, int64_t width, const Axis* ax, int k, bool other) {
  if (k == 0) return other && delta < width && -delta < width;
  __int128 span = width;  // of the axes after this one
  for (int i = 1; i < k; ++i) span += static_cast<__int128>(ax[i].n - 1) * ax[i].stride;
  const __int128 s = ax->stride, n = ax->n;
  auto floor_div = [](__int128 a, __int128 b) { return a / b - (a % b < 0 ? 1 : 0); };
  const __int128 lo = floor_div(-span - delta, s) + 1, hi = -(floor_div(delta - span, s) + 1);  // |delta + d s| < span
  for (__int128 d = lo < 1 - n ? 1 - n : lo; d <= hi && d < n; ++d)
    if (rows_meet(delta + d * s, width, ax + 1, k - 1, other || d != 0)) return true;
  return false;
}
// The axes of more than one row, by falling stride; returns how many.
int order_axes(Axis* ax, int k) {
  k = static_cast<int>(std::remove_if(ax, ax + k, [](const Axis& a) { return a.n <= 1; }) - ax);
  std::sort(ax, ax + k, [](const Axis& a, const Axis& b) { return a.stride > b.stride; });
  return k;
}
// Does some byte belong to two of a view's rows?
bool rows_overlap(int64_t width, Axis* ax, int k) {
  k = order_axes(ax, k);
  if (k > 0 && ax[k - 1].stride < 1) return true;
  __int128 span = width;
  for (int i = k - 1; i >= 0; --i) {
    if (ax[i].stride < span) return rows_meet(0, width, ax, k, false);
    span += static_cast<__int128>(ax[i].n - 1) * ax[i].stride;
  }
  return false;
}
bool rows_overlap(int64_t es, int64_t n, int64_t h, int64_t d, int64_t tok, int64_t head) {
  if (head >= d && tok >= static_cast<__int128>(h - 1) * head + d) return false;  // as nearly always: heads within a token
  Axis ax[2] = {{tok * es, n}, {head * es, h}};
  return rows_overlap(d * es, ax, 2);
}
bool codes_overlap(const pcd::PagesView& c) {
  // as nearly always: slots within heads or heads within slots, both within pages
  const int64_t slots = int64_t{1} << c.page_log2, lo = std::min(c.tok_stride, c.head_stride), hi = std::max(c.tok_stride, c.head_stride);
  const int64_t n_lo = c.tok_stride < c.head_stride ? slots : c.Hkv, n_hi = c.tok_stride < c.head_stride ? c.Hkv : slots;
  const __int128 inner = static_cast<__int128>(n_lo - 1) * lo + c.dim;
  if (lo >= c.dim && hi >= inner && c.page_stride >= static_cast<__int128>(n_hi - 1) * hi + inner) return false;
  Axis ax[3] = {{c.page_stride, c.n_pages}, {c.head_stride, c.Hkv}, {c.tok_stride, int64_t{1} << c.page_log2}};
  return rows_overlap(c.dim, ax, 3);
}
// Do keys and values, or their scales, share a byte?  (Of a cache whose rows share none.)
bool keys_meet_values(const pcd::PagesView& c) {
  const int64_t scales = static_cast<int64_t>(c.n_pages) * c.Hkv;
  if (c.ks < c.vs + scales && c.vs < c.ks + scales) return true;
  Axis ax[3] = {{c.page_stride, c.n_pages}, {c.head_stride, c.Hkv}, {c.tok_stride, int64_t{1} << c.page_log2}};
  const __int128 delta = reinterpret_cast<intptr_t>(c.v) - reinterpret_cast<intptr_t>(c.k);
  __int128 span = c.dim;
  for (const Axis& a : ax) span += static_cast<__int128>(a.n - 1) * a.stride;
  if (delta >= span || -delta >= span) return false;
  const int k = order_axes(ax, 3);
  return rows_meet(delta, c.dim, ax, k, true);
}

// The cache as the kernels take it.
int view_pages(const pcd_kv_pages* c, pcd::PagesView* v) {
  PCD_REFUSE(!c || !c->k || !c->v || !c->k_scale || !c->v_scale, PCD_ERR_INVALID_ARG, "cache: NULL");
  const int shift = log2_page(c->page_size);
  PCD_REFUSE(shift < 0, PCD_ERR_INVALID_ARG, "page_size is 16, 32, 64 or 128");
  PCD_REFUSE(c->n_pages < 1 || c->n_kv_heads < 1 || c->n_kv_heads > 65535, PCD_ERR_INVALID_ARG,
             "cache: pages or KV heads out of range");
  PCD_REFUSE(c->format != PCD_KV_E4M3 && c->format != PCD_KV_INT8, PCD_ERR_INVALID_ARG, "cache: unknown format");
  PCD_REFUSE(c->head_dim != 64 && c->head_dim != 128, PCD_ERR_SHAPE_MISMATCH, "cache: head_dim is 64 or 128");
  const int64_t tok = c->token_stride, head = c->head_stride, page = c->page_stride;
  PCD_REFUSE(!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 4) || !aligned(c->v_scale, 4) ||
                 page % 16 || head % 16 || tok % 16,
             PCD_ERR_INVALID_ARG, "cache: rows of codes start at multiples of 16 bytes");
  PCD_REFUSE(tok > (1 << 24), PCD_ERR_INVALID_ARG, "cache: token_stride is at most 2^24");
  PCD_REFUSE(tok < c->head_dim || (c->n_kv_heads > 1 && head < c->head_dim) || (c->n_pages > 1 && page < c->head_dim),
             PCD_ERR_INVALID_ARG, "cache: strides overlap rows");
  *v = pcd::PagesView{static_cast<uint8_t*>(c->k), static_cast<uint8_t*>(c->v), c->k_scale, c->v_scale, page, head, tok,
                      c->n_pages, shift, c->n_kv_heads, c->head_dim, c->format};
  return PCD_OK;
}

int view_seqs(const int32_t* q_off, const int32_t* kv_len, const int32_t* table, int n_seq, int n_tok, int table_stride,
              int table_width, pcd::SeqView* v) {
  PCD_REFUSE(n_seq < 0 || n_tok < 0 || table_stride < 0 || table_width < 0 || n_seq > kMaxSeqs || n_tok > kMaxRows,
             PCD_ERR_INVALID_ARG, "sequences, rows or table width out of range");
  PCD_REFUSE(table_width > table_stride, PCD_ERR_INVALID_ARG, "table_width is at most table_stride");
  PCD_REFUSE(n_seq > 0 && (!q_off || !kv_len || (table_width > 0 && !table)), PCD_ERR_INVALID_ARG,
             "q_off, kv_len or table: NULL");
  PCD_REFUSE(!aligned(q_off, 4) || !aligned(kv_len, 4) || !aligned(table, 4), PCD_ERR_INVALID_ARG,
             "q_off, kv_len or table: unaligned pointer");
  *v = pcd::SeqView{q_off, kv_len, table, n_seq, n_tok, table_stride, table_width};
  return PCD_OK;
}

// May a kernel that reads the rows of x and then writes the same rows of y run
// on these two views (no two rows of y meet)?  They are the same view, or share
// no byte; that is decided exactly where their strides are equal, else by the
// span of their rows within a common token stride, or of all.
bool views_ok(const void* x, const void* y, int64_t es, int64_t n, int64_t h, int64_t d, int64_t xt, int64_t xh, int64_t yt,
              int64_t yh) {
  const int64_t xa = reinterpret_cast<int64_t>(x), ya = reinterpret_cast<int64_t>(y);
  const bool same = (xt == yt || n <= 1) && (xh == yh || h <= 1);
  if (x == y && same) return true;
  const int64_t xs = ((n - 1) * xt + (h - 1) * xh + d) * es, ys = ((n - 1) * yt + (h - 1) * yh + d) * es;
  if (xa + xs <= ya || ya + ys <= xa) return true;
  if (same) {
    Axis ax[2] = {{yt * es, n}, {yh * es, h}};
    const int k = order_axes(ax, 2);
    return !rows_meet(ya - xa, d * es, ax, k, true);
  }
  if (xt != yt || xt <= 0) return false;
  // rows interleave: side by side within the common token stride
  const int64_t row = xt * es, xr = ((h - 1) * xh + d) * es, yr = ((h - 1) * yh + d) * es;
  int64_t off = (ya - xa) % row;
  if (off < 0) off += row;
  return off >= xr && off + yr <= row;
}

}  // namespace

extern "C" int pcd_rope_freqs(int rot_dim, double theta, int scaling, double factor, double orig_len, double lo_turns,
                              double hi_turns, int64_t* freqs, float* amp) {
  PCD_REFUSE(rot_dim < 2 || rot_dim % 2 || !freqs, PCD_ERR_INVALID_ARG, "rot_dim is even and at least 2");
  PCD_REFUSE(!(theta > 1.0) || !std::isfinite(theta), PCD_ERR_INVALID_ARG, "theta is over 1");
  PCD_REFUSE(scaling < PCD_ROPE_NONE || scaling > PCD_ROPE_RAMP, PCD_ERR_INVALID_ARG, "unknown scaling");
  PCD_REFUSE(scaling != PCD_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor)), PCD_ERR_INVALID_ARG,
             "factor is at least 1");
  PCD_REFUSE(scaling == PCD_ROPE_BASE && rot_dim < 4, PCD_ERR_INVALID_ARG, "PCD_ROPE_BASE needs rot_dim >= 4");
  PCD_REFUSE(scaling >= PCD_ROPE_BANDS && (!(orig_len >= 1.0) || !std::isfinite(orig_len) || !(lo_turns > 0.0) ||
                                           !(hi_turns > lo_turns) || !std::isfinite(hi_turns)),
             PCD_ERR_INVALID_ARG, "orig_len >= 1 and 0 < lo_turns < hi_turns");
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  double base = theta;
  if (scaling == PCD_ROPE_BASE) base *= std::pow(factor, rot_dim / (rot_dim - 2.0));
  double lo = 0.0, hi = 0.0;
  if (scaling == PCD_ROPE_RAMP) {
    // pair index at which a pair turns `t` times over the original length
    auto at = [&](double t) { return rot_dim * std::log(orig_len / (t * kTwoPi)) / (2.0 * std::log(theta)); };
    lo = std::fmax(std::floor(at(hi_turns)), 0.0);
    hi = std::fmin(std::ceil(at(lo_turns)), rot_dim - 1.0);
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    const double f0 = std::pow(base, -2.0 * i / rot_dim);
    double stretched = 0.0;  // share of the pair that takes the divided frequency
    if (scaling == PCD_ROPE_LINEAR) {
      stretched = 1.0;
    } else if (scaling == PCD_ROPE_BANDS) {
      const double turns = orig_len * f0 / kTwoPi;
      stretched = 1.0 - std::fmin(std::fmax((turns - lo_turns) / (hi_turns - lo_turns), 0.0), 1.0);
    } else if (scaling == PCD_ROPE_RAMP) {
      // (hi below 0: the length is so short that even the first pair turns fewer than lo_turns times)
      stretched = hi > 0.0 ? std::fmin(std::fmax((i - lo) / std::fmax(hi - lo, 1e-3), 0.0), 1.0) : 1.0;
    }
    const double f = stretched > 0.0 ? f0 / factor * stretched + f0 * (1.0 - stretched) : f0;
    const double turns = f / kTwoPi;  // < 1/6: theta > 1 and factor >= 1
    freqs[i] = static_cast<int64_t>(static_cast<uint64_t>(std::ldexp(turns, 64)));
  }
  if (amp) *amp = scaling == PCD_ROPE_RAMP ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.f;
  return PCD_OK;
}

extern "C" int pcd_k_rope(const void* x, void* y, int dtype, int n_tok, int heads, int head_dim, int64_t x_tok,
                          int64_t x_head, int64_t y_tok, int64_t y_head, const int64_t* freqs, int rot_dim,
                          int interleaved, float amp, const int32_t* pos, int base, int transpose, void* stream) {
  const int es = elem_size(dtype);
  PCD_REFUSE(!es, PCD_ERR_INVALID_ARG, "unknown dtype");
  PCD_REFUSE(n_tok < 0 || heads < 0 || head_dim < 1 || head_dim > 1024, PCD_ERR_INVALID_ARG, "sizes out of range");
  pcd::RopeKArgs a{x, y, dtype, n_tok, heads, head_dim, x_tok, x_head, y_tok, y_head, {}, pos, base};
  a.rope = pcd::RopeSpec{freqs, rot_dim, interleaved != 0, amp, transpose != 0};
  const int rc = check_rope(a.rope, head_dim);
  if (rc != PCD_OK) return rc;
  if (n_tok == 0 || heads == 0) return PCD_OK;
  PCD_REFUSE(!x || !y || !aligned(x, es) || !aligned(y, es) || !aligned(pos, 4), PCD_ERR_INVALID_ARG,
             "NULL or unaligned pointer");
  PCD_REFUSE(x_tok < 0 || x_head < 0 || y_tok < 0 || y_head < 0, PCD_ERR_INVALID_ARG, "negative stride");
  PCD_REFUSE(rows_overlap(es, n_tok, heads, head_dim, y_tok, y_head), PCD_ERR_INVALID_ARG, "strides of y overlap rows");
  PCD_REFUSE(!views_ok(x, y, es, n_tok, heads, head_dim, x_tok, x_head, y_tok, y_head), PCD_ERR_INVALID_ARG,
             "x and y overlap without being the same view");
  PCD_REFUSE(static_cast<int64_t>(n_tok) * head_dim >= (int64_t{1} << 31), PCD_ERR_INVALID_ARG,
             "n_tok * head_dim is under 2^31");
  return launched(pcd::launch_rope(a, device_sms(), static_cast<cudaStream_t>(stream)));
}

extern "C" int pcd_k_kv_append_cols(const pcd_kv_pages* cache, const void* k, const void* v, int dtype, int64_t k_tok,
                                    int64_t k_head, int64_t v_tok, int64_t v_head, const int32_t* q_off,
                                    const int32_t* kv_len, const int32_t* table, int n_seq, int n_tok, int table_stride,
                                    int table_width, const int64_t* freqs, int rot_dim, int interleaved, float amp,
                                    const int32_t* pos, int* dev_err, void* stream) {
  pcd::AppendArgs a{};
  int rc = view_pages(cache, &a.c);
  if (rc == PCD_OK) rc = view_seqs(q_off, kv_len, table, n_seq, n_tok, table_stride, table_width, &a.q);
  if (rc != PCD_OK) return rc;
  const int es = elem_size(dtype);
  PCD_REFUSE(!es, PCD_ERR_INVALID_ARG, "unknown dtype");
  a.rope = pcd::RopeSpec{freqs, rot_dim, interleaved != 0, amp, 0};
  rc = check_rope(a.rope, a.c.dim);
  if (rc != PCD_OK) return rc;
  if (n_tok == 0 || n_seq == 0) return PCD_OK;
  PCD_REFUSE(!k || !v || !aligned(k, es) || !aligned(v, es) || !aligned(pos, 4) || !aligned(dev_err, 4),
             PCD_ERR_INVALID_ARG, "NULL or unaligned pointer");
  PCD_REFUSE(k_tok < 0 || k_head < 0 || v_tok < 0 || v_head < 0, PCD_ERR_INVALID_ARG, "negative stride");
  PCD_REFUSE(codes_overlap(a.c), PCD_ERR_INVALID_ARG, "cache: strides overlap rows");
  PCD_REFUSE(keys_meet_values(a.c), PCD_ERR_INVALID_ARG, "cache: keys and values in one place");
  a.k = k;
  a.v = v;
  a.dtype = dtype;
  a.k_tok = k_tok, a.k_head = k_head, a.v_tok = v_tok, a.v_head = v_head;
  a.pos = pos;
  a.err = dev_err;
  return launched(pcd::launch_kv_append(a, device_sms(), static_cast<cudaStream_t>(stream)));
}

extern "C" int pcd_k_kv_append(const pcd_kv_pages* cache, const void* k, const void* v, int dtype, int64_t k_tok,
                               int64_t k_head, int64_t v_tok, int64_t v_head, const int32_t* q_off,
                               const int32_t* kv_len, const int32_t* table, int n_seq, int n_tok, int table_stride,
                               const int64_t* freqs, int rot_dim, int interleaved, float amp, const int32_t* pos,
                               int* dev_err, void* stream) {
  return pcd_k_kv_append_cols(cache, k, v, dtype, k_tok, k_head, v_tok, v_head, q_off, kv_len, table, n_seq, n_tok,
                              table_stride, table_stride, freqs, rot_dim, interleaved, amp, pos, dev_err, stream);
}

namespace {
// Rows of partial states in scratch, and rows that say where theirs are.
int64_t attn_parts(int n_tok, int Hq, const pcd::PagedPlan& p) {
  if (p.stream) return static_cast<int64_t>(p.n_splits) * 2 * 16;
  return p.n_splits <= 1 || p.cluster ? 0 : static_cast<int64_t>(p.n_splits) * n_tok * Hq;
}
int64_t attn_scratch(int n_tok, int Hq, int dim, const pcd::PagedPlan& p) {
  return attn_parts(n_tok, Hq, p) * (dim * 4 + 8) + (p.stream ? static_cast<int64_t>(n_tok) * Hq * 8 : 0);
}
}  // namespace

extern "C" int64_t pcd_k_paged_attention_scratch_bytes(int n_tok, int n_seq, int n_q_heads, int n_kv_heads, int head_dim,
                                                       int64_t max_kv) {
  if (n_tok < 1 || n_seq < 1 || n_q_heads < 1 || n_kv_heads < 1 || n_q_heads % n_kv_heads || head_dim < 1 || max_kv < 0 ||
      static_cast<int64_t>(n_tok) * n_q_heads > kMaxRows)
    return 0;
  pcd::PagedPlan p;
  pcd::plan_paged_attention(n_tok, n_seq, n_q_heads / n_kv_heads, n_kv_heads, max_kv, device_sms(), &p);
  return attn_scratch(n_tok, n_q_heads, head_dim, p);
}

extern "C" int pcd_k_paged_attention_cols(const pcd_kv_pages* cache, const void* q, void* out, float* lse, int dtype,
                                          int n_q_heads, int64_t q_tok, int64_t q_head, int64_t out_tok,
                                          int64_t out_head, const int32_t* q_off, const int32_t* kv_len,
                                          const int32_t* table, int n_seq, int n_tok, int table_stride, int table_width,
                                          int64_t max_kv, int causal, float scale, void* scratch, int64_t scratch_bytes,
                                          int* dev_err, void* stream) {
  pcd::PagedAttnArgs a{};
  int rc = view_pages(cache, &a.c);
  if (rc == PCD_OK) rc = view_seqs(q_off, kv_len, table, n_seq, n_tok, table_stride, table_width, &a.q);
  if (rc != PCD_OK) return rc;
  PCD_REFUSE(dtype != PCD_DTYPE_F16 && dtype != PCD_DTYPE_BF16, PCD_ERR_INVALID_ARG, "queries are fp16 or bf16");
  PCD_REFUSE(n_q_heads < 1 || n_q_heads % a.c.Hkv || n_q_heads / a.c.Hkv > 128, PCD_ERR_INVALID_ARG,
             "query heads are 1 to 128 times the KV heads");
  PCD_REFUSE(!(scale > 0.f) || !std::isfinite(scale) || max_kv < 0, PCD_ERR_INVALID_ARG, "scale or max_kv out of range");
  PCD_REFUSE(static_cast<int64_t>(n_tok) * n_q_heads > kMaxRows, PCD_ERR_INVALID_ARG, "too many query rows");
  if (n_tok == 0 || n_seq == 0) return PCD_OK;
  PCD_REFUSE(!q || !out || !aligned(q, 2) || !aligned(out, 2) || !aligned(lse, 4) || !aligned(dev_err, 4),
             PCD_ERR_INVALID_ARG, "NULL or unaligned pointer");
  PCD_REFUSE(q_tok < 0 || q_head < 0 || out_tok < 0 || out_head < 0, PCD_ERR_INVALID_ARG, "negative stride");
  PCD_REFUSE(rows_overlap(2, n_tok, n_q_heads, a.c.dim, out_tok, out_head), PCD_ERR_INVALID_ARG,
             "strides of out overlap rows");
  PCD_REFUSE(!views_ok(q, out, 2, n_tok, n_q_heads, a.c.dim, q_tok, q_head, out_tok, out_head), PCD_ERR_INVALID_ARG,
             "q and out overlap without being the same view");
  a.x = q;
  a.out = out;
  a.lse = lse;
  a.dtype = dtype;
  a.Hq = n_q_heads;
  a.G = n_q_heads / a.c.Hkv;
  a.causal = causal != 0;
  a.x_tok = q_tok, a.x_head = q_head, a.out_tok = out_tok, a.out_head = out_head;
  a.scale_log2 = scale * 1.4426950408889634f;
  a.err = dev_err;
  a.wait_ns = wait_limit_ns();
  pcd::plan_paged_attention(n_tok, n_seq, a.G, a.c.Hkv, max_kv, device_sms(), &a.plan);
  const int64_t need = attn_scratch(n_tok, n_q_heads, a.c.dim, a.plan);
  if (need > 0) {
    PCD_REFUSE(!scratch || !aligned(scratch, 16) || scratch_bytes < need, PCD_ERR_INVALID_ARG,
               "scratch is smaller than pcd_k_paged_attention_scratch_bytes, or unaligned");
    const int64_t parts = attn_parts(n_tok, n_q_heads, a.plan);
    a.part_o = static_cast<float*>(scratch);
    a.part_ml = reinterpret_cast<float2*>(a.part_o + parts * a.c.dim);
    a.part_at = reinterpret_cast<int2*>(a.part_ml + parts);
  }
  return launched(pcd::launch_paged_attention(a, static_cast<cudaStream_t>(stream)));
}

extern "C" int pcd_k_paged_attention(const pcd_kv_pages* cache, const void* q, void* out, float* lse, int dtype,
                                     int n_q_heads, int64_t q_tok, int64_t q_head, int64_t out_tok, int64_t out_head,
                                     const int32_t* q_off, const int32_t* kv_len, const int32_t* table, int n_seq,
                                     int n_tok, int table_stride, int64_t max_kv, int causal, float scale, void* scratch,
                                     int64_t scratch_bytes, int* dev_err, void* stream) {
  return pcd_k_paged_attention_cols(cache, q, out, lse, dtype, n_q_heads, q_tok, q_head, out_tok, out_head, q_off, kv_len,
                                    table, n_seq, n_tok, table_stride, table_stride, max_kv, causal, scale, scratch,
                                    scratch_bytes, dev_err, stream);
}
