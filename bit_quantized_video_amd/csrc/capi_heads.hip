// capi_heads.hip -- C entry points of the 4-bit group-scaled layer, the head
// norms with rotary positions and the key-value cache: every argument is
// checked before anything is enqueued, as in capi.hip.
#include "hdq.h"
#include "heads.h"
#include "w4.h"

#include <math.h>

#include <algorithm>

namespace {

using namespace hdq;

int hip_status(hipError_t e) { return e == hipSuccess ? HDQ_OK : HDQ_ERR_HIP; }
bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

// ---- 4-bit weights -----------------------------------------------------------
bool w4_shape_ok(int64_t N, int64_t K, int32_t group) {
  return N > 0 && N <= HDQ_W4_MAX_ROWS && K > 0 && K <= HDQ_FP8_MAX_COLS && K % 32 == 0 &&
         (group == 32 || group == 64 || group == 128) && K % group == 0;
}

int check_w4(const hdq_w4_tensor& w) {
  if (!w4_shape_ok(w.N, w.K, w.group)) return HDQ_ERR_SHAPE;
  if (w.codes == nullptr || w.scale == nullptr) return HDQ_ERR_INVALID;
  if (!aligned(w.codes, 16) || !aligned(w.scale, 16) || !aligned(w.zero, 16)) return HDQ_ERR_SHAPE;
  return HDQ_OK;
}

// ---- heads -------------------------------------------------------------------
bool valid_dtype(int32_t t) { return t == HDQ_DTYPE_F32 || t == HDQ_DTYPE_BF16; }
// Strides past this cannot be those of device memory.
constexpr int64_t kMaxStride = int64_t(1) << 40;

// Whether a view's heads lie apart: strides in order, each at least what the smaller ones span.
bool apart(const hdq_heads& h, int64_t batch, int64_t length, int32_t dim) {
  struct { int64_t stride, n; } d[3] = {{h.batch_stride, batch}, {h.token_stride, length}, {h.head_stride, h.heads}};
  std::sort(d, d + 3, [](const auto& a, const auto& b) { return a.stride < b.stride; });
  __int128 span = dim;
  for (const auto& v : d) {
    if (v.n == 1) continue;
    if (v.stride < span) return false;
    span += (__int128)(v.n - 1) * v.stride;
  }
  return true;
}

// A view's own checks; `out`: no two of its elements may be one.
int check_heads(const hdq_heads& h, int64_t batch, int64_t length, int32_t dim, bool out) {
  if (h.data == nullptr) return HDQ_ERR_INVALID;
  if (!valid_dtype(h.dtype)) return HDQ_ERR_UNSUPPORTED;
  if (h.heads <= 0 || h.heads > HDQ_HEAD_MAX_HEADS) return HDQ_ERR_SHAPE;
  if (!aligned(h.data, h.dtype == HDQ_DTYPE_F32 ? 4 : 2)) return HDQ_ERR_SHAPE;
  for (const int64_t s : {h.batch_stride, h.token_stride, h.head_stride})
    if (s < 0 || s > kMaxStride) return HDQ_ERR_SHAPE;
  return out && !apart(h, batch, length, dim) ? HDQ_ERR_SHAPE : HDQ_OK;
}

// An output at its own input has the input's type and strides.
bool in_place_ok(const hdq_heads& in, const hdq_heads& out, int64_t batch, int64_t length) {
  return in.data != out.data || (in.dtype == out.dtype && (batch == 1 || in.batch_stride == out.batch_stride) &&
                                 (length == 1 || in.token_stride == out.token_stride) &&
                                 (in.heads == 1 || in.head_stride == out.head_stride));
}

// Whether the view's chunks of 8 elements are whole 16-byte words.
bool vectors(const hdq_heads& h, int32_t dim) {
  const int64_t step = h.dtype == HDQ_DTYPE_F32 ? 4 : 8;
  return dim % 8 == 0 && aligned(h.data, 16) && h.batch_stride % step == 0 && h.token_stride % step == 0 &&
         h.head_stride % step == 0;
}

bool tokens_ok(int64_t batch, int64_t length) {
  return batch >= 0 && length >= 0 && batch <= HDQ_FP8_MAX_ROWS && length <= HDQ_FP8_MAX_ROWS &&
         batch * length <= HDQ_FP8_MAX_ROWS;
}

int check_norm(const hdq_head_norm* n) {
  if (n == nullptr || n->kind == HDQ_HEAD_NORM_NONE) return HDQ_OK;
  if (n->kind != HDQ_HEAD_NORM_LAYER && n->kind != HDQ_HEAD_NORM_RMS) return HDQ_ERR_INVALID;
  if (!(n->eps >= 0.0f) || n->eps > 1e30f) return HDQ_ERR_INVALID;
  for (const float* p : {n->q_weight, n->q_bias, n->k_weight, n->k_bias})
    if (!aligned(p, 4)) return HDQ_ERR_SHAPE;
  return HDQ_OK;
}

int check_rope(const hdq_rope* r, int32_t dim) {
  if (r == nullptr || r->dim == 0) return HDQ_OK;
  if (r->layout != HDQ_ROPE_INTERLEAVED && r->layout != HDQ_ROPE_HALF) return HDQ_ERR_INVALID;
  if (r->turns == nullptr || r->positions == nullptr || !isfinite(r->scale)) return HDQ_ERR_INVALID;
  if (r->dim < 0 || r->dim > dim || r->dim % 2 != 0 || r->axes < 1 || r->axes > HDQ_ROPE_MAX_AXES) return HDQ_ERR_SHAPE;
  int64_t sum = 0;
  for (int a = 0; a < r->axes; ++a) {
    if (r->axis_dim[a] < 0 || r->axis_dim[a] % 2 != 0) return HDQ_ERR_SHAPE;
    sum += r->axis_dim[a];
  }
  if (sum != r->dim || !aligned(r->turns, 8) || !aligned(r->positions, 8)) return HDQ_ERR_SHAPE;
  for (const int64_t s : {r->pos_axis_stride, r->pos_batch_stride, r->pos_token_stride})
    if (s < 0 || s > kMaxStride) return HDQ_ERR_SHAPE;
  return HDQ_OK;
}

int check_cache(const hdq_kv_cache& c) {
  if (c.fmt != HDQ_CACHE_INT8 && c.fmt != HDQ_CACHE_FP8 && c.fmt != HDQ_CACHE_INT4) return HDQ_ERR_UNSUPPORTED;
  if (c.k_codes == nullptr || c.k_scale == nullptr || c.v_codes == nullptr || c.v_scale == nullptr) return HDQ_ERR_INVALID;
  if (c.dim <= 0 || c.dim > HDQ_HEAD_MAX_DIM || c.dim % 8 != 0 || c.heads <= 0 || c.heads > HDQ_HEAD_MAX_HEADS / 2)
    return HDQ_ERR_SHAPE;
  if (c.slots < 0 || c.slots > kMaxStride / ((int64_t)c.heads * c.dim)) return HDQ_ERR_SHAPE;
  const auto power = [](int32_t v) { return v > 0 && (v & (v - 1)) == 0; };
  if (c.group != c.dim && !(power(c.group) && c.group >= 8 && c.group <= c.dim && c.dim % c.group == 0)) return HDQ_ERR_SHAPE;
  if (!power(c.had_block) || c.had_block > 128 || c.dim % c.had_block != 0) return HDQ_ERR_SHAPE;
  if (!aligned(c.k_codes, 8) || !aligned(c.v_codes, 8) || !aligned(c.k_scale, 4) || !aligned(c.v_scale, 4)) return HDQ_ERR_SHAPE;
  return HDQ_OK;
}

HeadRows rows(const hdq_heads* in, const hdq_heads* out, const float* weight, const float* bias) {
  HeadRows r{};
  if (in != nullptr) r.x = in->data, r.xb = in->batch_stride, r.xt = in->token_stride, r.xh = in->head_stride;
  if (out != nullptr) r.y = out->data, r.yb = out->batch_stride, r.yt = out->token_stride, r.yh = out->head_stride;
  r.heads = in != nullptr ? in->heads : 0;
  r.weight = weight;
  r.bias = bias;
  return r;
}

void set_rope(const hdq_rope* r, HeadArgs& g) {
  if (r == nullptr || r->dim == 0) return;
  g.half = r->dim / 2;
  g.split = r->layout == HDQ_ROPE_HALF;
  g.axes = r->axes;
  g.axis_end[0] = r->axes > 1 ? r->axis_dim[0] / 2 : g.half;
  g.axis_end[1] = r->axes > 2 ? g.axis_end[0] + r->axis_dim[1] / 2 : g.half;
  g.scale = r->scale;
  g.turns = r->turns;
  g.positions = r->positions;
  g.pos_axis = r->pos_axis_stride;
  g.pos_batch = r->pos_batch_stride;
  g.pos_token = r->pos_token_stride;
}

void set_norm(const hdq_head_norm* n, HeadArgs& g) {
  if (n == nullptr) return;
  g.norm = n->kind;
  g.eps = n->eps;
}

}  // namespace

static_assert(HDQ_HEAD_MAX_DIM == kHeadMaxDim && HDQ_HEAD_MAX_HEADS == kHeadMaxHeads, "the header's limits are the kernels'");
static_assert(HDQ_HEAD_NORM_LAYER == kHeadNormLayer && HDQ_HEAD_NORM_RMS == kHeadNormRms, "as above");
static_assert(HDQ_CACHE_INT8 == kCacheInt8 && HDQ_CACHE_FP8 == kCacheFp8 && HDQ_CACHE_INT4 == kCacheInt4, "as above");

extern "C" {

size_t hdq_w4_bytes(int64_t N, int64_t K, int32_t group, int32_t buffer) {
  if (!w4_shape_ok(N, K, group)) return 0;
  switch (buffer) {
    case HDQ_W4_CODES: return w4_code_bytes(N, K);
    case HDQ_W4_SCALE: return w4_scale_count(N, K, group) * 2;
    case HDQ_W4_ZERO: return w4_scale_count(N, K, group);
    default: return 0;
  }
}

int hdq_w4_pack(const uint8_t* codes, const void* scale, const uint8_t* zero, const hdq_w4_tensor* out, void* stream) {
  if (codes == nullptr || scale == nullptr || out == nullptr || (zero == nullptr) != (out->zero == nullptr)) return HDQ_ERR_INVALID;
  const int st = check_w4(*out);
  if (st != HDQ_OK) return st;
  if (!aligned(codes, 4) || !aligned(scale, 2)) return HDQ_ERR_SHAPE;
  return hip_status(launch_w4_pack(codes, static_cast<const uint16_t*>(scale), zero, out->N, out->K, out->group,
                                   W4Out{out->codes, out->scale, out->zero}, static_cast<hipStream_t>(stream)));
}

int hdq_w4_quantize(const void* w, const hdq_w4_tensor* out, void* stream) {
  if (w == nullptr || out == nullptr) return HDQ_ERR_INVALID;
  const int st = check_w4(*out);
  if (st != HDQ_OK) return st;
  if (!aligned(w, 16)) return HDQ_ERR_SHAPE;
  return hip_status(launch_w4_quantize(static_cast<const uint16_t*>(w), out->N, out->K, out->group,
                                       W4Out{out->codes, out->scale, out->zero}, static_cast<hipStream_t>(stream)));
}

size_t hdq_w4_linear_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (M <= 0 || M > HDQ_W4_MAX_TOKENS || !w4_shape_ok(N, K, 32)) return 0;
  return w4_workspace(M, N, K);
}

int hdq_w4_linear(const void* x, int64_t M, const hdq_w4_tensor* w, void* y, int32_t y_dtype, void* ws, size_t ws_bytes,
                  void* stream) {
  if (w == nullptr || ((x == nullptr || y == nullptr) && M != 0)) return HDQ_ERR_INVALID;
  if (!valid_dtype(y_dtype)) return HDQ_ERR_UNSUPPORTED;
  if (M < 0 || M > HDQ_W4_MAX_TOKENS) return HDQ_ERR_SHAPE;
  const int st = check_w4(*w);
  if (st != HDQ_OK) return st;
  if (M == 0) return HDQ_OK;
  if (!aligned(x, 16) || !aligned(y, y_dtype == HDQ_DTYPE_F32 ? 4 : 2)) return HDQ_ERR_SHAPE;
  const size_t need = w4_workspace(M, w->N, w->K);
  if (need > 0 && (ws == nullptr || ws_bytes < need)) return HDQ_ERR_WORKSPACE;
  if (need > 0 && !aligned(ws, 16)) return HDQ_ERR_SHAPE;
  return hip_status(launch_w4(static_cast<const uint16_t*>(x), M, W4Weights{w->codes, w->scale, w->zero, w->N, w->K, w->group},
                              y, y_dtype == HDQ_DTYPE_F32, ws, static_cast<hipStream_t>(stream)));
}

int hdq_rope_turns(int32_t dim, double base, int32_t scaling, double factor, double length, double slow, double fast,
                   double* turns_host) {
  if (turns_host == nullptr || scaling < HDQ_ROPE_SCALE_NONE || scaling > HDQ_ROPE_SCALE_RAMP) return HDQ_ERR_INVALID;
  if (dim <= 0 || dim % 2 != 0 || dim > HDQ_HEAD_MAX_DIM) return HDQ_ERR_SHAPE;
  if (!(base > 0.0) || !isfinite(base)) return HDQ_ERR_INVALID;
  if (scaling != HDQ_ROPE_SCALE_NONE && (!(factor >= 1.0) || !isfinite(factor))) return HDQ_ERR_INVALID;
  if (scaling == HDQ_ROPE_SCALE_BASE) {
    if (dim <= 2) return HDQ_ERR_SHAPE;
    base *= pow(factor, (double)dim / (dim - 2));
  }
  if (scaling == HDQ_ROPE_SCALE_RAMP && !(length > 0.0 && isfinite(length) && slow >= 0.0 && slow < fast && isfinite(fast)))
    return HDQ_ERR_INVALID;
  for (int j = 0; j < dim / 2; ++j) {
    const double t = pow(base, -2.0 * j / dim) / 6.283185307179586476925286766559;
    double keep = 1.0;  // share of the unscaled frequency
    if (scaling == HDQ_ROPE_SCALE_LINEAR) keep = 0.0;
    if (scaling == HDQ_ROPE_SCALE_RAMP) keep = fmin(fmax((length * t - slow) / (fast - slow), 0.0), 1.0);
    turns_host[j] = keep == 1.0 ? t : t * keep + t / factor * (1.0 - keep);
  }
  return HDQ_OK;
}

int hdq_qk_norm_rope(const hdq_heads* q, const hdq_heads* k, int64_t batch, int64_t length, int32_t dim,
                     const hdq_head_norm* norm, const hdq_rope* rope, const hdq_heads* q_out,
                     const hdq_heads* k_out, void* stream) {
  if (q == nullptr || q_out == nullptr || (k == nullptr) != (k_out == nullptr)) return HDQ_ERR_INVALID;
  if (!tokens_ok(batch, length) || dim <= 0 || dim > HDQ_HEAD_MAX_DIM) return HDQ_ERR_SHAPE;
  int st;
  if ((st = check_norm(norm)) != HDQ_OK || (st = check_rope(rope, dim)) != HDQ_OK) return st;
  if (batch * length == 0) return HDQ_OK;
  bool vec = true;
  for (const hdq_heads* h : {q, k, q_out, k_out}) {
    if (h == nullptr) continue;
    if ((st = check_heads(*h, batch, length, dim, h == q_out || h == k_out)) != HDQ_OK) return st;
    vec = vec && vectors(*h, dim);
  }
  if (q_out->heads != q->heads) return HDQ_ERR_SHAPE;
  if (k != nullptr) {
    if (k->dtype != q->dtype || k_out->dtype != q_out->dtype) return HDQ_ERR_UNSUPPORTED;
    if (k_out->heads != k->heads || k->heads > HDQ_HEAD_MAX_HEADS - q->heads) return HDQ_ERR_SHAPE;
    if (!in_place_ok(*k, *k_out, batch, length)) return HDQ_ERR_SHAPE;
    if (q_out->data == k->data || k_out->data == q->data || q_out->data == k_out->data) return HDQ_ERR_INVALID;
  }
  if (!in_place_ok(*q, *q_out, batch, length)) return HDQ_ERR_SHAPE;
  HeadArgs g{};
  g.q = rows(q, q_out, norm ? norm->q_weight : nullptr, norm ? norm->q_bias : nullptr);
  g.k = rows(k, k_out, norm ? norm->k_weight : nullptr, norm ? norm->k_bias : nullptr);
  g.tokens = batch * length;
  g.length = length;
  g.dim = dim;
  g.y_f32 = q_out->dtype == HDQ_DTYPE_F32;
  g.hb = 1;
  set_norm(norm, g);
  set_rope(rope, g);
  return hip_status(launch_heads(g, q->dtype == HDQ_DTYPE_F32, vec, false, static_cast<hipStream_t>(stream)));
}

int hdq_qkv_to_cache(const hdq_heads* q, const hdq_heads* k, const hdq_heads* v, int64_t batch, int64_t length,
                     const hdq_head_norm* norm, const hdq_rope* rope, const hdq_heads* q_out,
                     const int64_t* slots, const hdq_kv_cache* cache, void* stream) {
  if (k == nullptr || v == nullptr || cache == nullptr || (q == nullptr) != (q_out == nullptr)) return HDQ_ERR_INVALID;
  int st;
  if ((st = check_cache(*cache)) != HDQ_OK) return st;
  if (!tokens_ok(batch, length)) return HDQ_ERR_SHAPE;
  const int32_t dim = cache->dim;
  if ((st = check_norm(norm)) != HDQ_OK || (st = check_rope(rope, dim)) != HDQ_OK) return st;
  if (batch * length == 0) return HDQ_OK;
  if (slots == nullptr) return HDQ_ERR_INVALID;
  if (!aligned(slots, 8)) return HDQ_ERR_SHAPE;
  bool vec = true;
  for (const hdq_heads* h : {q, k, v, q_out}) {
    if (h == nullptr) continue;
    if ((st = check_heads(*h, batch, length, dim, h == q_out)) != HDQ_OK) return st;
    vec = vec && vectors(*h, dim);
  }
  if (k->heads != cache->heads || v->heads != cache->heads) return HDQ_ERR_SHAPE;
  if (v->dtype != k->dtype || (q != nullptr && q->dtype != k->dtype)) return HDQ_ERR_UNSUPPORTED;
  if (q != nullptr) {
    if (q_out->heads != q->heads || q->heads > HDQ_HEAD_MAX_HEADS - 2 * k->heads) return HDQ_ERR_SHAPE;
    if (!in_place_ok(*q, *q_out, batch, length)) return HDQ_ERR_SHAPE;
    if (q_out->data == k->data || q_out->data == v->data) return HDQ_ERR_INVALID;
  }
  HeadArgs g{};
  g.q = rows(q, q_out, norm ? norm->q_weight : nullptr, norm ? norm->q_bias : nullptr);
  g.k = rows(k, nullptr, norm ? norm->k_weight : nullptr, norm ? norm->k_bias : nullptr);
  g.v = rows(v, nullptr, nullptr, nullptr);
  g.tokens = batch * length;
  g.length = length;
  g.dim = dim;
  g.y_f32 = q_out != nullptr && q_out->dtype == HDQ_DTYPE_F32;
  set_norm(norm, g);
  set_rope(rope, g);
  g.fmt = cache->fmt;
  g.group = cache->group;
  g.groups = dim / cache->group;
  g.hb = cache->had_block;
  g.c_b = hadamard_scale(g.hb);
  g.top = cache_top(g.fmt);
  g.slots = slots;
  g.n_slots = cache->slots;
  g.codes[0] = cache->k_codes, g.codes[1] = cache->v_codes;
  g.scales[0] = cache->k_scale, g.scales[1] = cache->v_scale;
  return hip_status(launch_heads(g, k->dtype == HDQ_DTYPE_F32, vec, true, static_cast<hipStream_t>(stream)));
}

int hdq_cache_read(const hdq_kv_cache* cache, const int64_t* slots, int64_t tokens, void* k_out, void* v_out,
                   int32_t y_dtype, void* stream) {
  if (cache == nullptr) return HDQ_ERR_INVALID;
  if (!valid_dtype(y_dtype)) return HDQ_ERR_UNSUPPORTED;
  int st;
  if ((st = check_cache(*cache)) != HDQ_OK) return st;
  if (tokens < 0 || tokens > HDQ_FP8_MAX_ROWS) return HDQ_ERR_SHAPE;
  if (tokens == 0) return HDQ_OK;
  if (slots == nullptr || k_out == nullptr || v_out == nullptr) return HDQ_ERR_INVALID;
  if (!aligned(slots, 8) || !aligned(k_out, 16) || !aligned(v_out, 16)) return HDQ_ERR_SHAPE;
  CacheReadArgs g{};
  g.codes[0] = cache->k_codes, g.codes[1] = cache->v_codes;
  g.scales[0] = cache->k_scale, g.scales[1] = cache->v_scale;
  g.y[0] = k_out, g.y[1] = v_out;
  g.tokens = tokens;
  g.n_slots = cache->slots;
  g.slots = slots;
  g.heads = cache->heads;
  g.dim = cache->dim;
  g.fmt = cache->fmt;
  g.group = cache->group;
  g.groups = cache->dim / cache->group;
  g.hb = cache->had_block;
  g.c_b = hadamard_scale(g.hb);
  g.y_f32 = y_dtype == HDQ_DTYPE_F32;
  return hip_status(launch_cache_read(g, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
