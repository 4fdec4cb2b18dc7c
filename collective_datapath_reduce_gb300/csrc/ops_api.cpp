// C entry points of the index-driven operators: argument checks, then one of
// the launch functions of ops_*.cu.
#include <algorithm>
#include <cmath>
#include <exception>
#include <vector>

#include "ops.h"

namespace {

size_t size_of(int dtype) { return dtype == PL_F32 ? 4 : 2; }

purlin_status check_dtype(int dtype) { return dtype == PL_F32 || dtype == PL_BF16 ? PL_OK : PL_ERR_UNSUPPORTED; }

// Bytes from the first to past the last of `rows` rows of `width` elements,
// `stride` elements apart; false where they do not fit 64 bits.
bool extent(uint64_t rows, uint64_t width, uint64_t stride, uint64_t elem, uint64_t* bytes) {
  *bytes = 0;
  if (rows == 0 || width == 0) return true;
  uint64_t e;
  return !__builtin_mul_overflow(rows - 1, stride, &e) && !__builtin_add_overflow(e, width, &e) &&
         !__builtin_mul_overflow(e, elem, bytes);
}

// The buffers of one call: checked one by one, then against each other.
class Buffers {
 public:
  explicit Buffers(const pl::OpHandle& h) : h_(h) {}

  // `p`: rows x width elements; the address for the kernels comes back in it.
  template <typename P>
  purlin_status add(P** p, bool written, uint64_t rows, uint64_t width, uint64_t stride, uint64_t elem) {
    uint64_t bytes;
    if (stride < width || !extent(rows, width, stride, elem, &bytes)) return PL_ERR_INVALID_ARG;
    if (bytes == 0) return PL_OK;
    if (!*p) return PL_ERR_INVALID_ARG;
    const uintptr_t a = (uintptr_t)*p;
    if (a % elem) return PL_ERR_ALIGNMENT;
    if (a + bytes < a) return PL_ERR_INVALID_ARG;
    if (n_ == kMost) return PL_ERR_UNSUPPORTED;
    lo_[n_] = a;
    hi_[n_] = a + bytes;
    written_[n_++] = written;
    const void* q = nullptr;
    if (purlin_status st = pl::op_locate(h_, (const void*)*p, &q, &host_)) return st;
    *p = (P*)const_cast<void*>(q);
    return PL_OK;
  }

  // Some of them are host memory.
  bool host() const { return host_; }

  // No written buffer overlaps another one.
  purlin_status apart() const {
    for (int i = 0; i < n_; ++i)
      for (int j = 0; j < i; ++j)
        if ((written_[i] || written_[j]) && lo_[i] < hi_[j] && lo_[j] < hi_[i]) return PL_ERR_INVALID_ARG;
    return PL_OK;
  }

 private:
  static constexpr int kMost = 12;
  const pl::OpHandle& h_;
  uintptr_t lo_[kMost], hi_[kMost];
  bool written_[kMost], host_ = false;
  int n_ = 0;
};

purlin_status check_routing(const purlin_routing* r) {
  if (!r) return PL_ERR_INVALID_ARG;
  if (r->experts < 1 || r->experts > PURLIN_MAX_EXPERTS) return PL_ERR_INVALID_ARG;
  if (r->top_k < 1 || r->top_k > PURLIN_MAX_TOP_K || r->top_k > r->experts) return PL_ERR_INVALID_ARG;
  if (r->scores != PL_SCORES_SOFTMAX && r->scores != PL_SCORES_SIGMOID) return PL_ERR_UNSUPPORTED;
  if (r->groups < 1 || r->groups > PURLIN_MAX_GROUPS || r->experts % r->groups) return PL_ERR_INVALID_ARG;
  if (r->kept_groups < 1 || r->kept_groups > r->groups) return PL_ERR_INVALID_ARG;
  if (r->top_k > r->kept_groups * (r->experts / r->groups)) return PL_ERR_INVALID_ARG;
  if (r->group_best != 1 && r->group_best != 2) return PL_ERR_UNSUPPORTED;
  if (!std::isfinite(r->scale)) return PL_ERR_INVALID_ARG;
  return PL_OK;
}

// tokens x top_k picks are numbered by 32-bit places
purlin_status check_picks(size_t tokens, int top_k) {
  if (top_k < 1 || top_k > PURLIN_MAX_TOP_K) return PL_ERR_INVALID_ARG;
  return tokens > (size_t)0x7FFFFFFF / (size_t)top_k ? PL_ERR_UNSUPPORTED : PL_OK;
}

// `a` is `b` itself: read and written row by row in place.
bool same(const void* a, size_t a_stride, const void* b, size_t b_stride) { return a && a == b && a_stride == b_stride; }

purlin_status check_scores(int experts, int top_k, int scores, float scale) {
  if (experts < 1 || experts > PURLIN_MAX_EXPERTS) return PL_ERR_INVALID_ARG;
  if (top_k < 1 || top_k > PURLIN_MAX_TOP_K || top_k > experts) return PL_ERR_INVALID_ARG;
  if (scores != PL_SCORES_SOFTMAX && scores != PL_SCORES_SIGMOID) return PL_ERR_UNSUPPORTED;
  return std::isfinite(scale) ? PL_OK : PL_ERR_INVALID_ARG;
}

// The values that both directions of the distillation share.
purlin_status distil_args(const purlin_distillation* d, size_t tokens, pl::DistilArgs* a) {
  if (!d) return PL_ERR_INVALID_ARG;
  if (d->picks < 1 || d->picks > PURLIN_MAX_PICKS) return PL_ERR_INVALID_ARG;
  if (d->id_bytes != 4 && d->id_bytes != 8) return PL_ERR_UNSUPPORTED;
  if (check_dtype(d->teacher_dtype)) return PL_ERR_UNSUPPORTED;
  if (!(d->temperature >= 1e-30f && d->temperature <= 1e30f) || !std::isfinite(d->scale)) return PL_ERR_INVALID_ARG;
  if (d->first < 0 || d->vocabulary < d->first || (uint64_t)(d->vocabulary - d->first) < d->width) return PL_ERR_INVALID_ARG;
  if (tokens > SIZE_MAX / PURLIN_MAX_PICKS / 8) return PL_ERR_INVALID_ARG;
  *a = {};
  a->tokens = tokens;
  a->width = d->width;
  a->first = d->first;
  a->vocabulary = d->vocabulary;
  a->wide_ids = d->id_bytes == 8;
  a->picks = d->picks;
  a->teacher_bf16 = d->teacher_dtype == PL_BF16;
  a->temperature = d->temperature;
  a->scale = d->scale;
  a->log2e_per_temperature = (float)(1.4426950408889634 / (double)d->temperature);
  return PL_OK;
}

pl::RouteArgs route_args(const purlin_routing* r, size_t tokens) {
  pl::RouteArgs a = {};
  a.tokens = tokens;
  a.experts = r->experts;
  a.top_k = r->top_k;
  a.sigmoid = r->scores == PL_SCORES_SIGMOID;
  a.groups = r->groups;
  a.kept = r->kept_groups;
  a.best = r->group_best;
  a.renormalise = r->renormalise != 0;
  a.scale = r->scale;
  return a;
}

}  // namespace

extern "C" {

purlin_status purlin_route_experts(purlin_handle handle, const void* logits, size_t stride, purlin_dtype dtype,
                                   const float* bias, size_t tokens, const purlin_routing* routing, int32_t* ids,
                                   float* weights, purlin_stream_t stream) {
  pl::OpHandle h;
  purlin_status st;
  if ((st = pl::op_begin(handle, &h)) || (st = check_dtype(dtype)) || (st = check_routing(routing)) ||
      (st = check_picks(tokens, routing->top_k)))
    return st;
  const uint64_t E = (uint64_t)routing->experts, k = (uint64_t)routing->top_k;
  pl::RouteArgs a = route_args(routing, tokens);
  Buffers b(h);
  if ((st = b.add(&logits, false, tokens, E, stride, size_of(dtype))) ||
      (bias && (st = b.add(&bias, false, 1, E, E, 4))) || (st = b.add(&ids, true, tokens, k, k, 4)) ||
      (st = b.add(&weights, true, tokens, k, k, 4)) || (st = b.apart()))
    return st;
  if (tokens == 0) return PL_OK;
  a.logits = logits;
  a.ld = stride;
  a.bias = bias;
  a.ids = ids;
  a.weights = weights;
  return pl::launch_route(a, dtype, (cudaStream_t)stream);
}

purlin_status purlin_route_experts_grad(purlin_handle handle, const void* logits, size_t stride, purlin_dtype dtype,
                                        size_t tokens, const purlin_routing* routing, const int32_t* ids,
                                        const float* grad_weights, void* grad_logits, size_t grad_stride,
                                        purlin_stream_t stream) {
  pl::OpHandle h;
  purlin_status st;
  if ((st = pl::op_begin(handle, &h)) || (st = check_dtype(dtype)) || (st = check_routing(routing)) ||
      (st = check_picks(tokens, routing->top_k)))
    return st;
  const uint64_t E = (uint64_t)routing->experts, k = (uint64_t)routing->top_k;
  pl::RouteArgs a = route_args(routing, tokens);
  Buffers b(h);
  if ((st = b.add(&logits, false, tokens, E, stride, size_of(dtype))) || (st = b.add(&ids, false, tokens, k, k, 4)) ||
      (st = b.add(&grad_weights, false, tokens, k, k, 4)) ||
      (st = b.add(&grad_logits, true, tokens, E, grad_stride, size_of(dtype))) || (st = b.apart()))
    return st;
  if (tokens == 0) return PL_OK;
  a.logits = logits;
  a.ld = stride;
  a.ids = const_cast<int32_t*>(ids);
  a.grad_weights = grad_weights;
  a.grad_logits = grad_logits;
  a.grad_ld = grad_stride;
  return pl::launch_route_grad(a, dtype, (cudaStream_t)stream);
}

size_t purlin_expert_plan_bytes(size_t tokens, int top_k, int experts) {
  if (check_picks(tokens, top_k) || experts < 1 || experts > PURLIN_MAX_EXPERTS) return 0;
  return pl::expert_plan_bytes((uint64_t)tokens * (uint64_t)top_k, experts);
}

purlin_status purlin_expert_plan(purlin_handle handle, const int32_t* ids, size_t tokens, int top_k, int experts,
                                 int32_t* offsets, int32_t* places, void* workspace, size_t workspace_bytes,
                                 purlin_stream_t stream) {
  pl::OpHandle h;
  purlin_status st;
  if ((st = pl::op_begin(handle, &h)) || (st = check_picks(tokens, top_k))) return st;
  if (experts < 1 || experts > PURLIN_MAX_EXPERTS) return PL_ERR_INVALID_ARG;
  const uint64_t slots = (uint64_t)tokens * (uint64_t)top_k, need = pl::expert_plan_bytes(slots, experts);
  if (workspace_bytes < need) return PL_ERR_WORKSPACE;
  Buffers b(h);
  if ((st = b.add(&ids, false, 1, slots, slots, 4)) ||
      (st = b.add(&offsets, true, 1, (uint64_t)experts + 1, (uint64_t)experts + 1, 4)) ||
      (st = b.add(&places, true, 1, slots, slots, 4)) || (st = b.add(&workspace, true, 1, need / 4, need / 4, 4)) ||
      (st = b.apart()))
    return st;
  pl::PlanArgs a = {};
  a.ids = ids;
  a.slots = slots;
  a.experts = experts;
  a.offsets = offsets;
  a.places = places;
  a.counts = (uint32_t*)workspace;
  return pl::launch_expert_plan(a, (cudaStream_t)stream);
}

purlin_status purlin_dispatch_rows(purlin_handle handle, const void* x, size_t x_stride, const int32_t* places,
                                   size_t tokens, int top_k, size_t width, purlin_dtype dtype, void* rows,
                                   size_t rows_stride, purlin_stream_t stream) {
  pl::OpHandle h;
  purlin_status st;
  if ((st = pl::op_begin(handle, &h)) || (st = check_dtype(dtype)) || (st = check_picks(tokens, top_k))) return st;
  const uint64_t slots = (uint64_t)tokens * (uint64_t)top_k, es = size_of(dtype);
  Buffers b(h);
  if ((st = b.add(&x, false, tokens, width, x_stride, es)) || (st = b.add(&places, false, 1, slots, slots, 4)) ||
      (st = b.add(&rows, true, slots, width, rows_stride, es)) || (st = b.apart()))
    return st;
  if (slots == 0 || width == 0) return PL_OK;
  pl::RowsArgs a = {};
  a.x = x;
  a.ldx = x_stride;
  a.y = rows;
  a.ldy = rows_stride;
  a.places = places;
  a.tokens = tokens;
  a.width = width;
  a.top_k = top_k;
  a.status = h.status;
  return pl::launch_dispatch(a, dtype, (cudaStream_t)stream);
}

purlin_status purlin_combine_rows(purlin_handle handle, const void* rows, size_t rows_stride, const int32_t* places,
                                  const float* weights, size_t tokens, int top_k, size_t width, purlin_dtype dtype,
                                  void* y, size_t y_stride, purlin_stream_t stream) {
  pl::OpHandle h;
  purlin_status st;
  if ((st = pl::op_begin(handle, &h)) || (st = check_dtype(dtype)) || (st = check_picks(tokens, top_k))) return st;
  const uint64_t slots = (uint64_t)tokens * (uint64_t)top_k, es = size_of(dtype);
  Buffers b(h);
  if ((st = b.add(&rows, false, slots, width, rows_stride, es)) || (st = b.add(&places, false, 1, slots, slots, 4)) ||
      (weights && (st = b.add(&weights, false, 1, slots, slots, 4))) ||
      (st = b.add(&y, true, tokens, width, y_stride, es)) || (st = b.apart()))
    return st;
  if (slots == 0 || width == 0) return PL_OK;
  pl::RowsArgs a = {};
  a.x = rows;
  a.ldx = rows_stride;
  a.y = y;
  a.ldy = y_stride;
  a.places = places;
  a.weights = weights;
  a.tokens = tokens;
  a.width = width;
  a.top_k = top_k;
  a.status = h.status;
  a.host = b.host();
  return pl::launch_combine(a, dtype, (cudaStream_t)stream);
}

purlin_status purlin_combine_rows_grad(purlin_handle handle, const void* rows, size_t rows_stride, const int32_t* places,
                                       const float* weights, const void* grad_y, size_t grad_y_stride, size_t tokens,
                                       int top_k, size_t width, purlin_dtype dtype, void* grad_rows,
                                       size_t grad_rows_stride, float* grad_weights, purlin_stream_t stream) {
  pl::OpHandle h;
  purlin_status st;
  if ((st = pl::op_begin(handle, &h)) || (st = check_dtype(dtype)) || (st = check_picks(tokens, top_k))) return st;
  const uint64_t slots = (uint64_t)tokens * (uint64_t)top_k, es = size_of(dtype);
  Buffers b(h);
  if ((st = b.add(&rows, false, slots, width, rows_stride, es)) || (st = b.add(&places, false, 1, slots, slots, 4)) ||
      (st = b.add(&weights, false, 1, slots, slots, 4)) ||
      (st = b.add(&grad_y, false, tokens, width, grad_y_stride, es)) ||
      (st = b.add(&grad_rows, true, slots, width, grad_rows_stride, es)) ||
      (st = b.add(&grad_weights, true, 1, slots, slots, 4)) || (st = b.apart()))
    return st;
  if (slots == 0) return PL_OK;
  pl::RowsArgs a = {};
  a.x = rows;
  a.ldx = rows_stride;
  a.y = grad_rows;
  a.ldy = grad_rows_stride;
  a.places = places;
  a.weights = weights;
  a.tokens = tokens;
  a.width = width;
  a.top_k = top_k;
  a.status = h.status;
  a.grad_y = grad_y;
  a.ldg = grad_y_stride;
  a.grad_weights = grad_weights;
  return pl::launch_combine_grad(a, dtype, (cudaStream_t)stream);
}

purlin_status purlin_embed(purlin_handle handle, const void* table, size_t table_stride, size_t rows, int64_t first,
                           const void* tokens, int token_bytes, size_t n, size_t width, float scale, purlin_dtype dtype,
                           void* out, size_t out_stride, purlin_stream_t stream) {
  pl::OpHandle h;
  purlin_status st;
  if ((st = pl::op_begin(handle, &h)) || (st = check_dtype(dtype))) return st;
  if (token_bytes != 4 && token_bytes != 8) return PL_ERR_UNSUPPORTED;
  const uint64_t es = size_of(dtype);
  Buffers b(h);
  if ((st = b.add(&table, false, rows, width, table_stride, es)) || (st = b.add(&tokens, false, 1, n, n, token_bytes)) ||
      (st = b.add(&out, true, n, width, out_stride, es)) || (st = b.apart()))
    return st;
  if (n == 0 || width == 0) return PL_OK;
  pl::EmbedArgs a = {};
  a.tokens = tokens;
  a.wide_tokens = token_bytes == 8;
  a.first = first;
  a.rows = rows;
  a.n = n;
  a.width = width;
  a.scale = scale;
  a.x = table;
  a.ldx = table_stride;
  a.y = out;
  a.ldy = out_stride;
  return pl::launch_embed(a, dtype, (cudaStream_t)stream);
}

size_t purlin_embed_grad_bytes(size_t tokens, size_t rows, size_t width) {
  if (tokens > 0x7FFFFFFFu || rows > 0x7FFFFFFFu || width > 0x7FFFFFFFu) return 0;
  return pl::embed_grad_bytes(tokens, rows, width);
}

purlin_status purlin_embed_grad(purlin_handle handle, const void* grad_out, size_t grad_out_stride,
                                purlin_dtype grad_out_dtype, const void* tokens, int token_bytes, size_t n, size_t width,
                                float scale, const void* base, size_t base_stride, void* grad_table,
                                size_t grad_table_stride, purlin_dtype grad_table_dtype, size_t rows, int64_t first,
                                void* workspace, size_t workspace_bytes, purlin_stream_t stream) {
  pl::OpHandle h;
  purlin_status st;
  if ((st = pl::op_begin(handle, &h)) || (st = check_dtype(grad_out_dtype)) || (st = check_dtype(grad_table_dtype)))
    return st;
  if (token_bytes != 4 && token_bytes != 8) return PL_ERR_UNSUPPORTED;
  if (n > 0x7FFFFFFFu || rows > 0x7FFFFFFFu || width > 0x7FFFFFFFu) return PL_ERR_UNSUPPORTED;
  const uint64_t xs = size_of(grad_out_dtype), ts = size_of(grad_table_dtype);
  const size_t need = pl::embed_grad_bytes(n, rows, width);
  if (workspace_bytes < need) return PL_ERR_WORKSPACE;
  if (need && ((uintptr_t)workspace & 15u)) return PL_ERR_ALIGNMENT;
  const bool in_place = base && base == grad_table && base_stride == grad_table_stride;
  Buffers b(h);
  if ((st = b.add(&grad_out, false, n, width, grad_out_stride, xs)) ||
      (st = b.add(&tokens, false, 1, n, n, token_bytes)) ||
      (base && !in_place && (st = b.add(&base, false, rows, width, base_stride, ts))) ||
      (st = b.add(&grad_table, true, rows, width, grad_table_stride, ts)) ||
      (st = b.add(&workspace, true, 1, need / 4, need / 4, 4)) || (st = b.apart()))
    return st;
  if (rows == 0 || width == 0) return PL_OK;
  pl::EmbedArgs a = {};
  a.tokens = tokens;
  a.wide_tokens = token_bytes == 8;
  a.first = first;
  a.rows = rows;
  a.n = n;
  a.width = width;
  a.scale = scale;
  a.x = grad_out;
  a.ldx = grad_out_stride;
  a.y = grad_table;
  a.ldy = grad_table_stride;
  a.base = in_place ? grad_table : base;
  a.ldb = in_place ? grad_table_stride : base ? base_stride : 0;
  a.workspace = workspace;
  return pl::launch_embed_grad(a, grad_out_dtype, grad_table_dtype, (cudaStream_t)stream);
}

size_t purlin_clip_grad_norm_bytes(void) { return pl::clip_bytes(); }

purlin_status purlin_clip_grad_norm(purlin_handle handle, const void* const* grads, void* const* outs, const size_t* counts,
                                    size_t n, purlin_dtype dtype, float scale, float max_norm, float* norm,
                                    void* workspace, size_t workspace_bytes, purlin_stream_t stream) {
  pl::OpHandle h;
  purlin_status st;
  if ((st = pl::op_begin(handle, &h)) || (st = check_dtype(dtype))) return st;
  if (n && (!grads || !counts)) return PL_ERR_INVALID_ARG;
  if (!std::isfinite(scale) || !(max_norm >= 0.f)) return PL_ERR_INVALID_ARG;
  if (workspace_bytes < pl::clip_bytes()) return PL_ERR_WORKSPACE;
  const uint64_t es = size_of(dtype);
  struct Span {
    uintptr_t lo, hi;
    bool written;
    size_t of;
  };
  try {
    bool host = false;  // either kind goes
    std::vector<Span> spans;
    std::vector<pl::ClipTensor> t;
    spans.reserve(2 * n + 2);
    t.reserve(n);
    auto add = [&](const void* p, uint64_t bytes, bool written, size_t of, uint64_t align, const void** q) {
      const uintptr_t a = (uintptr_t)p;
      if (!p || a + bytes < a) return PL_ERR_INVALID_ARG;
      if (a % align) return PL_ERR_ALIGNMENT;
      spans.push_back(Span{a, a + bytes, written, of});
      return pl::op_locate(h, p, q, &host);
    };
    for (size_t i = 0; i < n; ++i) {
      if (counts[i] == 0) continue;
      if (counts[i] > UINT64_MAX / es) return PL_ERR_INVALID_ARG;
      const void *in = nullptr, *out = nullptr;
      if ((st = add(grads[i], counts[i] * es, false, i, es, &in))) return st;
      if (outs && (st = add(outs[i], counts[i] * es, true, i, es, &out))) return st;
      t.push_back(pl::ClipTensor{in, const_cast<void*>(out), counts[i]});
    }
    const void *nq = nullptr, *wq = nullptr;
    if ((st = add(norm, 4, true, n, 4, &nq)) || (st = add(workspace, pl::clip_bytes(), true, n + 1, 8, &wq))) return st;
    // In the order of their starts (reads before writes), a span overlaps an
    // earlier one exactly if it starts before the furthest end so far.  Reads
    // may overlap reads; a write may lie on the read of its own gradient.
    std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) {
      return a.lo != b.lo ? a.lo < b.lo : a.written < b.written;
    });
    uintptr_t end_read = 0, end_read_before = 0, end_written = 0;  // _before: without the last span
    for (size_t i = 0; i < spans.size(); ++i) {
      const Span& s = spans[i];
      const Span* last = i ? &spans[i - 1] : nullptr;
      const bool in_place = s.written && last && !last->written && last->lo == s.lo && last->hi == s.hi &&
                            last->of == s.of && end_read_before <= s.lo;
      if (s.lo < end_written || (s.written && !in_place && s.lo < end_read)) return PL_ERR_INVALID_ARG;
      end_read_before = end_read;
      uintptr_t& end = s.written ? end_written : end_read;
      end = std::max(end, s.hi);
    }
    return pl::launch_clip(t.data(), t.size(), dtype, scale, max_norm, outs != nullptr, (float*)const_cast<void*>(nq),
                           (double*)const_cast<void*>(wq), h.sm_count, (cudaStream_t)stream);
  } catch (const std::exception&) {  // no memory for so many gradients
    return PL_ERR_INVALID_ARG;
  }
}

purlin_status purlin_layer_norm(purlin_handle handle, const void* x, size_t x_stride, const void* residual,
                                size_t residual_stride, size_t tokens, size_t width, purlin_dtype dtype,
                                const void* weight, const void* bias, purlin_dtype weight_dtype, float eps, void* y,
                                size_t y_stride, void* total, size_t total_stride, float* stats,
                                purlin_stream_t stream) {
  pl::OpHandle h;
  purlin_status st;
  if ((st = pl::op_begin(handle, &h)) || (st = check_dtype(dtype)) || (st = check_dtype(weight_dtype))) return st;
  if (!(eps >= 0.f) || !std::isfinite(eps)) return PL_ERR_INVALID_ARG;
  const uint64_t es = size_of(dtype), ws = size_of(weight_dtype);
  // y and the total may lie on x or on the residual, one on each
  const bool x_y = same(x, x_stride, y, y_stride), x_t = same(x, x_stride, total, total_stride);
  const bool r_y = same(residual, residual_stride, y, y_stride), r_t = same(residual, residual_stride, total, total_stride);
  Buffers b(h);
  if ((!x_y && !x_t && (st = b.add(&x, false, tokens, width, x_stride, es))) ||
      (residual && !r_y && !r_t && (st = b.add(&residual, false, tokens, width, residual_stride, es))) ||
      (weight && (st = b.add(&weight, false, 1, width, width, ws))) ||
      (bias && (st = b.add(&bias, false, 1, width, width, ws))) || (st = b.add(&y, true, tokens, width, y_stride, es)) ||
      (total && (st = b.add(&total, true, tokens, width, total_stride, es))) ||
      (stats && (st = b.add(&stats, true, tokens, 2, 2, 4))) || (st = b.apart()))
    return st;
  if (tokens == 0 || width == 0) return PL_OK;
  pl::NormArgs a = {};
  a.x = x_y ? y : x_t ? total : x;
  a.ldx = x_stride;
  a.residual = r_y ? y : r_t ? total : residual;
  a.ldr = residual_stride;
  a.weight = weight;
  a.bias = bias;
  a.y = y;
  a.ldy = y_stride;
  a.total = total;
  a.ldt = total_stride;
  a.stats = stats;
  a.tokens = tokens;
  a.width = width;
  a.eps = eps;
  return pl::launch_norm(a, dtype, weight_dtype, (cudaStream_t)stream);
}

size_t purlin_layer_norm_grad_bytes(size_t tokens, size_t width) {
  return width > 0x7FFFFFFFu ? 0 : pl::norm_grad_bytes(tokens, width);
}

purlin_status purlin_layer_norm_grad(purlin_handle handle, const void* grad_y, size_t grad_y_stride, const void* x,
                                     size_t x_stride, const float* stats, size_t tokens, size_t width,
                                     purlin_dtype dtype, const void* weight, purlin_dtype weight_dtype,
                                     const void* grad_total, size_t grad_total_stride, void* grad_x,
                                     size_t grad_x_stride, void* grad_weight, void* grad_bias, void* workspace,
                                     size_t workspace_bytes, purlin_stream_t stream) {
  pl::OpHandle h;
  purlin_status st;
  if ((st = pl::op_begin(handle, &h)) || (st = check_dtype(dtype)) || (st = check_dtype(weight_dtype))) return st;
  if (width > 0x7FFFFFFFu) return PL_ERR_UNSUPPORTED;
  const uint64_t es = size_of(dtype), ws = size_of(weight_dtype);
  const size_t need = grad_weight || grad_bias ? pl::norm_grad_bytes(tokens, width) : 0;
  if (workspace_bytes < need) return PL_ERR_WORKSPACE;
  // grad_x may lie on one of the three that have its rows
  const bool on_x = same(x, x_stride, grad_x, grad_x_stride), on_g = same(grad_y, grad_y_stride, grad_x, grad_x_stride);
  const bool on_t = same(grad_total, grad_total_stride, grad_x, grad_x_stride);
  Buffers b(h);
  if ((!on_g && (st = b.add(&grad_y, false, tokens, width, grad_y_stride, es))) ||
      (!on_x && (st = b.add(&x, false, tokens, width, x_stride, es))) ||
      (grad_total && !on_t && (st = b.add(&grad_total, false, tokens, width, grad_total_stride, es))) ||
      (st = b.add(&stats, false, tokens, 2, 2, 4)) || (weight && (st = b.add(&weight, false, 1, width, width, ws))) ||
      (st = b.add(&grad_x, true, tokens, width, grad_x_stride, es)) ||
      (grad_weight && (st = b.add(&grad_weight, true, 1, width, width, ws))) ||
      (grad_bias && (st = b.add(&grad_bias, true, 1, width, width, ws))) ||
      (st = b.add(&workspace, true, 1, need / 4, need / 4, 4)) || (st = b.apart()))
    return st;
  if (width == 0) return PL_OK;
  pl::NormArgs a = {};
  a.x = on_x ? grad_x : x;
  a.ldx = x_stride;
  a.stats = const_cast<float*>(stats);
  a.tokens = tokens;
  a.width = width;
  a.weight = weight;
  a.grad_y = on_g ? grad_x : grad_y;
  a.ldg = grad_y_stride;
  a.grad_total = on_t ? grad_x : grad_total;
  a.ldgt = grad_total_stride;
  a.y = grad_x;
  a.ldy = grad_x_stride;
  a.grad_weight = grad_weight;
  a.grad_bias = grad_bias;
  a.parts = (float*)workspace;
  return pl::launch_norm_grad(a, dtype, weight_dtype, (cudaStream_t)stream);
}

size_t purlin_balance_loss_bytes(size_t tokens, int experts) {
  return experts < 1 || experts > PURLIN_MAX_EXPERTS ? 0 : pl::balance_bytes(tokens, experts);
}

purlin_status purlin_balance_loss(purlin_handle handle, const void* logits, size_t stride, purlin_dtype dtype,
                                  const int32_t* ids, size_t tokens, int top_k, int experts, purlin_scores scores,
                                  float scale, int32_t* counts, float* sums, float* loss, void* workspace,
                                  size_t workspace_bytes, purlin_stream_t stream) {
  pl::OpHandle h;
  purlin_status st;
  if ((st = pl::op_begin(handle, &h)) || (st = check_dtype(dtype)) || (st = check_scores(experts, top_k, scores, scale)) ||
      (st = check_picks(tokens, top_k)))
    return st;
  const uint64_t E = (uint64_t)experts, k = (uint64_t)top_k;
  const size_t need = pl::balance_bytes(tokens, experts);
  if (workspace_bytes < need) return PL_ERR_WORKSPACE;
  Buffers b(h);
  if ((st = b.add(&logits, false, tokens, E, stride, size_of(dtype))) || (st = b.add(&ids, false, tokens, k, k, 4)) ||
      (st = b.add(&counts, true, 1, E, E, 4)) || (st = b.add(&sums, true, 1, 2 * E + 1, 2 * E + 1, 4)) ||
      (loss && (st = b.add(&loss, true, 1, 1, 1, 4))) || (st = b.add(&workspace, true, 1, need / 4, need / 4, 4)) ||
      (st = b.apart()))
    return st;
  pl::BalanceArgs a = {};
  a.logits = logits;
  a.ld = stride;
  a.tokens = tokens;
  a.experts = experts;
  a.top_k = top_k;
  a.sigmoid = scores == PL_SCORES_SIGMOID;
  a.scale = scale;
  a.ids = ids;
  a.counts = counts;
  a.sums = sums;
  a.loss = loss;
  a.parts = (uint32_t*)workspace;
  return pl::launch_balance(a, dtype, (cudaStream_t)stream);
}

purlin_status purlin_balance_join(purlin_handle handle, const float* sums, int experts, float scale, float* loss,
                                  purlin_stream_t stream) {
  pl::OpHandle h;
  purlin_status st;
  if ((st = pl::op_begin(handle, &h)) || (st = check_scores(experts, 1, PL_SCORES_SOFTMAX, scale))) return st;
  const uint64_t n = 2 * (uint64_t)experts + 1;
  Buffers b(h);
  if ((st = b.add(&sums, false, 1, n, n, 4)) || (st = b.add(&loss, true, 1, 1, 1, 4)) || (st = b.apart())) return st;
  pl::BalanceArgs a = {};
  a.experts = experts;
  a.scale = scale;
  a.sums = const_cast<float*>(sums);
  a.loss = loss;
  return pl::launch_balance_join(a, (cudaStream_t)stream);
}

purlin_status purlin_balance_loss_grad(purlin_handle handle, const void* logits, size_t stride, purlin_dtype dtype,
                                       const int32_t* ids, size_t tokens, int top_k, int experts, purlin_scores scores,
                                       float scale, const float* sums, const float* grad_loss, const void* base,
                                       size_t base_stride, void* grad_logits, size_t grad_stride,
                                       purlin_stream_t stream) {
  pl::OpHandle h;
  purlin_status st;
  if ((st = pl::op_begin(handle, &h)) || (st = check_dtype(dtype)) || (st = check_scores(experts, top_k, scores, scale)) ||
      (st = check_picks(tokens, top_k)))
    return st;
  const uint64_t E = (uint64_t)experts, k = (uint64_t)top_k, es = size_of(dtype);
  const bool in_place = same(base, base_stride, grad_logits, grad_stride);
  Buffers b(h);
  if ((st = b.add(&logits, false, tokens, E, stride, es)) || (st = b.add(&ids, false, tokens, k, k, 4)) ||
      (st = b.add(&sums, false, 1, 2 * E + 1, 2 * E + 1, 4)) ||
      (grad_loss && (st = b.add(&grad_loss, false, 1, 1, 1, 4))) ||
      (base && !in_place && (st = b.add(&base, false, tokens, E, base_stride, es))) ||
      (st = b.add(&grad_logits, true, tokens, E, grad_stride, es)) || (st = b.apart()))
    return st;
  if (tokens == 0) return PL_OK;
  pl::BalanceArgs a = {};
  a.logits = logits;
  a.ld = stride;
  a.tokens = tokens;
  a.experts = experts;
  a.top_k = top_k;
  a.sigmoid = scores == PL_SCORES_SIGMOID;
  a.scale = scale;
  a.ids = ids;
  a.sums = const_cast<float*>(sums);
  a.grad_loss = grad_loss;
  a.base = in_place ? grad_logits : base;
  a.ldb = base_stride;
  a.grad_logits = grad_logits;
  a.ldg = grad_stride;
  return pl::launch_balance_grad(a, dtype, (cudaStream_t)stream);
}

purlin_status purlin_distil_loss(purlin_handle handle, const void* logits, size_t stride, purlin_dtype dtype,
                                 size_t tokens, const purlin_distillation* d, const void* ids, const void* teacher,
                                 float* loss, float* stats, purlin_stream_t stream) {
  pl::OpHandle h;
  pl::DistilArgs a;
  purlin_status st;
  if ((st = pl::op_begin(handle, &h)) || (st = check_dtype(dtype)) || (st = distil_args(d, tokens, &a))) return st;
  if (d->first != 0 || (uint64_t)d->vocabulary != d->width) return PL_ERR_INVALID_ARG;  // purlin_distil_parts
  const uint64_t k = (uint64_t)d->picks;
  Buffers b(h);
  if ((st = b.add(&logits, false, tokens, d->width, stride, size_of(dtype))) ||
      (st = b.add(&ids, false, tokens, k, k, d->id_bytes)) ||
      (st = b.add(&teacher, false, tokens, k, k, size_of(d->teacher_dtype))) ||
      (st = b.add(&loss, true, 1, tokens, tokens, 4)) || (st = b.add(&stats, true, tokens, 2, 2, 4)) || (st = b.apart()))
    return st;
  if (tokens == 0) return PL_OK;
  a.logits = logits;
  a.ld = stride;
  a.ids = ids;
  a.teacher = teacher;
  a.loss = loss;
  a.stats = stats;
  return pl::launch_distil(a, dtype, (cudaStream_t)stream);
}

purlin_status purlin_distil_parts(purlin_handle handle, const void* logits, size_t stride, purlin_dtype dtype,
                                  size_t tokens, const purlin_distillation* d, const void* ids, const void* teacher,
                                  float* parts, purlin_stream_t stream) {
  pl::OpHandle h;
  pl::DistilArgs a;
  purlin_status st;
  if ((st = pl::op_begin(handle, &h)) || (st = check_dtype(dtype)) || (st = distil_args(d, tokens, &a))) return st;
  const uint64_t k = (uint64_t)d->picks;
  Buffers b(h);
  if ((st = b.add(&logits, false, tokens, d->width, stride, size_of(dtype))) ||
      (st = b.add(&ids, false, tokens, k, k, d->id_bytes)) ||
      (st = b.add(&teacher, false, tokens, k, k, size_of(d->teacher_dtype))) ||
      (st = b.add(&parts, true, tokens, 4, 4, 4)) || (st = b.apart()))
    return st;
  if ((uintptr_t)parts & 7u) return PL_ERR_ALIGNMENT;
  if (tokens == 0) return PL_OK;
  a.logits = logits;
  a.ld = stride;
  a.ids = ids;
  a.teacher = teacher;
  a.parts = parts;
  return pl::launch_distil(a, dtype, (cudaStream_t)stream);
}

purlin_status purlin_distil_join(purlin_handle handle, const float* parts, int ranges, size_t tokens, float temperature,
                                 float scale, float* loss, float* stats, purlin_stream_t stream) {
  pl::OpHandle h;
  pl::DistilArgs a;
  purlin_status st;
  const purlin_distillation d = {0, 0, 0, 1, 8, PL_F32, temperature, scale};
  if ((st = pl::op_begin(handle, &h)) || (st = distil_args(&d, tokens, &a))) return st;
  if (ranges < 1 || (uint64_t)ranges > UINT64_MAX / 16 / std::max<uint64_t>(1, tokens)) return PL_ERR_INVALID_ARG;
  Buffers b(h);
  if ((st = b.add(&parts, false, (uint64_t)ranges * tokens, 4, 4, 4)) || (st = b.add(&loss, true, 1, tokens, tokens, 4)) ||
      (st = b.add(&stats, true, tokens, 2, 2, 4)) || (st = b.apart()))
    return st;
  if (tokens == 0) return PL_OK;
  a.parts = const_cast<float*>(parts);
  a.ranks = ranges;
  a.loss = loss;
  a.stats = stats;
  return pl::launch_distil_join(a, (cudaStream_t)stream);
}

purlin_status purlin_distil_loss_grad(purlin_handle handle, const void* logits, size_t stride, purlin_dtype dtype,
                                      size_t tokens, const purlin_distillation* d, const void* ids, const void* teacher,
                                      const float* stats, const float* grad_loss, void* grad_logits, size_t grad_stride,
                                      purlin_stream_t stream) {
  pl::OpHandle h;
  pl::DistilArgs a;
  purlin_status st;
  if ((st = pl::op_begin(handle, &h)) || (st = check_dtype(dtype)) || (st = distil_args(d, tokens, &a))) return st;
  const uint64_t k = (uint64_t)d->picks, es = size_of(dtype);
  const bool in_place = same(logits, stride, grad_logits, grad_stride);
  Buffers b(h);
  if ((!in_place && (st = b.add(&logits, false, tokens, d->width, stride, es))) ||
      (st = b.add(&ids, false, tokens, k, k, d->id_bytes)) ||
      (st = b.add(&teacher, false, tokens, k, k, size_of(d->teacher_dtype))) ||
      (st = b.add(&stats, false, tokens, 2, 2, 4)) || (st = b.add(&grad_loss, false, 1, tokens, tokens, 4)) ||
      (st = b.add(&grad_logits, true, tokens, d->width, grad_stride, es)) || (st = b.apart()))
    return st;
  if (tokens == 0 || d->width == 0) return PL_OK;
  a.logits = in_place ? grad_logits : logits;
  a.ld = stride;
  a.ids = ids;
  a.teacher = teacher;
  a.stats = const_cast<float*>(stats);
  a.grad_loss = grad_loss;
  a.grad_logits = grad_logits;
  a.ldg = grad_stride;
  return pl::launch_distil_grad(a, dtype, (cudaStream_t)stream);
}

}  // extern "C"
