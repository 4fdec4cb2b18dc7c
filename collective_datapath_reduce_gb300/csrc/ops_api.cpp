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
  static constexpr int kMost = 8;
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

}  // extern "C"
