// The index-driven operators around the collectives: arguments of their
// kernels and the host functions that launch them.  ops_api.cpp checks the
// callers' arguments and fills these; each launch function picks a kernel
// variant, launches it on the stream and returns the launch's status.
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "purlin_gb.h"

namespace pl {

// What an operator needs of the handle it is called on.
struct OpHandle {
  int device = 0;
  int sm_count = 0;
  uint32_t* status = nullptr;  // the operators' device status word
};

// The handle is live and its device is current (api.cpp).
purlin_status op_begin(purlin_handle h, OpHandle* out);
// Where a caller's pointer lives, and the address the kernels use (api.cpp).
purlin_status op_locate(const OpHandle& h, const void* p, const void** dev_p, bool* host);

struct RouteArgs {
  const void* logits;
  uint64_t ld;        // elements from one token's logits to the next's
  const float* bias;  // or nullptr
  uint64_t tokens;
  int experts, top_k;
  int sigmoid;
  int groups, kept, best;
  int group_size, group_shift;  // set by launch_route
  int renormalise;
  float scale;
  int32_t* ids;
  float* weights;
  // gradient only (ids are then read)
  const float* grad_weights;
  void* grad_logits;
  uint64_t grad_ld;
};
purlin_status launch_route(const RouteArgs& a, int dtype, cudaStream_t s);
purlin_status launch_route_grad(const RouteArgs& a, int dtype, cudaStream_t s);

struct PlanArgs {
  const int32_t* ids;
  uint64_t slots;
  int experts;
  int32_t* offsets;
  int32_t* places;
  uint32_t* counts;  // workspace: one row of `experts` counts per CTA
};
size_t expert_plan_bytes(uint64_t slots, int experts);
purlin_status launch_expert_plan(const PlanArgs& a, cudaStream_t s);

struct RowsArgs {
  const void* x;      // dispatch: token rows; combine: expert rows
  uint64_t ldx;
  void* y;            // dispatch: expert rows; combine: token rows
  uint64_t ldy;
  const int32_t* places;
  const float* weights;  // combine: or nullptr
  uint64_t tokens;
  uint64_t width;
  int top_k;
  uint32_t* status;
  bool host;          // some rows are host memory
  // gradient of combine: x = expert rows, y = gradient of the expert rows
  const void* grad_y;
  uint64_t ldg;
  float* grad_weights;
};
purlin_status launch_dispatch(const RowsArgs& a, int dtype, cudaStream_t s);
purlin_status launch_combine(const RowsArgs& a, int dtype, cudaStream_t s);
purlin_status launch_combine_grad(const RowsArgs& a, int dtype, cudaStream_t s);

struct EmbedArgs {
  const void* tokens;  // int32 or int64
  int wide_tokens;
  int64_t first;
  uint64_t rows;       // of the table (this rank's range)
  uint64_t n;          // tokens
  uint64_t width;
  float scale;
  const void* x;       // forward: the table; gradient: the output's gradient
  uint64_t ldx;
  void* y;             // forward: the output; gradient: the table's gradient
  uint64_t ldy;
  const void* base;    // gradient: added to, or nullptr
  uint64_t ldb;
  void* workspace;
};
size_t embed_grad_bytes(uint64_t tokens, uint64_t rows, uint64_t width);
purlin_status launch_embed(const EmbedArgs& a, int dtype, cudaStream_t s);
purlin_status launch_embed_grad(const EmbedArgs& a, int x_dtype, int y_dtype, cudaStream_t s);

struct ClipTensor {
  const void* in;
  void* out;
  uint64_t n;
};
size_t clip_bytes();
purlin_status launch_clip(const ClipTensor* t, size_t n, int dtype, float scale, float max_norm, bool write, float* norm,
                          double* partials, int sm_count, cudaStream_t s);

}  // namespace pl
