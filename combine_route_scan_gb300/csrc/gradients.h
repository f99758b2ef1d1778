// Parameters and launchers of the gradients of combine and dispatch.
#pragma once
#include "internal.h"

namespace crs {

// Dispatch's gradient: the combine's reduce with expert_out the rows' gradients, x_out
// the tokens', no scales and no x.
struct DispatchGradParams : CombineParams {
  const void* residual;      // [W*bs][h] that the sums start from, or null
  const float* row_weights;  // [W*A] gradients of expand_scales, or null
  float* pick_weights;       // [W*bs*K] where they go
};

// Combine's gradient: of CombineParams' arrays it reads x, expert_out, scales and the
// routing's, and writes these.
struct CombineGradParams : CombineParams {
  const void* grad_out;     // [W*bs][h]
  void* grad_rows;          // [W*A][h], or null
  float* grad_scales;       // [W*bs*K], or null
  void* grad_x;             // [W*bs][h], or null
};

// The gradients; search: by looking for each pick's row, where the workspace has no row map of these buffers.
cudaError_t launch_dispatch_grad(const DispatchGradParams& p, bool search, cudaStream_t st, int num_sms);
cudaError_t launch_dispatch_grad_reduce(const DispatchGradParams& p, cudaStream_t st, int num_sms);
cudaError_t launch_combine_grad(const CombineGradParams& p, bool search, cudaStream_t st, int num_sms);

}  // namespace crs
