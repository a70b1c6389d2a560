// Internal launch interface of the operators at the expert block's edge: expert routing, the
// norm and 8-bit activation checkpoints; not part of the public C ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/mxfp4_moe.h"

namespace moe {

cudaError_t launch_route(const mxfp4_moe_routing& r, const float* logits, const float* bias,
                         int32_t* idx, float* w, int32_t* counts, int sms, cudaStream_t st);
cudaError_t launch_route_backward(const mxfp4_moe_routing& r, const float* logits,
                                  const int32_t* idx, const float* w, const float* d_w,
                                  float* d_logits, cudaStream_t st);
// A caller's routing into the workspace (idx, w in slot order) with the expert histograms of
// its 32-token segments in `scratch`, as launch_router_topk leaves them; an index outside
// [0, E) is recorded in err (tag 0x120) and becomes expert 0 with weight 0.
cudaError_t launch_import_routing(const int32_t* topk_idx, const float* topk_w, int T, int E,
                                  int k, int32_t* idx, float* w, int32_t* scratch, int* err,
                                  cudaStream_t st);

// Rows or a checkpoint in (x, or codes / scales), everything a norm pass may write out.
struct NormArgs {
  int T, H;
  bool rms, rows_f32, param_f32;
  float eps;
  const void* x;                 // rows, or null: `from`
  mxfp4_moe_checkpoint from, to; // codes null: none
  const void* y;
  const void* weight;
  const void* bias;
  void* x_out;
  void* out;
  float* mean;
  float* rstd;
};
struct NormGradArgs {
  int T, H;
  bool rms, rows_f32, param_f32;
  const void* d_out;
  const void* x;
  mxfp4_moe_checkpoint from;
  const float* mean;
  const float* rstd;
  const void* weight;
  const void* g;
  void* dx;
  float* d_weight;
  float* d_bias;
  float* partial;                // scratch
};
cudaError_t launch_norm_forward(const NormArgs& a, int sms, cudaStream_t st);
size_t norm_scratch_bytes(int T, int H);
cudaError_t launch_norm_backward(const NormGradArgs& a, int sms, cudaStream_t st);
cudaError_t launch_checkpoint_pack(int T, int H, bool rows_f32, const void* x,
                                   const mxfp4_moe_checkpoint& to, cudaStream_t st);
cudaError_t launch_checkpoint_unpack(int T, int H, bool rows_f32,
                                     const mxfp4_moe_checkpoint& from, void* x, cudaStream_t st);

}  // namespace moe
