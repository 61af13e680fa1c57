// What the two kernels of the projection down to the rank share.
#pragma once
#include "lora_mma.cuh"

namespace gptq {

struct ShrinkArgs {
  LoraArgs a;
  const void* X;
  int64_t ldx;
  int64_t K;
  const void* W;
  int64_t stride_w;  // between slots
  int64_t ldw;       // between ranks (ranks outer) or between k (ranks inner)
  int scaled;
  int vec_x, vec_w;
  float* out;
  int64_t ldo;
  int vec_o;         // out's rows are 16-byte aligned
};

// bf16 X and W with 16-byte aligned rows
cudaError_t launch_lora_shrink_tc(const ShrinkArgs& p, bool ranks_inner, cudaStream_t s);

}  // namespace gptq
