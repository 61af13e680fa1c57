// What the low-rank adapter kernels share: the adapters' layout on the device
// and the search for a task's slot in the token plan.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

#include "gptq_internal.cuh"

namespace gptq {

// gptq_lora with the element types out of the way (see include/gptq.h).
struct LoraArgs {
  const void* A;
  const void* B;
  int wt_bf16;
  int n_slots, max_rank;
  int64_t n, rows, lda, stride_a, ldb, stride_b;
  const int32_t* ranks;
  const float* scales;
  const int32_t* order;
  const int32_t* slot_start;
  int64_t ntok;
};

__device__ __forceinline__ int lora_rank(const LoraArgs& p, int slot) {
  const int r = p.ranks ? p.ranks[slot] : p.max_rank;
  return min(max(r, 0), p.max_rank);
}
__device__ __forceinline__ float lora_scale(const LoraArgs& p, int slot) {
  return p.scales ? p.scales[slot] : 1.f;
}
// first position of slot a's tokens in `order`, clamped to [0, ntok]
__device__ __forceinline__ int lora_start(const LoraArgs& p, int a) {
  return (int)min((int64_t)max(p.slot_start[a], 0), p.ntok);
}

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

}  // namespace gptq
