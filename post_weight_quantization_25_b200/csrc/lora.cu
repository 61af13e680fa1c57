// Low-rank adapters beside a frozen projection: the token plan, the forward
// product y += s (x A^T) B^T and its gradients.
#include <cuda_runtime.h>

#include "lora_internal.cuh"

namespace gptq {
namespace {

constexpr int kPlanThreads = 1024;

// One CTA per slot (the last one: tokens without a slot).  Each warp has a
// stretch of the ids and reads it twice: first to count its tokens of lower
// slots (the slot's base in `order`) and of the slot, then, the stretches'
// counts added up, to write its tokens in ascending order by warp ballots.  No
// atomics, so the order is the same every time.
__global__ void __launch_bounds__(kPlanThreads)
    lora_plan_kernel(const int32_t* __restrict__ ids, int ntok, int n_slots,
                     int32_t* __restrict__ order, int32_t* __restrict__ slot_start,
                     int32_t* __restrict__ info) {
  constexpr int kWarps = kPlanThreads / 32;
  const int a = blockIdx.x;  // n_slots: none
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ int s_below[kWarps], s_mine[kWarps];
  const int each = ((ntok + kWarps - 1) / kWarps + 31) / 32 * 32;
  const int begin = min(warp * each, ntok), end = min(begin + each, ntok);
  int below = 0, mine = 0;
  bool bad = false;
#pragma unroll 4
  for (int i = begin + lane; i < end; i += 32) {
    const int id = ids[i];
    const bool real = id >= 0 && id < n_slots;
    bad |= id >= n_slots;
    below += real && id < a;
    mine += real ? id == a : a == n_slots;
  }
  below = __reduce_add_sync(~0u, below);
  mine = __reduce_add_sync(~0u, mine);
  if (lane == 0) {
    s_below[warp] = below;
    s_mine[warp] = mine;
  }
  bad = __syncthreads_or(bad);
  int before = lane < warp ? s_mine[lane] : 0;
  before = __reduce_add_sync(~0u, before);
  const int base = __reduce_add_sync(~0u, s_below[lane]);
  if (threadIdx.x == 0) {
    slot_start[a] = base;
    if (a == 0 && info) *info = bad ? GPTQ_ERR_INVALID_ARG : 0;
  }
  if (mine == 0) return;
  int at = base + before;
#pragma unroll 4
  for (int i0 = begin; i0 < end; i0 += 32) {
    const int i = i0 + lane;
    const int id = i < end ? ids[i] : 0;
    const bool is = i < end && ((id >= 0 && id < n_slots) ? id == a : a == n_slots);
    const unsigned m = __ballot_sync(~0u, is);
    if (is) order[at + __popc(m & ((1u << lane) - 1))] = i;
    at += __popc(m);
  }
}

}  // namespace

cudaError_t launch_lora_plan(const int32_t* ids, int64_t ntok, int64_t n_slots, int32_t* order,
                             int32_t* slot_start, int32_t* info, cudaStream_t s) {
  lora_plan_kernel<<<(unsigned)n_slots + 1, kPlanThreads, 0, s>>>(ids, (int)ntok, (int)n_slots,
                                                                  order, slot_start, info);
  note_launch();
  return cudaGetLastError();
}

// A row of u or v in the workspace: fp32, a multiple of 16 bytes.
static int64_t factor_ld(const LoraArgs& a) { return (a.max_rank + 3) / 4 * 4; }
static size_t factor_bytes(const LoraArgs& a) {
  return ((size_t)a.ntok * factor_ld(a) * sizeof(float) + 255) / 256 * 256;
}

// [u or v | backward: partial sums of the gradients]; few tokens keep u to
// themselves
size_t lora_workspace_bytes(const LoraArgs& a, bool backward) {
  return (backward || !lora_few(a) ? factor_bytes(a) : 0) + (backward ? lora_grad_workspace_bytes(a) : 0);
}

cudaError_t launch_lora_apply(const LoraArgs& a, const void* x, int x_bf16, int64_t ldx, void* y,
                              int y_bf16, int64_t ldy, float* u, int64_t ldu, void* ws,
                              cudaStream_t s) {
  if (lora_few(a))
    return launch_lora_few(a, true, x, x_bf16, ldx, u, ldu, y, y_bf16, ldy, s);
  if (!u) {
    u = static_cast<float*>(ws);
    ldu = factor_ld(a);
  }
  const cudaError_t e = launch_lora_shrink(a, true, x, x_bf16, ldx, u, ldu, s);
  if (e != cudaSuccess) return e;
  return launch_lora_expand(a, true, u, ldu, y, y_bf16, ldy, s);
}

cudaError_t launch_lora_backward(const LoraArgs& a, const void* dy, int dy_bf16, int64_t lddy,
                                 const void* x, int x_bf16, int64_t ldx, const int8_t* codes,
                                 const float* code_scales, int code_group, const float* u,
                                 int64_t ldu, void* dx, int dx_bf16, int64_t lddx, float* dA,
                                 float* dB, void* ws, cudaStream_t s) {
  float* v = static_cast<float*>(ws);
  const int64_t ldv = factor_ld(a);
  cudaError_t e = cudaSuccess;
  const bool few = lora_few(a);
  if (few && (dx || dA))
    e = launch_lora_few(a, false, dy, dy_bf16, lddy, dA ? v : nullptr, ldv, dx, dx_bf16, lddx, s);
  else if (dx || dA)
    e = launch_lora_shrink(a, false, dy, dy_bf16, lddy, v, ldv, s);
  if (e == cudaSuccess && (dA || dB)) {
    const GradArgs g = {v, ldv, codes ? static_cast<const void*>(codes) : x,
                        codes ? 2 : x_bf16 ? 0 : 1, ldx, code_scales, code_group, dA,
                        u, ldu, dy, dy_bf16, lddy, dB, dx || dA};
    e = launch_lora_grad(a, g, static_cast<char*>(ws) + factor_bytes(a), s);
  }
  if (e == cudaSuccess && dx && !few)
    e = launch_lora_expand(a, false, v, ldv, dx, dx_bf16, lddx, s);
  return e;
}

}  // namespace gptq
