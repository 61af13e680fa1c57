// What the low-rank adapter kernels share: the adapters' layout on the device
// and the search for a task's slot in the token plan.
#pragma once
#include <atomic>
#include <cstdint>
#include <cstring>
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

// Host: whether every row of a matrix (element size esz, row stride ld, slot
// stride `stride`, in elements) starts on a multiple of `bytes`.
inline int rows_aligned(const void* p, int64_t ld, int64_t stride, int esz, int bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && (ld * esz) % bytes == 0 &&
         (stride * esz) % bytes == 0;
}
// Host: whether a tensor map can hold an adapter matrix: rows on multiples of 16
// bytes, and slots a multiple of the row stride apart, as each stride of a map
// has to be of the one before.
inline int slots_mappable(const void* p, int64_t ld, int64_t stride, int64_t n_slots) {
  return rows_aligned(p, ld, n_slots > 1 ? stride : 0, 2, 16) &&
         (n_slots == 1 || stride % ld == 0);
}
// Host: raises a kernel's limits (dynamic shared memory; clusters of more than
// 8) the first time it is launched on a device.  `done` is the launch
// function's own record, one bit a device: setting the limits costs as much
// host time as a third of the launch.
inline cudaError_t raise_limits(const void* kernel, size_t smem, bool large_clusters,
                                std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess && large_clusters)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

// Host: few tokens, or few to a slot: both projections in one launch
// (lora_few.cu) instead of one each for many.  The one launch reads the
// adapters again for every 16 tokens and costs time with tokens x rank x
// columns, twice that above rank 16; the two cost two latencies, and tiles of
// 128 tokens that several slots leave half empty.  Device times of both (us, one
// / two launches, bf16): 4096 x 4096, rank 16, one slot: 256 tokens 9 / 12, 1024
// 11 / 14, 2048 17 / 18, 4096 32 / 24; eight slots: 1024 12 / 22, 2048 18 / 28,
// 4096 33 / 33; rank 64: one slot 128 tokens 14 / 14, 512 17 / 16, 1024 24 / 19;
// 32 slots 512 tokens 24 / 52, 1024 40 / 41.  11008 x 4096, rank 16, eight slots:
// 2048 tokens 25 / 37, 4096 61 / 47.  Whole calls with cold caches (about 8 us
// more): 28672 x 8192, rank 16: 128 tokens 18 / 38, 256 24 / 38, 512 29 / 42, 1024
// 47 / 48; 4096 x 4096, rank 128: 64 tokens 25 / 32, 256 35 / 33, 1024 56 / 52; rank
// 256: 32 tokens 43 / 34, 64 43 / 45, 256 59 / 46; fp32 at rank 16: 1024 tokens
// 25 / 40, 2048 40 / 60, 4096 69 / 89 (here one launch would pay for longer than
// the rule lets it); 256 slots of which one is used: 1024 tokens 33 / 212, 4096
// 51 / 126, 8000 92 / 101 (both look tokens up among all slots, and two launches
// have a piece for each).
inline bool lora_few(const LoraArgs& a) {
  const int64_t used = a.n_slots < a.ntok ? a.n_slots : a.ntok;
  const int64_t r = (a.max_rank + 15) / 16 * 16;
  const int64_t work = a.ntok * r * (a.n + a.rows) * (r > 16 ? 2 : 1);
  return a.ntok < 32 * used || work < (int64_t)(used > 1 ? 2 : 1) << 28;
}

// out[t] (may be null) and Y[t] (may be null) of both projections: forward
// out = X[t] A^T, Y[t] += scale out B^T; else out = scale X[t] B,
// Y[t] += out A.
cudaError_t launch_lora_few(const LoraArgs& a, bool forward, const void* X, int x_bf16,
                            int64_t ldx, float* out, int64_t ldo, void* Y, int y_bf16,
                            int64_t ldy, cudaStream_t s);

// out[t] (ntok x max_rank fp32) = X[t] A^T (forward) or scale X[t] B
cudaError_t launch_lora_shrink(const LoraArgs& a, bool forward, const void* X, int x_bf16,
                               int64_t ldx, float* out, int64_t ldo, cudaStream_t s);
// Y[t] += scale u[t] B^T (forward) or u[t] A.  Enqueued right behind a kernel
// of this library that writes u (see dep_wait in lora_mma.cuh).
cudaError_t launch_lora_expand(const LoraArgs& a, bool forward, const float* u, int64_t ldu,
                               void* Y, int y_bf16, int64_t ldy, cudaStream_t s);

// dA = sum v^T x and dB = scale sum dy^T u over each slot's tokens (either
// may be absent: null).
struct GradArgs {
  const float* v;
  int64_t ldv;
  const void* x;             // x or codes
  int x_kind;                // 0: bf16, 1: fp32, 2: 8-bit codes
  int64_t ldx;
  const float* code_scales;
  int code_group;
  float* dA;
  const float* u;
  int64_t ldu;
  const void* dy;
  int dy_bf16;
  int64_t lddy;
  float* dB;
  bool behind;               // enqueued right behind a kernel of the same call
};
size_t lora_grad_workspace_bytes(const LoraArgs& a);
cudaError_t launch_lora_grad(const LoraArgs& a, const GradArgs& g, void* ws, cudaStream_t s);

}  // namespace gptq
