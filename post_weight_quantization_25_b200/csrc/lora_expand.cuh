// What the kernels of the projection back from the rank share.
#pragma once
#include "lora_mma.cuh"

namespace gptq {

struct ExpandArgs {
  LoraArgs a;
  const float* u;
  int64_t ldu;
  const void* W;
  int64_t stride_w;
  int64_t ldw;  // between columns of Y (ranks inner) or between ranks (columns inner)
  int scaled;
  int tile;     // tokens per piece
  int strips;   // CTAs side by side in the columns
  int turns;    // column strips a CTA takes one after the other
  int vec_u, vec_w, vec_y;
  void* Y;
  int64_t ldy;
  int64_t C;    // columns of Y
};

// bf16 W with 16-byte aligned rows, Y with 16-byte aligned rows, max_rank at
// most kExpandTcRank.
constexpr int kExpandTcRank = 64;
cudaError_t launch_lora_expand_tc(const ExpandArgs& p, bool columns_inner, int y_bf16,
                                  cudaStream_t s);

namespace {

template <class T, int E>
__device__ __forceinline__ void add_row(float (&v)[E], const Raw<T, E>& y) {
#pragma unroll
  for (int i = 0; i < E; ++i) {
    if constexpr (sizeof(T) == 2)
      v[i] += __uint_as_float((i & 1) ? y.w[i / 2] & 0xffff0000u : y.w[i / 2] << 16);
    else
      v[i] += y.w[i];
  }
}
template <class T, int E>
__device__ __forceinline__ Raw<T, E> round_row(const float (&v)[E]) {
  Raw<T, E> o;
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      memcpy(o.w + i, &h, 4);
    }
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i) o.w[i] = v[i];
  }
  return o;
}

}  // namespace
}  // namespace gptq
