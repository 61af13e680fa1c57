// Activations in 8 bits with one scale per row or per group of columns.
#include <cuda_runtime.h>

#include "lora_internal.cuh"

namespace gptq {
namespace {

// One warp per (row, group).
template <class TX>
__global__ void act8_quantize_simple(const TX* __restrict__ x, int64_t rows, int64_t n,
                                     int64_t ldx, int64_t group, int64_t G,
                                     int8_t* __restrict__ codes, int64_t ldc,
                                     float* __restrict__ scales) {
  const int64_t w = ((int64_t)blockIdx.x * blockDim.x + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (w >= rows * G) return;
  const int64_t r = w / G, g = w % G;
  const int64_t c0 = g * group, c1 = min(c0 + group, n);
  const TX* xr = x + r * ldx;
  float m = 0.f;
  bool bad = false;
  for (int64_t c = c0 + lane; c < c1; c += 32) {
    const float v = fabsf(to_f32(xr[c]));
    bad |= !(v <= 3.402823466e38f);
    m = fmaxf(m, v);
  }
  for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
  bad = __any_sync(~0u, bad);
  const float sc = bad ? __int_as_float(0x7fffffff) : fmaxf(__fdiv_rn(m, 127.f), 0x1p-126f);
  if (lane == 0) scales[w] = sc;
  for (int64_t c = c0 + lane; c < c1; c += 32) {
    const float q = bad ? 0.f : (float)rint((double)to_f32(xr[c]) / (double)sc);
    codes[r * ldc + c] = (int8_t)min(max((int)q, -127), 127);
  }
}

template <class TO>
__global__ void act8_dequant_simple(const int8_t* __restrict__ codes, int64_t n, int64_t ldc,
                                    const float* __restrict__ scales, int64_t group, int64_t G,
                                    TO* __restrict__ out, int64_t ldo) {
  const int64_t r = blockIdx.x;
  for (int64_t c = (int64_t)blockIdx.y * blockDim.x + threadIdx.x; c < n;
       c += (int64_t)gridDim.y * blockDim.x)
    out[r * ldo + c] = from_f32<TO>(scales[r * G + c / group] * (float)codes[r * ldc + c]);
}

}  // namespace

cudaError_t launch_quantize_act8(const void* x, int x_bf16, int64_t rows, int64_t n, int64_t ldx,
                                 int group, int8_t* codes, int64_t ldc, float* scales,
                                 cudaStream_t s) {
  const int64_t gs = group > 0 ? group : n, G = (n + gs - 1) / gs;
  const unsigned blocks = (unsigned)((rows * G + 7) / 8);
  if (x_bf16)
    act8_quantize_simple<<<blocks, 256, 0, s>>>(static_cast<const __nv_bfloat16*>(x), rows, n, ldx,
                                                gs, G, codes, ldc, scales);
  else
    act8_quantize_simple<<<blocks, 256, 0, s>>>(static_cast<const float*>(x), rows, n, ldx, gs, G,
                                                codes, ldc, scales);
  note_launch();
  return cudaGetLastError();
}

cudaError_t launch_dequant_act8(const int8_t* codes, int64_t rows, int64_t n, int64_t ldc,
                                const float* scales, int group, void* out, int out_bf16,
                                int64_t ldo, cudaStream_t s) {
  const int64_t gs = group > 0 ? group : n, G = (n + gs - 1) / gs;
  dim3 grid((unsigned)rows, (unsigned)min((int64_t)16, (n + 255) / 256));
  if (out_bf16)
    act8_dequant_simple<<<grid, 256, 0, s>>>(codes, n, ldc, scales, gs, G,
                                             static_cast<__nv_bfloat16*>(out), ldo);
  else
    act8_dequant_simple<<<grid, 256, 0, s>>>(codes, n, ldc, scales, gs, G,
                                             static_cast<float*>(out), ldo);
  note_launch();
  return cudaGetLastError();
}

}  // namespace gptq
