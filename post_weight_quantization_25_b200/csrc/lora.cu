// Low-rank adapters beside a frozen projection: the token plan, the forward
// product y += s (x A^T) B^T and its gradients.
#include <cuda_runtime.h>

#include "lora_internal.cuh"

namespace gptq {
namespace {

constexpr int kPlanThreads = 1024;

// One CTA per slot (the last one: tokens without a slot).  Each CTA reads
// every id twice: first to count the ids of lower slots (its base in
// `order`), then to compact its own tokens in ascending order with warp
// ballots.  No atomics, so the order is the same every time.
__global__ void __launch_bounds__(kPlanThreads)
    lora_plan_kernel(const int32_t* __restrict__ ids, int ntok, int n_slots,
                     int32_t* __restrict__ order, int32_t* __restrict__ slot_start,
                     int32_t* __restrict__ info) {
  const int a = blockIdx.x;  // n_slots: none
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __shared__ int s_warp[kPlanThreads / 32];
  __shared__ int s_bad;
  if (tid == 0) s_bad = 0;
  __syncthreads();
  int below = 0;
  bool bad = false;
  for (int i = tid; i < ntok; i += kPlanThreads) {
    const int id = ids[i];
    bad |= id >= n_slots;
    below += (id >= 0 && id < n_slots && id < a) ? 1 : 0;
  }
  if (bad) s_bad = 1;
  for (int o = 16; o; o >>= 1) below += __shfl_xor_sync(~0u, below, o);
  if (lane == 0) s_warp[warp] = below;
  __syncthreads();
  int base = 0;
  for (int w = 0; w < kPlanThreads / 32; ++w) base += s_warp[w];
  if (tid == 0) {
    slot_start[a] = base;
    if (a == 0 && info) *info = s_bad ? GPTQ_ERR_INVALID_ARG : 0;
  }
  for (int i0 = 0; i0 < ntok; i0 += kPlanThreads) {
    const int i = i0 + tid;
    bool mine = false;
    if (i < ntok) {
      const int id = ids[i];
      mine = (id >= 0 && id < n_slots) ? id == a : a == n_slots;
    }
    const unsigned m = __ballot_sync(~0u, mine);
    __syncthreads();  // s_warp of the previous round has been read
    if (lane == 0) s_warp[warp] = __popc(m);
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w < kPlanThreads / 32; ++w) {
      const int c = s_warp[w];
      before += w < warp ? c : 0;
      total += c;
    }
    if (mine) order[base + before + __popc(m & ((1u << lane) - 1))] = i;
    base += total;
  }
}

// The slot whose range holds position p, or -1 (positions past the last
// slot's range belong to tokens without an adapter).
__device__ __forceinline__ int slot_of(const LoraArgs& a, int p) {
  if (p < lora_start(a, 0) || p >= lora_start(a, a.n_slots)) return -1;
  int lo = 0, hi = a.n_slots;  // start[lo] <= p < start[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (lora_start(a, mid) <= p) lo = mid; else hi = mid;
  }
  return lo;
}

// out[t][i] = scale * sum_k X[t][k] W(i, k): one warp per position and rank.
template <class TX, class TW>
__global__ void lora_shrink_simple(LoraArgs a, const TX* __restrict__ X, int64_t ldx, int64_t K,
                                   const TW* __restrict__ W, int64_t stride_w, int64_t ld_rank,
                                   int64_t ld_k, int scaled, float* __restrict__ out,
                                   int64_t ldo) {
  const int p = blockIdx.x, i = blockIdx.y * blockDim.y + threadIdx.y;
  const int s = slot_of(a, p);
  if (s < 0 || i >= a.max_rank) return;
  const int t = a.order[p];
  if (t < 0 || t >= a.ntok) return;
  float acc = 0.f;
  if (i < lora_rank(a, s)) {
    const TX* x = X + (int64_t)t * ldx;
    const TW* w = W + s * stride_w + i * ld_rank;
    for (int64_t k = threadIdx.x; k < K; k += 32) acc = fmaf(to_f32(x[k]), to_f32(w[k * ld_k]), acc);
    for (int o = 16; o; o >>= 1) acc += __shfl_xor_sync(~0u, acc, o);
    if (scaled) acc *= lora_scale(a, s);
  }
  if (threadIdx.x == 0) out[(int64_t)t * ldo + i] = acc;
}

// Y[t][c] += scale * sum_i u[t][i] W(i, c)
template <class TW, class TY>
__global__ void lora_expand_simple(LoraArgs a, const float* __restrict__ u, int64_t ldu,
                                   const TW* __restrict__ W, int64_t stride_w, int64_t ld_rank,
                                   int64_t ld_c, int scaled, TY* __restrict__ Y, int64_t ldy,
                                   int64_t C) {
  const int p = blockIdx.x;
  const int64_t c = (int64_t)blockIdx.y * blockDim.x + threadIdx.x;
  const int s = slot_of(a, p);
  if (s < 0 || c >= C) return;
  const int t = a.order[p];
  if (t < 0 || t >= a.ntok) return;
  const float sc = scaled ? lora_scale(a, s) : 1.f;
  const int r = lora_rank(a, s);
  float acc = 0.f;
  for (int i = 0; i < r; ++i)
    acc = fmaf(u[(int64_t)t * ldu + i] * sc, to_f32(W[s * stride_w + i * ld_rank + c * ld_c]), acc);
  TY* y = Y + (int64_t)t * ldy + c;
  *y = from_f32<TY>(to_f32(*y) + acc);
}

// out(slot, i, c) = sum over the slot's tokens of scale v[t][i] X[t][c]
template <class TX>
__global__ void lora_grad_simple(LoraArgs a, const float* __restrict__ v, int64_t ldv, int scaled,
                                 const TX* __restrict__ X, int64_t ldx,
                                 const float* __restrict__ xs, int group, int64_t C,
                                 float* __restrict__ out, int64_t ld_rank, int64_t ld_c) {
  const int s = blockIdx.z, i = blockIdx.y;
  const int64_t c = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (c >= C) return;
  float acc = 0.f;
  if (i < lora_rank(a, s)) {
    const float sc = scaled ? lora_scale(a, s) : 1.f;
    const int64_t G = group > 0 ? (C + group - 1) / group : 1;
    const int64_t g = group > 0 ? c / group : 0;
    const int p1 = lora_start(a, s + 1);
    for (int p = lora_start(a, s); p < p1; ++p) {
      const int t = a.order[p];
      if (t < 0 || t >= a.ntok) continue;
      float x = (float)X[(int64_t)t * ldx + c];
      if (xs) x *= xs[t * G + g];
      acc = fmaf(v[(int64_t)t * ldv + i] * sc, x, acc);
    }
  }
  out[(int64_t)s * a.max_rank * C + i * ld_rank + c * ld_c] = acc;
}

}  // namespace

cudaError_t launch_lora_plan(const int32_t* ids, int64_t ntok, int64_t n_slots, int32_t* order,
                             int32_t* slot_start, int32_t* info, cudaStream_t s) {
  lora_plan_kernel<<<(unsigned)n_slots + 1, kPlanThreads, 0, s>>>(ids, (int)ntok, (int)n_slots,
                                                                  order, slot_start, info);
  note_launch();
  return cudaGetLastError();
}

namespace {

template <class TX, class TW>
cudaError_t shrink(const LoraArgs& a, const void* X, int64_t ldx, int64_t K, const void* W,
                   int64_t stride_w, int64_t ld_rank, int64_t ld_k, int scaled, float* out,
                   int64_t ldo, cudaStream_t s) {
  dim3 grid((unsigned)a.ntok, (a.max_rank + 7) / 8);
  lora_shrink_simple<TX, TW><<<grid, dim3(32, 8), 0, s>>>(
      a, static_cast<const TX*>(X), ldx, K, static_cast<const TW*>(W), stride_w, ld_rank, ld_k,
      scaled, out, ldo);
  note_launch();
  return cudaGetLastError();
}

cudaError_t shrink_any(const LoraArgs& a, const void* X, int x_bf16, int64_t ldx, int64_t K,
                       const void* W, int64_t stride_w, int64_t ld_rank, int64_t ld_k, int scaled,
                       float* out, int64_t ldo, cudaStream_t s) {
  using B = __nv_bfloat16;
  if (x_bf16)
    return a.wt_bf16 ? shrink<B, B>(a, X, ldx, K, W, stride_w, ld_rank, ld_k, scaled, out, ldo, s)
                     : shrink<B, float>(a, X, ldx, K, W, stride_w, ld_rank, ld_k, scaled, out, ldo, s);
  return a.wt_bf16 ? shrink<float, B>(a, X, ldx, K, W, stride_w, ld_rank, ld_k, scaled, out, ldo, s)
                   : shrink<float, float>(a, X, ldx, K, W, stride_w, ld_rank, ld_k, scaled, out, ldo, s);
}

template <class TW, class TY>
cudaError_t expand(const LoraArgs& a, const float* u, int64_t ldu, const void* W, int64_t stride_w,
                   int64_t ld_rank, int64_t ld_c, int scaled, void* Y, int64_t ldy, int64_t C,
                   cudaStream_t s) {
  dim3 grid((unsigned)a.ntok, (unsigned)((C + 255) / 256));
  lora_expand_simple<TW, TY><<<grid, 256, 0, s>>>(a, u, ldu, static_cast<const TW*>(W), stride_w,
                                                  ld_rank, ld_c, scaled, static_cast<TY*>(Y), ldy, C);
  note_launch();
  return cudaGetLastError();
}

cudaError_t expand_any(const LoraArgs& a, const float* u, int64_t ldu, const void* W,
                       int64_t stride_w, int64_t ld_rank, int64_t ld_c, int scaled, void* Y,
                       int y_bf16, int64_t ldy, int64_t C, cudaStream_t s) {
  using B = __nv_bfloat16;
  if (y_bf16)
    return a.wt_bf16 ? expand<B, B>(a, u, ldu, W, stride_w, ld_rank, ld_c, scaled, Y, ldy, C, s)
                     : expand<float, B>(a, u, ldu, W, stride_w, ld_rank, ld_c, scaled, Y, ldy, C, s);
  return a.wt_bf16 ? expand<B, float>(a, u, ldu, W, stride_w, ld_rank, ld_c, scaled, Y, ldy, C, s)
                   : expand<float, float>(a, u, ldu, W, stride_w, ld_rank, ld_c, scaled, Y, ldy, C, s);
}

template <class TX>
cudaError_t grad(const LoraArgs& a, const float* v, int64_t ldv, int scaled, const void* X,
                 int64_t ldx, const float* xs, int group, int64_t C, float* out, int64_t ld_rank,
                 int64_t ld_c, cudaStream_t s) {
  dim3 grid((unsigned)((C + 127) / 128), a.max_rank, a.n_slots);
  lora_grad_simple<TX><<<grid, 128, 0, s>>>(a, v, ldv, scaled, static_cast<const TX*>(X), ldx, xs,
                                            group, C, out, ld_rank, ld_c);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

size_t lora_workspace_bytes(const LoraArgs& a, bool backward) {
  (void)backward;
  return (size_t)a.ntok * (size_t)((a.max_rank + 3) / 4 * 4) * sizeof(float);
}

cudaError_t launch_lora_apply(const LoraArgs& a, const void* x, int x_bf16, int64_t ldx, void* y,
                              int y_bf16, int64_t ldy, float* u, int64_t ldu, void* ws,
                              cudaStream_t s) {
  if (!u) {
    u = static_cast<float*>(ws);
    ldu = (a.max_rank + 3) / 4 * 4;
  }
  cudaError_t e = shrink_any(a, x, x_bf16, ldx, a.n, a.A, a.stride_a, a.lda, 1, 0, u, ldu, s);
  if (e != cudaSuccess) return e;
  return expand_any(a, u, ldu, a.B, a.stride_b, 1, a.ldb, 1, y, y_bf16, ldy, a.rows, s);
}

cudaError_t launch_lora_backward(const LoraArgs& a, const void* dy, int dy_bf16, int64_t lddy,
                                 const void* x, int x_bf16, int64_t ldx, const int8_t* codes,
                                 const float* code_scales, int code_group, const float* u,
                                 int64_t ldu, void* dx, int dx_bf16, int64_t lddx, float* dA,
                                 float* dB, void* ws, cudaStream_t s) {
  using B = __nv_bfloat16;
  float* v = static_cast<float*>(ws);
  const int64_t ldv = (a.max_rank + 3) / 4 * 4;
  cudaError_t e = cudaSuccess;
  if (dx || dA)
    e = shrink_any(a, dy, dy_bf16, lddy, a.rows, a.B, a.stride_b, 1, a.ldb, 1, v, ldv, s);
  if (e == cudaSuccess && dx)
    e = expand_any(a, v, ldv, a.A, a.stride_a, a.lda, 1, 0, dx, dx_bf16, lddx, a.n, s);
  if (e == cudaSuccess && dA)
    e = codes ? grad<int8_t>(a, v, ldv, 0, codes, ldx, code_scales, code_group, a.n, dA, a.n, 1, s)
        : x_bf16 ? grad<B>(a, v, ldv, 0, x, ldx, nullptr, 0, a.n, dA, a.n, 1, s)
                 : grad<float>(a, v, ldv, 0, x, ldx, nullptr, 0, a.n, dA, a.n, 1, s);
  if (e == cudaSuccess && dB)
    e = dy_bf16 ? grad<B>(a, u, ldu, 1, dy, lddy, nullptr, 0, a.rows, dB, 1, a.max_rank, s)
                : grad<float>(a, u, ldu, 1, dy, lddy, nullptr, 0, a.rows, dB, 1, a.max_rank, s);
  return e;
}

}  // namespace gptq
