// out[t] = scale (X[t] W_a) for the adapter a of every token: the projection
// down to the rank (u = x A^T forward, v = s dy B backward).
//
// Ranks are the 16 rows of a matrix instruction, tokens its 8 columns, and
// the long axis K is summed (shrink_sum).  This kernel serves many tokens of
// the types and alignments that lora_shrink_tc.cu does not take: 64 tokens a
// CTA, whose warps split the tokens in two and K in four.  The CTAs of a
// cluster split K further and add their sums through distributed shared
// memory in rank order.  Bound by the bytes that registers can have under way,
// one block of 32 k ahead: 1500 x 2056 fp32 at rank 16 takes 19 us.
#include <cuda_runtime.h>

#include "lora_shrink.cuh"
#include "sm100_ptx.cuh"

namespace gptq {
namespace {

constexpr int kWarps = 8;

// RI: the ranks are W's contiguous axis.  NT: 8-token columns per warp, WT:
// warps side by side in the tokens, MR: 16-rank rows per CTA.
template <class TX, class TW, bool RI, int NT, int WT, int MR>
__global__ void __launch_bounds__(kWarps * 32)
    lora_shrink_kernel(const ShrinkArgs p) {
  constexpr int WK = kWarps / WT, TT = WT * NT * 8, RL = 16 * MR + 4;
  extern __shared__ float red[];  // [WK][TT][RL]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2;
  const int wt = warp % WT, wk = warp / WT;
  const int splits = gridDim.y, split = blockIdx.y;
  dep_launch();
  const Piece pc = find_piece(p.a, blockIdx.x, TT, 0);
  if (pc.slot < 0) return;  // the same in every CTA of the cluster
  const int r0 = blockIdx.z * 16 * MR;
  const int rank = lora_rank(p.a, pc.slot);
  float acc[MR][NT][4];
#pragma unroll
  for (int i = 0; i < MR; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;

  if (r0 < rank) {
    const TX* xrow[NT];
    int xvalid[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      const int t = piece_token(p.a, pc, (wt * NT + j) * 8 + g);
      xvalid[j] = t >= 0;
      xrow[j] = static_cast<const TX*>(p.X) + (int64_t)max(t, 0) * p.ldx;
    }
    const bool live = pc.count > wt * NT * 8;
    const TW* W = static_cast<const TW*>(p.W) + (int64_t)pc.slot * p.stride_w;
    const int K = (int)p.K;
    const bool vx = p.vec_x, vw = p.vec_w;

    if (live)
      shrink_sum<TX, TW, RI, NT, MR>(acc, xrow, xvalid, W, p.ldw, r0, rank, p.a.max_rank, K,
                                     32 * (split * WK + wk), 32 * WK * splits, vx, vw);
  }
  // sums of the warps along K
  shrink_put<RI, NT, MR, RL>(acc, red + (wk * TT + wt * NT * 8) * RL);
  __syncthreads();
  const float sc = p.scaled ? lora_scale(p.a, pc.slot) : 1.f;
  const int rmax = p.a.max_rank;
  auto store = [&](int tok, int r, float v) {
    const int t = piece_token(p.a, pc, tok);
    if (t >= 0 && r < rmax) p.out[(int64_t)t * p.ldo + r] = r < rank ? v * sc : 0.f;
  };
  for (int e = threadIdx.x; e < TT * 16 * MR; e += kWarps * 32) {
    const int tok = e / (16 * MR), r = e % (16 * MR);
    float s = red[tok * RL + r];
#pragma unroll
    for (int w = 1; w < WK; ++w) s += red[(w * TT + tok) * RL + r];
    if (splits == 1)
      store(tok, r0 + r, s);
    else
      red[tok * RL + r] = s;
  }
  if (splits == 1) return;
  // ... and of the cluster's CTAs, each finishing its share of the outputs
  ptx::cluster_sync();
  for (int e = split * kWarps * 32 + threadIdx.x; e < TT * 16 * MR; e += splits * kWarps * 32) {
    const int tok = e / (16 * MR), r = e % (16 * MR);
    float s = 0.f;
    for (int c = 0; c < splits; ++c) {
      float v;
      asm volatile("ld.shared::cluster.f32 %0, [%1];"
                   : "=f"(v)
                   : "r"(ptx::mapa_shared(red + tok * RL + r, c)));
      s += v;
    }
    store(tok, r0 + r, s);
  }
  ptx::cluster_sync();  // no CTA leaves while its sums are read
}

template <class TX, class TW, bool RI, int NT, int WT, int MR>
cudaError_t launch(const ShrinkArgs& p, int pieces, int splits, int rblocks, cudaStream_t s) {
  auto k = lora_shrink_kernel<TX, TW, RI, NT, WT, MR>;
  constexpr size_t smem = sizeof(float) * (kWarps / WT) * (WT * NT * 8) * (16 * MR + 4);
  cudaError_t e;
  if (smem > 48 * 1024 &&
      (e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) !=
          cudaSuccess)
    return e;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3(pieces, splits, rblocks);
  c.blockDim = dim3(kWarps * 32);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 1;
  at[0].val.clusterDim.y = splits;
  at[0].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = splits > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&c, k, p);
  note_launch();
  return e;
}

template <class TX, class TW, bool RI>
cudaError_t by_size(const ShrinkArgs& p, cudaStream_t s) {
  constexpr int kTile = 64, kWk = kWarps / 2;
  const int64_t T = p.a.ntok;
  const int pieces = (int)((T + kTile - 1) / kTile + (p.a.n_slots < T ? p.a.n_slots : T));
  // fp32 X: 4 rows of ranks would not fit the registers
  constexpr int kWide = sizeof(TX) == 4 ? 2 : 4;
  const int mr = p.a.max_rank <= 16 ? 1 : kWide;
  const int rblocks = (p.a.max_rank + 16 * mr - 1) / (16 * mr);
  // K is split over the cluster until two CTAs per SM exist or a warp would
  // have nothing left to sum.
  const int64_t most = (p.K + 32 * kWk - 1) / (32 * kWk);
  const int64_t want = (2 * num_sms() + pieces * rblocks - 1) / (pieces * rblocks);
  int splits = (int)(want < most ? want : most);
  splits = splits > 8 ? 8 : splits < 1 ? 1 : splits;
  return mr == 1 ? launch<TX, TW, RI, 4, 2, 1>(p, pieces, splits, rblocks, s)
                 : launch<TX, TW, RI, 4, 2, kWide>(p, pieces, splits, rblocks, s);
}

}  // namespace

cudaError_t launch_lora_shrink(const LoraArgs& a, bool forward, const void* X, int x_bf16,
                               int64_t ldx, float* out, int64_t ldo, cudaStream_t s) {
  ShrinkArgs p;
  p.a = a;
  p.gate = current_wait_gate();
  p.X = X;
  p.ldx = ldx;
  p.K = forward ? a.n : a.rows;
  p.W = forward ? a.A : a.B;
  p.stride_w = forward ? a.stride_a : a.stride_b;
  p.ldw = forward ? a.lda : a.ldb;
  p.scaled = !forward;
  p.vec_x = rows_aligned(X, ldx, 0, x_bf16 ? 2 : 4, 16);
  const int ew = a.wt_bf16 ? 2 : 4;
  p.vec_w = rows_aligned(p.W, p.ldw, a.n_slots > 1 ? p.stride_w : 0, ew, forward ? 16 : 4 * ew);
  p.out = out;
  p.ldo = ldo;
  p.vec_o = rows_aligned(out, ldo, 0, 4, 16);
  if (x_bf16 && a.wt_bf16 && p.vec_x && slots_mappable(p.W, p.ldw, p.stride_w, a.n_slots))
    return launch_lora_shrink_tc(p, !forward, s);
  if (x_bf16) {
    if (forward)
      return a.wt_bf16 ? by_size<bf16, bf16, false>(p, s)
                       : by_size<bf16, float, false>(p, s);
    return a.wt_bf16 ? by_size<bf16, bf16, true>(p, s) : by_size<bf16, float, true>(p, s);
  }
  if (forward)
    return a.wt_bf16 ? by_size<float, bf16, false>(p, s)
                     : by_size<float, float, false>(p, s);
  return a.wt_bf16 ? by_size<float, bf16, true>(p, s) : by_size<float, float, true>(p, s);
}

}  // namespace gptq
