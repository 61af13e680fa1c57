// out[t] = scale (X[t] W_a) for the adapter a of every token: the projection
// down to the rank (u = x A^T forward, v = s dy B backward).
//
// Ranks are the 16 rows of a matrix instruction, tokens its 8 columns, and
// the long axis K is summed.  Nothing is staged in shared memory: each
// element of X and W is needed by exactly one warp of the CTA, and because a
// sum does not care for the order of its terms, the instruction's 16 inner
// slots may stand for any 16 values of k.  Thread q of a quad takes 8
// consecutive k of a block of 32 (one 16-byte load of bf16) and feeds
// elements 4s .. 4s + 3 to the block's s-th instruction, on both sides.  When
// W's ranks are its contiguous axis (B of the backward pass), threads load 4
// ranks of one k and the 8 x 8 register transpose turns them.
//
// Warps of a CTA split K (and, at 64 tokens, the tokens in two); the CTAs of
// a cluster split K further, so that few tokens still spread over many SMs,
// and add their sums through distributed shared memory in rank order.
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
  constexpr int NX = Parts<TX>::n, NW = Parts<TW>::n;
  extern __shared__ float red[];  // [WK][TT][RL]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
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

    struct Frag {
      Raw<TX, 8> x[NT];
      Raw<TW, 8> w[MR][2];  // RI: [l / 2] holds loads l = 0, 1 (4 elements each) of 16 ranks
    };
    auto load = [&](Frag& f, int k0) {
      const int k = k0 + 8 * q;
#pragma unroll
      for (int j = 0; j < NT; ++j) raw_load(f.x[j], xrow[j] + k, xvalid[j] ? K - k : 0, vx);
#pragma unroll
      for (int i = 0; i < MR; ++i) {
        if constexpr (!RI) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = r0 + 16 * i + 8 * h + g;
            raw_load(f.w[i][h], W + (int64_t)r * p.ldw + k, r < rank ? K - k : 0, vw);
          }
        } else {
          const int r = r0 + 16 * i + 4 * q;
#pragma unroll
          for (int l = 0; l < 4; ++l) {
            const int kk = k0 + 8 * (g >> 1) + 2 * l + (g & 1);
            Raw<TW, 4> v;
            raw_load(v, W + (int64_t)kk * p.ldw + r, kk < K ? rank - r : 0, vw);
#pragma unroll
            for (int e = 0; e < (int)(sizeof(v.w) / 4); ++e)
              f.w[i][l >> 1].w[(l & 1) * (int)(sizeof(v.w) / 4) + e] = v.w[e];
          }
        }
      }
    };
    auto compute = [&](const Frag& f) {
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        uint32_t b[NT][2][NX];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          raw_pair(f.x[j], 2 * s, b[j][0]);
          raw_pair(f.x[j], 2 * s + 1, b[j][1]);
        }
#pragma unroll
        for (int i = 0; i < MR; ++i) {
          if (r0 + 16 * i >= rank) break;
          uint32_t w[4][NW];  // a0..a3 as parts
          if constexpr (!RI) {
            raw_pair(f.w[i][0], 2 * s, w[0]);
            raw_pair(f.w[i][1], 2 * s, w[1]);
            raw_pair(f.w[i][0], 2 * s + 1, w[2]);
            raw_pair(f.w[i][1], 2 * s + 1, w[3]);
          } else {
            // load l = 2s + h: pair 0 -> rows 0..7, pair 1 -> rows 8..15
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                uint32_t t[NW];
                raw_pair(f.w[i][s], 2 * h + e, t);
#pragma unroll
                for (int c = 0; c < NW; ++c) w[2 * h + e][c] = transpose8x8(t[c]);
              }
          }
#pragma unroll
          for (int c = 0; c < NW; ++c) {
            const uint32_t a[4] = {w[0][c], w[1][c], w[2][c], w[3][c]};
#pragma unroll
            for (int d = 0; d < NX; ++d) {
              if (c + d > 2) continue;
#pragma unroll
              for (int j = 0; j < NT; ++j) mma16816(acc[i][j], a, b[j][0][d], b[j][1][d]);
            }
          }
        }
      }
    };
    const int step = 32 * WK * splits;
    int k0 = 32 * (split * WK + wk);
    if (live && k0 < K) {
      Frag f[2];
      load(f[0], k0);
#pragma unroll 1
      while (true) {
        if (k0 + step < K) load(f[1], k0 + step);
        compute(f[0]);
        k0 += step;
        if (k0 >= K) break;
        if (k0 + step < K) load(f[0], k0 + step);
        compute(f[1]);
        k0 += step;
        if (k0 >= K) break;
      }
    }
  }
  // sums of the warps along K
  {
    float* mine = red + (wk * TT + wt * NT * 8) * RL;
#pragma unroll
    for (int i = 0; i < MR; ++i) {
      const int ra = 16 * i + (RI ? 4 * (g >> 1) + (g & 1) : g);
      const int rb = ra + (RI ? 2 : 8);
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          mine[(8 * j + 2 * q + e) * RL + ra] = acc[i][j][e];
          mine[(8 * j + 2 * q + e) * RL + rb] = acc[i][j][2 + e];
        }
    }
  }
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
  if (splits > 8 &&
      (e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) !=
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
cudaError_t by_size(const ShrinkArgs& p, int tile, cudaStream_t s) {
  const int64_t T = p.a.ntok;
  const int pieces = (int)((T + tile - 1) / tile + (p.a.n_slots < T ? p.a.n_slots : T));
  // fp32 X at 64 tokens: 4 rows of ranks would not fit the registers
  constexpr int kWide = sizeof(TX) == 4 ? 2 : 4;
  const int mr = p.a.max_rank <= 16 ? 1 : tile == 16 ? 4 : kWide;
  const int rblocks = (p.a.max_rank + 16 * mr - 1) / (16 * mr);
  // K is split over the cluster until two CTAs per SM exist or a warp would
  // have nothing left to sum.
  const int wk = tile == 16 ? kWarps : kWarps / 2;
  const int64_t most = (p.K + 32 * wk - 1) / (32 * wk);
  const int64_t want = (2 * num_sms() + pieces * rblocks - 1) / (pieces * rblocks);
  int splits = (int)(want < most ? want : most);
  splits = splits > 16 ? 16 : splits < 1 ? 1 : splits;
  if (splits > 8 && splits < 16) splits = 8;
  if (tile == 16)
    return mr == 1 ? launch<TX, TW, RI, 2, 1, 1>(p, pieces, splits, rblocks, s)
                   : launch<TX, TW, RI, 2, 1, 4>(p, pieces, splits, rblocks, s);
  return mr == 1 ? launch<TX, TW, RI, 4, 2, 1>(p, pieces, splits, rblocks, s)
                 : launch<TX, TW, RI, 4, 2, kWide>(p, pieces, splits, rblocks, s);
}

}  // namespace

cudaError_t launch_lora_shrink(const LoraArgs& a, bool forward, const void* X, int x_bf16,
                               int64_t ldx, float* out, int64_t ldo, cudaStream_t s) {
  ShrinkArgs p;
  p.a = a;
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
  const int tile = lora_tile(a);
  if (tile == 64 && x_bf16 && a.wt_bf16 && p.vec_x &&
      rows_aligned(p.W, p.ldw, a.n_slots > 1 ? p.stride_w : 0, 2, 16))
    return launch_lora_shrink_tc(p, !forward, s);
  if (x_bf16) {
    if (forward)
      return a.wt_bf16 ? by_size<bf16, bf16, false>(p, tile, s)
                       : by_size<bf16, float, false>(p, tile, s);
    return a.wt_bf16 ? by_size<bf16, bf16, true>(p, tile, s) : by_size<bf16, float, true>(p, tile, s);
  }
  if (forward)
    return a.wt_bf16 ? by_size<float, bf16, false>(p, tile, s)
                     : by_size<float, float, false>(p, tile, s);
  return a.wt_bf16 ? by_size<float, bf16, true>(p, tile, s) : by_size<float, float, true>(p, tile, s);
}

}  // namespace gptq
