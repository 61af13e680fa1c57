// What the kernels of the projection down to the rank share.
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
  WaitGate gate;     // test gate and time limit of the tcgen05 kernel's waits
};

// bf16 X and W with 16-byte aligned rows
cudaError_t launch_lora_shrink_tc(const ShrinkArgs& p, bool ranks_inner, cudaStream_t s);

namespace {

// acc[i][j] += (ranks r0 + 16 i ..) x (8 tokens of column j) over the k of this
// warp: blocks of 32 from k0 on, `step` apart, one block loaded ahead.  Nothing
// is staged in shared memory: each element of X and W is needed by exactly one
// warp of the CTA, and because a sum does not care for the order of its terms,
// the instruction's 16 inner slots may stand for any 16 values of k.  Thread q
// of a quad takes 8 consecutive k of a block (one 16-byte load of bf16) and
// feeds elements 4s .. 4s + 3 to the block's s-th instruction, on both sides.
// RI (ranks are W's contiguous axis, B of the backward pass): threads load 4
// ranks of one k and the 8 x 8 register transpose turns them.
template <class TX, class TW, bool RI, int NT, int MR>
__device__ __forceinline__ void shrink_sum(float (&acc)[MR][NT][4], const TX* const (&xrow)[NT],
                                           const int (&xvalid)[NT], const TW* W, int64_t ldw,
                                           int r0, int rank, int rmax, int K, int k0, int step,
                                           bool vx, bool vw) {
  constexpr int NX = Parts<TX>::n, NW = Parts<TW>::n;
  const int g = (threadIdx.x & 31) >> 2, q = threadIdx.x & 3;
  struct Frag {
    Raw<TX, 8> x[NT];
    Raw<TW, 8> w[MR][2];  // RI: [l / 2] holds loads l = 0, 1 (4 elements each) of 16 ranks
  };
  auto load = [&](Frag& f, int kb) {
    const int k = kb + 8 * q;
#pragma unroll
    for (int j = 0; j < NT; ++j) raw_load(f.x[j], xrow[j] + k, xvalid[j] ? K - k : 0, vx);
#pragma unroll
    for (int i = 0; i < MR; ++i) {
      if constexpr (!RI) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = r0 + 16 * i + 8 * h + g;
          raw_load(f.w[i][h], W + (int64_t)r * ldw + k, r < rank ? K - k : 0, vw);
        }
      } else {
        const int r = r0 + 16 * i + 4 * q;
#pragma unroll
        for (int l = 0; l < 4; ++l) {
          const int kk = kb + 8 * (g >> 1) + 2 * l + (g & 1);
          Raw<TW, 4> v;
          raw_load_part(v, W + (int64_t)kk * ldw + r, kk < K ? rank - r : 0, rmax - r, vw);
#pragma unroll
          for (int e = 0; e < (int)(sizeof(v.w) / 4); ++e)
            f.w[i][l >> 1].w[(l & 1) * (int)(sizeof(v.w) / 4) + e] = v.w[e];
        }
      }
    }
  };
  // 16 ranks x 16 k of W for instruction s as parts: a0 .. a3
  auto factor = [&](const Frag& f, int i, int s, uint32_t (&w)[4][NW]) {
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
  };
  // The instruction cuts its sum off every time, so the products of a block (of
  // an instruction's 16 k, if X is fp32) are summed by themselves, the small
  // ones first, and added to the running sum with rounding.
  auto compute = [&](const Frag& f) {
    if constexpr (NX == 1) {
#pragma unroll
      for (int i = 0; i < MR; ++i) {
        if (r0 + 16 * i >= rank) break;
        uint32_t w[2][4][NW];
        factor(f, i, 0, w[0]);
        factor(f, i, 1, w[1]);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int c = NW - 1; c >= 0; --c)
#pragma unroll
            for (int s = 0; s < 2; ++s) {
              const uint32_t a[4] = {w[s][0][c], w[s][1][c], w[s][2][c], w[s][3][c]};
              mma16816(t, a, f.x[j].w[2 * s], f.x[j].w[2 * s + 1]);
            }
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] += t[e];
        }
      }
    } else {
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
          uint32_t w[4][NW];
          factor(f, i, s, w);
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int c = NW - 1; c >= 0; --c) {
              const uint32_t a[4] = {w[0][c], w[1][c], w[2][c], w[3][c]};
#pragma unroll
              for (int d = NX - 1; d >= 0; --d)
                if (c + d <= 2) mma16816(t, a, b[j][0][d], b[j][1][d]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][j][e] += t[e];
          }
        }
      }
    }
  };
  if (k0 >= K) return;
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

// The sums of a warp to red[token][rank], RL floats a token.
template <bool RI, int NT, int MR, int RL>
__device__ __forceinline__ void shrink_put(const float (&acc)[MR][NT][4], float* red) {
  const int g = (threadIdx.x & 31) >> 2, q = threadIdx.x & 3;
#pragma unroll
  for (int i = 0; i < MR; ++i) {
    const int ra = 16 * i + (RI ? 4 * (g >> 1) + (g & 1) : g);
    const int rb = ra + (RI ? 2 : 8);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        red[(8 * j + 2 * q + e) * RL + ra] = acc[i][j][e];
        red[(8 * j + 2 * q + e) * RL + rb] = acc[i][j][2 + e];
      }
  }
}

}  // namespace
}  // namespace gptq
