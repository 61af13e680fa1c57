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
  int strips;   // CTAs side by side in the columns
  int turns;    // column strips a CTA takes one after the other
  int vec_u, vec_w, vec_y;
  void* Y;
  int64_t ldy;
  int64_t C;    // columns of Y
  WaitGate gate;  // test gate and time limit of the tcgen05 kernel's waits
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

template <class T, int E>
__device__ __forceinline__ void add_store(T* p, const Raw<T, E>& y, const float (&d)[E], int valid,
                                          bool vec) {
  float v[E];
#pragma unroll
  for (int i = 0; i < E; ++i) v[i] = d[i];
  add_row(v, y);
  if (valid >= E && vec) {
    const Raw<T, E> o = round_row<T, E>(v);
    if constexpr (sizeof(o.w) == 16) {
      uint4 w;
      memcpy(&w, o.w, 16);
      *reinterpret_cast<uint4*>(p) = w;
    } else {
      uint2 w;
      memcpy(&w, o.w, 8);
      *reinterpret_cast<uint2*>(p) = w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (i < valid) p[i] = from_f32<T>(v[i]);
  }
}

// W's operands for 16 ranks (16 ch ..) and 8 NJ columns (c0 ..) of a warp:
// [instruction][rank pair][part].  CI: the columns are W's contiguous axis.
template <class TW, bool CI, int NJ, int E, int NW>
__device__ __forceinline__ void load_factor(uint32_t (&w)[NJ][2][NW], const TW* W, int64_t ldw,
                                            int ch, int rank, int rmax, int c0, int C,
                                            bool vec) {
  constexpr int NE = E / 2, NG = NJ / NE;
  const int g = (threadIdx.x & 31) >> 2, q = threadIdx.x & 3;
#pragma unroll
  for (int n = 0; n < NG; ++n) {
    const int cg = c0 + 4 * E * n;
    if constexpr (!CI) {  // a row of W holds the ranks of one column
#pragma unroll
      for (int h = 0; h < NE; ++h) {
        const int c = cg + E * (g >> 1) + 2 * h + (g & 1);
        Raw<TW, 4> r;
        const int i = 16 * ch + 4 * q;
        raw_load_part(r, W + (int64_t)c * ldw + i, c < C ? rank - i : 0, rmax - i, vec);
        raw_pair(r, 0, w[NE * n + h][0]);
        raw_pair(r, 1, w[NE * n + h][1]);
      }
    } else {  // a row of W holds the columns of one rank
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int i = 16 * ch + 4 * (g >> 1) + 2 * h + (g & 1);
        const int c = cg + E * q;
        Raw<TW, E> r;
        raw_load(r, W + (int64_t)i * ldw + c, i < rank ? C - c : 0, vec);
#pragma unroll
        for (int j = 0; j < NE; ++j) {
          uint32_t t[NW];
          raw_pair(r, j, t);
#pragma unroll
          for (int x = 0; x < NW; ++x) w[NE * n + j][h][x] = transpose8x8(t[x]);
        }
      }
    }
  }
}

}  // namespace
}  // namespace gptq
