// Y[t] += scale (u[t] W_a) for the adapter a of every token: the projection
// back from the rank (y += s u B^T forward, dx += v A backward).
//
// Bound by reading and writing Y once.  Tokens are the 16 rows of a matrix
// instruction, columns of Y its 8 columns, the ranks are summed 16 at a time
// (quad thread q takes ranks 4q .. 4q + 3 of the 16 on both sides).  The
// columns of two instructions are dealt out so that a thread ends up with 4
// consecutive columns of Y: one 16-byte access of fp32, 8 bytes of bf16.  u is
// fp32; it enters as 3 bf16 parts (exact) towards an fp32 Y, as 2 parts
// (2^-17) towards a bf16 Y, whose own rounding is 2^-8.
#include <cuda_runtime.h>

#include "lora_mma.cuh"

namespace gptq {
namespace {

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
  int vec_w, vec_y;
  void* Y;
  int64_t ldy;
  int64_t C;    // columns of Y
};

template <class T>
__device__ __forceinline__ void load4(float (&v)[4], const T* p, int valid, bool vec) {
  Raw<T, 4> r;
  raw_load<false>(r, p, valid, vec);  // Y is written by this kernel
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      v[2 * i] = __uint_as_float(r.w[i] << 16);
      v[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = r.w[i];
  }
}
template <class T>
__device__ __forceinline__ void store4(T* p, const float (&v)[4], int valid, bool vec) {
  if (valid >= 4 && vec) {
    if constexpr (sizeof(T) == 2) {
      __nv_bfloat162 h[2] = {__floats2bfloat162_rn(v[0], v[1]), __floats2bfloat162_rn(v[2], v[3])};
      *reinterpret_cast<uint2*>(p) = *reinterpret_cast<uint2*>(h);
    } else {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < valid) p[i] = from_f32<T>(v[i]);
  }
}

// CI: the columns of Y are W's contiguous axis.  NG: 16-column groups per
// warp.  ONE: max_rank <= 16, so W's piece stays in registers.
template <class TW, class TY, bool CI, int NG, bool ONE>
__global__ void __launch_bounds__(256) lora_expand_kernel(const ExpandArgs p) {
  constexpr int NU = sizeof(TY) == 2 ? 2 : 3, NW = Parts<TW>::n;
  extern __shared__ float us[];  // [tile][RL], then the tokens
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  dep_launch();
  const Piece pc = find_piece(p.a, blockIdx.x / p.strips, p.tile, 0);
  const int rank = pc.slot < 0 ? 0 : lora_rank(p.a, pc.slot);
  if (rank == 0) {
    dep_wait();
    return;
  }
  const int rp = (rank + 15) & ~15;
  const int RL = (rp & 16) ? rp : rp + 16;  // rows 16 floats apart modulo 32 banks
  int* toks = reinterpret_cast<int*>(us + p.tile * RL);
  const TW* W = static_cast<const TW*>(p.W) + (int64_t)pc.slot * p.stride_w;
  const int C = (int)p.C;
  const int c0 = (int)((blockIdx.x % p.strips) * (blockDim.x >> 5) + warp) * 16 * NG;
  const bool vw = p.vec_w, vy = p.vec_y;

  uint32_t w[2 * NG][2][NW];  // [instruction][rank pair][part]
  auto load_w = [&](int ch) {
#pragma unroll
    for (int n = 0; n < NG; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        Raw<TW, 4> r;
        if constexpr (!CI) {  // h: instruction; a row of W holds the ranks of one column
          const int c = c0 + 16 * n + 4 * (g >> 1) + 2 * h + (g & 1);
          raw_load(r, W + (int64_t)c * p.ldw + 16 * ch + 4 * q, c < C ? rank - 16 * ch - 4 * q : 0,
                   vw);
          raw_pair(r, 0, w[2 * n + h][0]);
          raw_pair(r, 1, w[2 * n + h][1]);
        } else {  // h: rank pair; a row of W holds the columns of one rank
          const int i = 16 * ch + 4 * (g >> 1) + 2 * h + (g & 1);
          const int c = c0 + 16 * n + 4 * q;
          raw_load(r, W + (int64_t)i * p.ldw + c, i < rank ? C - c : 0, vw);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t t[NW];
            raw_pair(r, j, t);
#pragma unroll
            for (int c2 = 0; c2 < NW; ++c2) w[2 * n + j][h][c2] = transpose8x8(t[c2]);
          }
        }
      }
  };
  if (ONE) load_w(0);
  for (int i = threadIdx.x; i < p.tile; i += blockDim.x) toks[i] = piece_token(p.a, pc, i);
  const float sc = p.scaled ? lora_scale(p.a, pc.slot) : 1.f;
  __syncthreads();
  dep_wait();  // u comes from the kernel before this one
  const int rows16 = (pc.count + 15) & ~15;
  for (int e = threadIdx.x; e < rows16 * rp; e += blockDim.x) {
    const int i = e / rp, r = e - i * rp;
    const int t = toks[i];
    us[i * RL + r] = (t >= 0 && r < rank) ? p.u[(int64_t)t * p.ldu + r] * sc : 0.f;
  }
  __syncthreads();
  if (c0 >= C) return;
  TY* Y = static_cast<TY*>(p.Y);
  for (int m0 = 0; m0 < pc.count; m0 += 16) {
    const int t0 = toks[m0 + g], t1 = toks[m0 + 8 + g];
    float y[NG][2][4];
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      const int c = c0 + 16 * n + 4 * q;
      load4(y[n][0], Y + (int64_t)max(t0, 0) * p.ldy + c, t0 >= 0 ? C - c : 0, vy);
      load4(y[n][1], Y + (int64_t)max(t1, 0) * p.ldy + c, t1 >= 0 ? C - c : 0, vy);
    }
    float acc[2 * NG][4];
#pragma unroll
    for (int j = 0; j < 2 * NG; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
    for (int ch = 0; ch < (ONE ? 1 : rp / 16); ++ch) {
      if (!ONE) load_w(ch);
      const float4 ua = *reinterpret_cast<const float4*>(us + (m0 + g) * RL + 16 * ch + 4 * q);
      const float4 ub = *reinterpret_cast<const float4*>(us + (m0 + 8 + g) * RL + 16 * ch + 4 * q);
      uint32_t a[4][NU];
      split_pair<NU>(ua.x, ua.y, a[0]);
      split_pair<NU>(ub.x, ub.y, a[1]);
      split_pair<NU>(ua.z, ua.w, a[2]);
      split_pair<NU>(ub.z, ub.w, a[3]);
#pragma unroll
      for (int c = 0; c < NU; ++c) {
        const uint32_t af[4] = {a[0][c], a[1][c], a[2][c], a[3][c]};
#pragma unroll
        for (int d = 0; d < NW; ++d) {
          if (c + d > 2) continue;
#pragma unroll
          for (int j = 0; j < 2 * NG; ++j) mma16816(acc[j], af, w[j][0][d], w[j][1][d]);
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NG; ++n) {
      const int c = c0 + 16 * n + 4 * q;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t = h ? t1 : t0;
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = y[n][h][e] + acc[2 * n + (e >> 1)][2 * h + (e & 1)];
        store4(Y + (int64_t)max(t, 0) * p.ldy + c, v, t >= 0 ? C - c : 0, vy);
      }
    }
  }
}

template <class TW, class TY, bool CI, int NG, bool ONE>
cudaError_t launch(ExpandArgs p, int threads, cudaStream_t s) {
  auto k = lora_expand_kernel<TW, TY, CI, NG, ONE>;
  const int rp = (p.a.max_rank + 15) / 16 * 16;
  const size_t smem = (size_t)p.tile * (rp + 16) * sizeof(float) + p.tile * sizeof(int);
  cudaError_t e;
  if (smem > 48 * 1024 &&
      (e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) !=
          cudaSuccess)
    return e;
  const int64_t T = p.a.ntok;
  const int64_t pieces = (T + p.tile - 1) / p.tile + (p.a.n_slots < T ? p.a.n_slots : T);
  const int strip = threads / 32 * 16 * NG;
  cudaLaunchConfig_t c = {};
  p.strips = (int)((p.C + strip - 1) / strip);
  if (pieces * p.strips > INT32_MAX) return cudaErrorInvalidConfiguration;
  c.gridDim = dim3((unsigned)(pieces * p.strips));
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  e = cudaLaunchKernelEx(&c, k, p);
  note_launch();
  return e;
}

template <class TW, class TY, bool CI>
cudaError_t by_size(const ExpandArgs& p, cudaStream_t s) {
  const bool one = p.a.max_rank <= 16;
  if (p.tile == 16)
    return one ? launch<TW, TY, CI, 1, true>(p, 128, s) : launch<TW, TY, CI, 1, false>(p, 128, s);
  return one ? launch<TW, TY, CI, 2, true>(p, 256, s) : launch<TW, TY, CI, 2, false>(p, 256, s);
}

template <class TW, class TY>
cudaError_t by_axis(const ExpandArgs& p, bool forward, cudaStream_t s) {
  return forward ? by_size<TW, TY, false>(p, s) : by_size<TW, TY, true>(p, s);
}

}  // namespace

cudaError_t launch_lora_expand(const LoraArgs& a, bool forward, const float* u, int64_t ldu,
                               void* Y, int y_bf16, int64_t ldy, cudaStream_t s) {
  ExpandArgs p;
  p.a = a;
  p.u = u;
  p.ldu = ldu;
  p.W = forward ? a.B : a.A;
  p.stride_w = forward ? a.stride_b : a.stride_a;
  p.ldw = forward ? a.ldb : a.lda;
  p.scaled = forward;
  p.tile = lora_tile(a);
  const int ew = a.wt_bf16 ? 2 : 4, ey = y_bf16 ? 2 : 4;
  p.vec_w = rows_aligned(p.W, p.ldw, a.n_slots > 1 ? p.stride_w : 0, ew, 4 * ew);
  p.vec_y = rows_aligned(Y, ldy, 0, ey, 4 * ey);
  p.Y = Y;
  p.ldy = ldy;
  p.C = forward ? a.rows : a.n;
  if (y_bf16)
    return a.wt_bf16 ? by_axis<bf16, bf16>(p, forward, s) : by_axis<float, bf16>(p, forward, s);
  return a.wt_bf16 ? by_axis<bf16, float>(p, forward, s) : by_axis<float, float>(p, forward, s);
}

}  // namespace gptq
