// Y[t] += scale (u[t] W_a) for the adapter a of every token: the projection
// back from the rank (y += s u B^T forward, dx += v A backward).
//
// Bound by reading and writing Y once.  Tokens are the 16 rows of a matrix
// instruction, columns of Y its 8 columns, the ranks are summed 16 at a time
// (quad thread q takes ranks 4q .. 4q + 3 of the 16 on both sides).  The
// columns of an fp32 Y's two instructions, a bf16 Y's four, are dealt out so
// that a thread ends up with consecutive columns: one 16-byte access.  u is
// fp32; it enters as 3 bf16 parts (exact) towards an fp32 Y, as 2 parts
// (2^-17) towards a bf16 Y, whose own rounding is 2^-8.  This kernel serves many
// tokens of the types, ranks and alignments that lora_expand_tc.cu does not
// take.
#include <cuda_runtime.h>

#include "lora_expand.cuh"

namespace gptq {
namespace {

// Many tokens: a warp takes 32 tokens x 32 columns at a time, two halves of the
// piece in turn.  The next half's Y is loaded before the current one is
// computed, so a warp always has 2 KB (bf16) or 4 KB on the way.  The parts of
// u are made once per CTA, in instruction order, and serve all its columns.
// Measured: 1500 x 2048 fp32 at rank 16 11 us, 2.3 TB/s.
constexpr int kRows = 64, kRowWarps = 4;

template <class TW, class TY, bool CI>
__global__ void __launch_bounds__(kRowWarps * 32) lora_expand_rows_kernel(const ExpandArgs p) {
  constexpr int NU = sizeof(TY) == 2 ? 2 : 3, NW = Parts<TW>::n;
  constexpr int E = sizeof(TY) == 2 ? 8 : 4, NJ = 4, NE = E / 2, NG = NJ / NE, MT = kRows / 16;
  extern __shared__ uint4 uf[];  // [16 tokens][16 ranks][part][lane]
  __shared__ int toks[kRows];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  dep_launch();
  const Piece pc = find_piece(p.a, blockIdx.x / p.strips, kRows, 0);
  const int rank = pc.slot < 0 ? 0 : lora_rank(p.a, pc.slot);
  if (rank == 0) {
    dep_wait();
    return;
  }
  const int chunks = (rank + 15) / 16;
  const TW* W = static_cast<const TW*>(p.W) + (int64_t)pc.slot * p.stride_w;
  const int C = (int)p.C;
  const bool vw = p.vec_w, vy = p.vec_y;
  for (int i = threadIdx.x; i < kRows; i += blockDim.x) toks[i] = piece_token(p.a, pc, i);
  const float sc = p.scaled ? lora_scale(p.a, pc.slot) : 1.f;
  __syncthreads();
  dep_wait();  // u comes from a kernel before this one
  for (int e = threadIdx.x; e < MT * chunks * 32; e += blockDim.x) {
    const int l = e & 31, ch = (e >> 5) % chunks, mt = (e >> 5) / chunks;
    const int r = 16 * ch + 4 * (l & 3);
    uint32_t a[4][NU];  // rows g, g + 8 of the first rank pair, then of the second
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = toks[16 * mt + 8 * h + (l >> 2)];
      float v[4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
        v[x] = (t >= 0 && r + x < rank) ? p.u[(int64_t)t * p.ldu + r + x] * sc : 0.f;
      split_pair<NU>(v[0], v[1], a[h]);
      split_pair<NU>(v[2], v[3], a[2 + h]);
    }
#pragma unroll
    for (int c = 0; c < NU; ++c)
      uf[((mt * chunks + ch) * NU + c) * 32 + l] = make_uint4(a[0][c], a[1][c], a[2][c], a[3][c]);
  }
  __syncthreads();
  TY* Y = static_cast<TY*>(p.Y);
  const int first = (int)(blockIdx.x % p.strips) * p.turns;
  struct Rows { Raw<TY, E> v[2][2][NG]; };  // [16 tokens][rows g, g + 8][columns]
  auto column = [&](int turn) { return ((first + turn) * kRowWarps + warp) * 8 * NJ; };
  auto load = [&](Rows& y, int c0, int half) {
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t = toks[32 * half + 16 * mt + 8 * h + g];
        const TY* row = Y + (int64_t)max(t, 0) * p.ldy;
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          const int c = c0 + 4 * E * n + E * q;
          raw_load<false>(y.v[mt][h][n], row + c, t >= 0 ? C - c : 0, vy);  // Y is written below
        }
      }
  };
  auto compute = [&](const Rows& y, int c0, int half) {
    float acc[2][NJ][4];
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[mt][j][e] = 0.f;
    const uint4* u = uf + (half * 2 * chunks * NU) * 32 + lane;
#pragma unroll 1
    for (int ch = 0; ch < chunks; ++ch) {
      uint32_t w[NJ][2][NW];
      load_factor<TW, CI, NJ, E>(w, W, p.ldw, ch, rank, p.a.max_rank, c0, C, vw);
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        // (towards an fp32 Y the products of 16 ranks are summed by themselves,
        // the small ones first, and added with rounding: the instruction cuts
        // its sum off)
        float t[NJ][4];
        if constexpr (NU == 3) {
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) t[j][e] = 0.f;
        }
#pragma unroll
        for (int c = NU - 1; c >= 0; --c) {
          const uint4 f = u[((mt * chunks + ch) * NU + c) * 32];
          const uint32_t a[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
          for (int d = NW - 1; d >= 0; --d) {
            if (c + d > 2) continue;
#pragma unroll
            for (int j = 0; j < NJ; ++j)
              mma16816(NU == 3 ? t[j] : acc[mt][j], a, w[j][0][d], w[j][1][d]);
          }
        }
        if constexpr (NU == 3) {
#pragma unroll
          for (int j = 0; j < NJ; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[mt][j][e] += t[j][e];
        }
      }
    }
#pragma unroll
    for (int mt = 0; mt < 2; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t = toks[32 * half + 16 * mt + 8 * h + g];
        TY* row = Y + (int64_t)max(t, 0) * p.ldy;
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          const int c = c0 + 4 * E * n + E * q;
          float d[E];
#pragma unroll
          for (int e = 0; e < E; ++e) d[e] = acc[mt][NE * n + (e >> 1)][2 * h + (e & 1)];
          add_store(row + c, y.v[mt][h][n], d, t >= 0 ? C - c : 0, vy);
        }
      }
  };
  const bool both = pc.count > kRows / 2;
  Rows y0, y1;
  if (column(0) < C) load(y0, column(0), 0);
#pragma unroll 1
  for (int turn = 0; turn < p.turns; ++turn) {
    const int c0 = column(turn);
    if (c0 >= C) break;
    if (both) load(y1, c0, 1);
    compute(y0, c0, 0);
    if (turn + 1 < p.turns && column(turn + 1) < C) load(y0, column(turn + 1), 0);
    if (both) compute(y1, c0, 1);
  }
}

template <class K>
cudaError_t launch(K k, ExpandArgs p, int threads, int strip, int turns, size_t smem,
                   cudaStream_t s) {
  const int64_t T = p.a.ntok;
  const int64_t pieces = (T + kRows - 1) / kRows + (p.a.n_slots < T ? p.a.n_slots : T);
  p.turns = turns;
  p.strips = (int)((p.C + strip * turns - 1) / (strip * turns));
  if (pieces * p.strips > INT32_MAX) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)(pieces * p.strips));
  c.blockDim = dim3(threads);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&c, k, p);
  note_launch();
  return e;
}

template <class TW, class TY, bool CI>
cudaError_t by_size(const ExpandArgs& p, cudaStream_t s) {
  auto bytes = [](int rp) {
    return (size_t)(kRows / 16) * (rp / 16) * (sizeof(TY) == 2 ? 2 : 3) * 32 * 16;
  };
  // the limit of the largest rank: another thread may be launching with a rank
  // of its own
  static std::atomic<uint64_t> raised{0};
  const cudaError_t e =
      raise_limits(reinterpret_cast<const void*>(lora_expand_rows_kernel<TW, TY, CI>),
                   bytes(kLoraMaxRank), false, raised);
  if (e != cudaSuccess) return e;
  const int rp = (p.a.max_rank + 15) / 16 * 16;
  // a CTA's turns share its parts of u; about four rounds of CTAs stay
  const int strip = kRowWarps * 32;
  const int64_t units = (p.a.ntok + kRows - 1) / kRows * ((p.C + strip - 1) / strip);
  const int64_t turns = units / (4 * 3 * num_sms());
  return launch(lora_expand_rows_kernel<TW, TY, CI>, p, kRowWarps * 32, strip,
                (int)(turns < 1 ? 1 : turns > 8 ? 8 : turns), bytes(rp), s);
}

template <class TW, class TY>
cudaError_t by_axis(const ExpandArgs& p, bool forward, cudaStream_t s) {
  return forward ? by_size<TW, TY, false>(p, s) : by_size<TW, TY, true>(p, s);
}

}  // namespace

cudaError_t launch_lora_expand(const LoraArgs& a, bool forward, const float* u, int64_t ldu,
                               void* Y, int y_bf16, int64_t ldy, cudaStream_t s) {
  ExpandArgs p = {};
  p.a = a;
  p.gate = current_wait_gate();
  p.u = u;
  p.ldu = ldu;
  p.W = forward ? a.B : a.A;
  p.stride_w = forward ? a.stride_b : a.stride_a;
  p.ldw = forward ? a.ldb : a.lda;
  p.scaled = forward;
  p.vec_u = rows_aligned(u, ldu, 0, 4, 16);
  // at most E elements, at most 16 bytes (E = 4, or 8 of a bf16 Y)
  const int ew = a.wt_bf16 ? 2 : 4, ey = y_bf16 ? 2 : 4;
  const int wide = y_bf16 ? 8 : 4;
  const int bw = (forward ? 4 : wide) * ew;
  p.vec_w = rows_aligned(p.W, p.ldw, a.n_slots > 1 ? p.stride_w : 0, ew, bw > 16 ? 16 : bw);
  p.vec_y = rows_aligned(Y, ldy, 0, ey, wide * ey);
  p.Y = Y;
  p.ldy = ldy;
  p.C = forward ? a.rows : a.n;
  if (a.wt_bf16 && a.max_rank <= kExpandTcRank &&
      slots_mappable(p.W, p.ldw, p.stride_w, a.n_slots) && rows_aligned(Y, ldy, 0, ey, 16))
    return launch_lora_expand_tc(p, !forward, y_bf16, s);
  if (y_bf16)
    return a.wt_bf16 ? by_axis<bf16, bf16>(p, forward, s) : by_axis<float, bf16>(p, forward, s);
  return a.wt_bf16 ? by_axis<bf16, float>(p, forward, s) : by_axis<float, float>(p, forward, s);
}

}  // namespace gptq
