// Both projections of an adapter in one launch, for few tokens (or few to a
// slot): u[t] = X[t] W1_a and Y[t] += scale u[t] W2_a.
//
// Bound by reading the adapters once (rank (n + rows) elements each) and by
// latency: a single token at 4096 x 4096 and rank 16 reads 256 KB, so it is a
// launch, two dependent trips to memory and an exchange.  A cluster of up to
// 16 CTAs takes 16 tokens of a slot.  Its warps split the long axis of the
// first projection (shrink_sum), the CTAs exchange their sums of u through
// distributed shared memory, each adding all of them in rank order, and then
// take the columns of Y in turn.  While the first projection runs, the CTA's
// parts of W2 and Y are on their way into L2.  Measured: 6 us of the device for
// one token at 4096 x 4096 and rank 16 (two launches: 13 us); 24 us (adapters
// in L2) to 30 us for 64 tokens of 32 adapters of ranks up to 64 at 4096 x 11008, 30 MB.
// There, and at 2048 tokens of 8 adapters (11008 x 4096, rank 16, 40 us), warps
// mostly wait for memory: 11 to 13 of them an SM issue in 17 % of the cycles, the
// long scoreboard is the largest stall, DRAM and L2 are at 14 to 20 %.  Every
// piece has the same number of CTAs, so those of the largest rank take longest.
#include <cuda_runtime.h>

#include "lora_expand.cuh"
#include "lora_shrink.cuh"
#include "sm100_ptx.cuh"

namespace gptq {
namespace {

constexpr int kWarps = 8, kTok = 16;

struct FewArgs {
  LoraArgs a;
  const void* X;
  int64_t ldx, K;
  const void* W1;
  int64_t stride1, ld1;
  const void* W2;
  int64_t stride2, ld2;
  float* out;
  int64_t ldo;
  void* Y;
  int64_t ldy, C;
  int strips;  // of 16 columns, per CTA
  int vec_x, vec_1, vec_2, vec_y;
  int fast;    // Y's columns and W2's contiguous axis come in whole pieces of 4
  int ahead, ahead_y;  // W2's and Y's part of a CTA are whole 16-byte pieces
};

// BWD: ranks are W1's, columns W2's contiguous axis.  MR: 16-rank rows per pass
// over X.
template <class TX, class TW, class TY, bool BWD, int MR>
__global__ void __launch_bounds__(kWarps * 32, 2)
    lora_few_kernel(const FewArgs p) {
  constexpr int RL = 16 * MR + 4;
  constexpr int NU = sizeof(TY) == 2 ? 2 : 3, NW = Parts<TW>::n, E = 4, NJ = 2;
  constexpr int kHeld = MR == 1 ? 1 : sizeof(TW) == 4 ? 2 : 4;  // chunks of W2 loaded ahead
  constexpr int kDeep = MR == 1 ? 4 : sizeof(TW) == 4 ? 2 : 3;  // strips under way in registers
  extern __shared__ float smem[];
  __shared__ int toks[kTok];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int ctas = gridDim.y, cta = blockIdx.y;
  dep_launch();
  const Piece pc = find_piece(p.a, blockIdx.x, kTok, 0);
  if (pc.slot < 0) return;  // the same in every CTA of the cluster
  const int rank = lora_rank(p.a, pc.slot), rmax = p.a.max_rank;
  const int rp = (rank + 15) & ~15;
  const int UL = (rp & 16) ? rp : rp + 16;  // rows 16 floats apart modulo 32 banks
  float* red = smem;                        // [warp][16 tokens][RL]
  float* sum = smem + kWarps * kTok * RL;   // [16 tokens][UL]: this CTA's part of u
  float* us = sum + kTok * UL;              // u, scaled
  uint4* uf = reinterpret_cast<uint4*>(us + kTok * UL);  // its parts, [16 ranks][part][lane]
  const TW* W1 = static_cast<const TW*>(p.W1) + (int64_t)pc.slot * p.stride1;
  const TW* W2 = static_cast<const TW*>(p.W2) + (int64_t)pc.slot * p.stride2;
  const int C = (int)p.C, K = (int)p.K;
  const int cbegin = p.Y ? min(cta * p.strips * 16, C) : 0;
  const int cend = p.Y ? min(cbegin + p.strips * 16, C) : 0;
  if (p.ahead && cend > cbegin) {
    // rows of W2: one stretch of all columns' ranks, or a stretch per rank
    const int rows = BWD ? rank : 1;
    const int bytes = (cend - cbegin) * (BWD ? 1 : rmax) * (int)sizeof(TW);
    for (int r = tid; r < rows; r += kWarps * 32)
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                       W2 + (BWD ? (int64_t)r * p.ld2 + cbegin : (int64_t)cbegin * p.ld2)),
                   "r"(bytes)
                   : "memory");
  }
  if (tid < kTok) {
    const int t = piece_token(p.a, pc, tid);
    toks[tid] = t;
    if (p.ahead_y && t >= 0 && cend > cbegin && rank > 0)
      asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                       static_cast<const TY*>(p.Y) + (int64_t)t * p.ldy + cbegin),
                   "r"((cend - cbegin) * (int)sizeof(TY))
                   : "memory");
  }
  {
    const TX* xrow[2];
    int xvalid[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int t = piece_token(p.a, pc, 8 * j + g);
      xvalid[j] = t >= 0;
      xrow[j] = static_cast<const TX*>(p.X) + (int64_t)max(t, 0) * p.ldx;
    }
    for (int r0 = 0; r0 < rank; r0 += 16 * MR) {
      float acc[MR][2][4];
#pragma unroll
      for (int i = 0; i < MR; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;
      shrink_sum<TX, TW, BWD, 2, MR>(acc, xrow, xvalid, W1, p.ld1, r0, rank, rmax, K,
                                     32 * (cta * kWarps + warp), 32 * kWarps * ctas, p.vec_x,
                                     p.vec_1);
      shrink_put<BWD, 2, MR, RL>(acc, red + warp * kTok * RL);
      __syncthreads();
      const int here = min(16 * MR, rp - r0);
      for (int e = tid; e < kTok * here; e += kWarps * 32) {
        const int tok = e / here, r = e % here;
        float s = red[tok * RL + r];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) s += red[(w * kTok + tok) * RL + r];
        sum[tok * UL + r0 + r] = s;
      }
      __syncthreads();
    }
  }
  // every CTA's sums are there; and toks, which without a cluster and at rank 0
  // no barrier has stood behind yet
  if (ctas > 1) ptx::cluster_sync();
  else __syncthreads();
  const float sc = lora_scale(p.a, pc.slot);
  for (int e = tid; e < kTok * rp; e += kWarps * 32) {
    const int tok = e / rp, r = e % rp;
    float s = 0.f;
    if (tok < pc.count && r < rank) {
      if (ctas > 1) {
        for (int c = 0; c < ctas; ++c) {
          float v;
          asm volatile("ld.shared::cluster.f32 %0, [%1];"
                       : "=f"(v)
                       : "r"(ptx::mapa_shared(sum + tok * UL + r, c)));
          s += v;
        }
      } else {
        s = sum[tok * UL + r];
      }
    }
    us[tok * UL + r] = s * sc;
    // forward: u as it is; backward: v is scaled
    if (p.out && tok % ctas == cta && toks[tok] >= 0 && r < rmax)
      p.out[(int64_t)toks[tok] * p.ldo + r] = BWD ? s * sc : s;
  }
  if (p.out)  // ranks from rp on
    for (int e = tid; e < kTok * (rmax - rp); e += kWarps * 32) {
      const int tok = e / (rmax - rp), r = rp + e % (rmax - rp);
      if (tok % ctas == cta && toks[tok] >= 0) p.out[(int64_t)toks[tok] * p.ldo + r] = 0.f;
    }
  // this CTA has read the others' sums; nobody leaves before all have
  __syncwarp();
  if (ctas > 1) asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
  __syncthreads();

  TY* Y = static_cast<TY*>(p.Y);
  const int chunks = rp / 16;
  if (p.Y) {  // the parts of u in instruction order, once for all columns
    for (int e = tid; e < chunks * 32; e += kWarps * 32) {
      const int l = e & 31, ch = e >> 5;
      const float4 ua = *reinterpret_cast<const float4*>(us + (l >> 2) * UL + 16 * ch + 4 * (l & 3));
      const float4 ub =
          *reinterpret_cast<const float4*>(us + (8 + (l >> 2)) * UL + 16 * ch + 4 * (l & 3));
      uint32_t a[4][NU];
      split_pair<NU>(ua.x, ua.y, a[0]);
      split_pair<NU>(ub.x, ub.y, a[1]);
      split_pair<NU>(ua.z, ua.w, a[2]);
      split_pair<NU>(ub.z, ub.w, a[3]);
#pragma unroll
      for (int c = 0; c < NU; ++c)
        uf[(ch * NU + c) * 32 + l] = make_uint4(a[0][c], a[1][c], a[2][c], a[3][c]);
    }
    __syncthreads();
  }
  const int t0 = toks[g], t1 = toks[8 + g];
  struct Strip {
    Raw<TY, E> y[2];
    Raw<TW, 4> w[kHeld][2];
  };
  // W2's operands of 16 ranks and 16 columns as loaded: forward 4 ranks of one
  // column for each of two instructions, backward 4 columns of one rank for
  // each of two rank pairs
  auto load_w = [&](Raw<TW, 4> (&w)[2], int c0, int ch) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if constexpr (!BWD) {
        const int c = c0 + 4 * (g >> 1) + 2 * h + (g & 1);
        const int i = 16 * ch + 4 * q;
        raw_load_part(w[h], W2 + (int64_t)c * p.ld2 + i, c < C ? rank - i : 0, rmax - i, p.vec_2);
      } else {
        const int i = 16 * ch + 4 * (g >> 1) + 2 * h + (g & 1), c = c0 + 4 * q;
        raw_load(w[h], W2 + (int64_t)i * p.ld2 + c, i < rank ? C - c : 0, p.vec_2);
      }
    }
  };
  // Whole aligned pieces of 4 (p.fast): few instructions a strip.  The pieces
  // of ranks that a thread reads are the same for all columns: bit ch of `on`.
  uint32_t on = 0;
#pragma unroll
  for (int ch = 0; ch < kHeld; ++ch)
    on |= (!BWD ? 16 * ch + 4 * q < rank : ch < chunks) ? 1u << ch : 0u;
  auto load = [&](Strip& s, int c0) {
    if (p.fast) {
      const int c = c0 + 4 * q;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int t = h ? t1 : t0;
        raw_zero(s.y[h]);
        if (t >= 0 && c < C) raw_fetch<false>(s.y[h], Y + (int64_t)t * p.ldy + c);
        if constexpr (!BWD) {
          const int cw = c0 + 4 * (g >> 1) + 2 * h + (g & 1);
          const TW* at = W2 + (int64_t)cw * p.ld2 + 4 * q;
          const uint32_t mine = cw < C ? on : 0u;
#pragma unroll
          for (int ch = 0; ch < kHeld; ++ch) {
            raw_zero(s.w[ch][h]);
            if (mine >> ch & 1) raw_fetch<true>(s.w[ch][h], at + 16 * ch);
          }
        } else {
          const int i = 4 * (g >> 1) + 2 * h + (g & 1);
          const TW* at = W2 + (int64_t)i * p.ld2 + c;
#pragma unroll
          for (int ch = 0; ch < kHeld; ++ch) {
            raw_zero(s.w[ch][h]);
            if (16 * ch + i < rank && c < C) raw_fetch<true>(s.w[ch][h], at);
            at += 16 * p.ld2;
          }
        }
      }
      return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = h ? t1 : t0, c = c0 + 4 * q;
      raw_load<false>(s.y[h], Y + (int64_t)max(t, 0) * p.ldy + c, t >= 0 ? C - c : 0, p.vec_y);
    }
#pragma unroll
    for (int ch = 0; ch < kHeld; ++ch)
      if (ch < chunks) load_w(s.w[ch], c0, ch);
  };
  auto multiply = [&](float (&acc)[NJ][4], const Raw<TW, 4> (&raw)[2], int ch) {
    uint32_t w[NJ][2][NW];  // [instruction][rank pair][part]
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t t[NW];
        raw_pair(raw[h], j, t);
#pragma unroll
        for (int x = 0; x < NW; ++x) {
          if constexpr (!BWD) w[h][j][x] = t[x];
          else w[j][h][x] = transpose8x8(t[x]);
        }
      }
    // (towards an fp32 Y the products of 16 ranks are summed by themselves, the
    // small ones first, and added with rounding: the instruction cuts its sum off)
    float t[NJ][4];
    if constexpr (NU == 3) {
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) t[j][e] = 0.f;
    }
#pragma unroll
    for (int c = NU - 1; c >= 0; --c) {
      const uint4 f = uf[(ch * NU + c) * 32 + lane];
      const uint32_t af[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
      for (int d = NW - 1; d >= 0; --d) {
        if (c + d > 2) continue;
#pragma unroll
        for (int j = 0; j < NJ; ++j)
          mma16816(NU == 3 ? t[j] : acc[j], af, w[j][0][d], w[j][1][d]);
      }
    }
    if constexpr (NU == 3) {
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[j][e] += t[j][e];
    }
  };
  auto finish = [&](const Strip& s, int c0) {
    float acc[NJ][4];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[j][e] = 0.f;
#pragma unroll
    for (int ch = 0; ch < kHeld; ++ch) {
      if (ch < chunks) {
        Raw<TW, 4> w[2] = {s.w[ch][0], s.w[ch][1]};
        if (!BWD && p.fast && ch == (rank - 1) / 16) {  // ranks behind the slot's last
          raw_keep(w[0], rank - 16 * ch - 4 * q);
          raw_keep(w[1], rank - 16 * ch - 4 * q);
        }
        multiply(acc, w, ch);
      }
    }
#pragma unroll 1
    for (int ch = kHeld; ch < chunks; ++ch) {
      Raw<TW, 4> w[2];
      load_w(w, c0, ch);
      multiply(acc, w, ch);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = h ? t1 : t0, c = c0 + 4 * q;
      float d[E];
#pragma unroll
      for (int e = 0; e < E; ++e) d[e] = acc[e >> 1][2 * h + (e & 1)];
      add_store(Y + (int64_t)max(t, 0) * p.ldy + c, s.y[h], d, t >= 0 ? C - c : 0, p.vec_y);
    }
  };
  constexpr int kStep = 16 * kWarps;
  int c0 = cbegin + 16 * warp;
  if (c0 < cend && chunks > 0) {
    Strip s[kDeep];
#pragma unroll
    for (int i = 0; i + 1 < kDeep; ++i)
      if (c0 + i * kStep < cend) load(s[i], c0 + i * kStep);
#pragma unroll 1
    while (c0 < cend) {
#pragma unroll
      for (int i = 0; i < kDeep; ++i) {
        const int next = c0 + (kDeep - 1) * kStep;
        if (next < cend) load(s[(i + kDeep - 1) % kDeep], next);
        finish(s[i], c0);
        c0 += kStep;
        if (c0 >= cend) break;
      }
    }
  }
  __syncwarp();
  if (ctas > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
}

template <class TX, class TW, class TY, bool BWD, int MR>
cudaError_t launch(FewArgs p, cudaStream_t s) {
  auto k = lora_few_kernel<TX, TW, TY, BWD, MR>;
  auto bytes = [](int rp) {
    return sizeof(float) * (kWarps * kTok * (16 * MR + 4) + 2 * kTok * (rp + 16)) +
           (size_t)(rp / 16) * 3 * 32 * sizeof(uint4);
  };
  static std::atomic<uint64_t> raised{0};
  cudaError_t e = raise_limits(reinterpret_cast<const void*>(k), bytes(kLoraMaxRank), true, raised);
  if (e != cudaSuccess) return e;
  const size_t smem = bytes((p.a.max_rank + 15) / 16 * 16);
  const int64_t T = p.a.ntok;
  const int64_t pieces = (T + kTok - 1) / kTok + (p.a.n_slots < T ? p.a.n_slots : T);
  // At most two CTAs per SM, all of them there at once, but each warp something
  // to do in one of the projections.  Clusters of 16 leave SMs idle where more
  // than a dozen have to be placed (17 pieces: 13.7 us with 16, 8.8 with 8).
  const int64_t step = 32 * kWarps, cols = p.Y ? (p.C + 16 * kWarps - 1) / (16 * kWarps) : 1;
  const int64_t deep = (p.K + step - 1) / step;
  const int64_t most = deep > cols ? deep : cols;
  int64_t ctas = 2 * num_sms() / pieces;
  ctas = ctas > most ? most : ctas;
  if (ctas > 8 && 16 * pieces > 3 * num_sms() / 2) ctas = 8;
  ctas = ctas >= 16 ? 16 : ctas >= 8 ? 8 : ctas >= 4 ? 4 : ctas >= 2 ? 2 : 1;
  p.strips = (int)(((p.C + 15) / 16 + ctas - 1) / ctas);
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)pieces, (unsigned)ctas);
  c.blockDim = dim3(kWarps * 32);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 1;
  at[0].val.clusterDim.y = (unsigned)ctas;
  at[0].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = ctas > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&c, k, p);
  note_launch();
  return e;
}

template <class TX, class TW, class TY>
cudaError_t by_rank(const FewArgs& p, bool forward, cudaStream_t s) {
  if (forward)
    return p.a.max_rank <= 16 ? launch<TX, TW, TY, false, 1>(p, s)
                              : launch<TX, TW, TY, false, 2>(p, s);
  return p.a.max_rank <= 16 ? launch<TX, TW, TY, true, 1>(p, s)
                            : launch<TX, TW, TY, true, 2>(p, s);
}
template <class TX, class TW>
cudaError_t by_y(const FewArgs& p, bool forward, int y_bf16, cudaStream_t s) {
  return y_bf16 ? by_rank<TX, TW, bf16>(p, forward, s) : by_rank<TX, TW, float>(p, forward, s);
}

}  // namespace

cudaError_t launch_lora_few(const LoraArgs& a, bool forward, const void* X, int x_bf16,
                            int64_t ldx, float* out, int64_t ldo, void* Y, int y_bf16,
                            int64_t ldy, cudaStream_t s) {
  FewArgs p = {};
  p.a = a;
  p.X = X;
  p.ldx = ldx;
  p.K = forward ? a.n : a.rows;
  p.C = forward ? a.rows : a.n;
  p.W1 = forward ? a.A : a.B;
  p.stride1 = forward ? a.stride_a : a.stride_b;
  p.ld1 = forward ? a.lda : a.ldb;
  p.W2 = forward ? a.B : a.A;
  p.stride2 = forward ? a.stride_b : a.stride_a;
  p.ld2 = forward ? a.ldb : a.lda;
  p.out = out;
  p.ldo = ldo;
  p.Y = Y;
  p.ldy = ldy;
  const int ew = a.wt_bf16 ? 2 : 4, ey = y_bf16 ? 2 : 4;
  const int64_t s1 = a.n_slots > 1 ? p.stride1 : 0, s2 = a.n_slots > 1 ? p.stride2 : 0;
  p.vec_x = rows_aligned(X, ldx, 0, x_bf16 ? 2 : 4, 16);
  p.vec_1 = rows_aligned(p.W1, p.ld1, s1, ew, forward ? 16 : 4 * ew);
  p.vec_2 = rows_aligned(p.W2, p.ld2, s2, ew, 4 * ew);
  p.vec_y = Y ? rows_aligned(Y, ldy, 0, ey, 4 * ey) : 0;
  // (16 columns or 16 columns' ranks are whole 16-byte pieces; the last ones
  // have to be, too)
  const int64_t end = forward ? p.C * a.max_rank : p.C;
  p.ahead = Y && rows_aligned(p.W2, forward ? 0 : p.ld2, s2, ew, 16) && (end * ew) % 16 == 0 &&
            (!forward || p.ld2 == a.max_rank);
  p.fast = p.vec_2 && p.vec_y && p.C % 4 == 0 && (!forward || a.max_rank % 4 == 0);
  p.ahead_y = Y && rows_aligned(Y, ldy, 0, ey, 16) && (p.C * ey) % 16 == 0;
  if (x_bf16)
    return a.wt_bf16 ? by_y<bf16, bf16>(p, forward, y_bf16, s)
                     : by_y<bf16, float>(p, forward, y_bf16, s);
  return a.wt_bf16 ? by_y<float, bf16>(p, forward, y_bf16, s)
                   : by_y<float, float>(p, forward, y_bf16, s);
}

}  // namespace gptq
