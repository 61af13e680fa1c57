// Gradients of the adapters: out(i, c) = sum over a slot's tokens of
// f[t][i] X[t][c], with f = v and X = x for dA, f = scale u and X = dy for dB.
//
// Ranks are the 16 rows of a matrix instruction, columns of X its 8 columns,
// tokens are summed.  X is read once: a warp owns 32 columns and every rank of
// the CTA, a thread loads 8 columns of one token (16 bytes of bf16, 8 of
// codes), and the 8 x 8 register transpose turns rows of columns into the
// pairs of tokens that the instruction wants.  f is fp32 and enters as 3 bf16
// parts (exact); it is small and shared by all columns, so a block of 128
// tokens of it is split once per CTA and laid out in shared memory in
// instruction order.  Codes are exact in bf16; their scale belongs to a token
// and a group of columns, which a CTA's columns never leave, so it is
// multiplied onto f.
//
// Warps that are not side by side in the columns take turns at the tokens and
// are summed at the end.  A slot's tokens are cut into pieces for more CTAs;
// a slot of several pieces goes through the workspace, where a second kernel
// sums the pieces in order.
#include <cuda_runtime.h>

#include "lora_mma.cuh"

namespace gptq {
namespace {

constexpr int kWarps = 8;
constexpr int kBlockTok = 128;  // tokens of f staged at a time

// One of the two products of a launch
struct GradSide {
  const float* f;
  int64_t ldf;
  int scaled;
  const void* X;
  int64_t ldx;
  const float* xs;   // codes: scales, one per token and group
  int group;         // codes: columns per group (C: one group)
  int64_t C;
  float* out;
  int64_t ld_rank, ld_c;  // of out within a slot
  int64_t part;           // its offset in a piece's partial sums
  int strips;             // CTAs side by side in the columns
  int wc;                 // warps side by side in the columns
  int vec;
};

struct GradKernelArgs {
  LoraArgs a;
  GradSide side[2];
  int piece;           // tokens per piece, a multiple of kBlockTok
  float* partial;      // [piece of a slot of several][part_size]
  int64_t part_size;
  int room;            // pieces that partial holds: enough for any real plan,
                       // checked for one that is not (slot_start not ascending)
};

// 8 columns of a token as loaded
struct Codes8 { uint32_t w[2]; };
template <class T>
struct Row8 { using type = Raw<T, 8>; static constexpr int parts = Parts<T>::n; };
template <>
struct Row8<int8_t> { using type = Codes8; static constexpr int parts = 1; };

template <class T>
__device__ __forceinline__ void row_load(Raw<T, 8>& r, const T* p, int valid, bool vec) {
  raw_load(r, p, valid, vec);
}
__device__ __forceinline__ void row_load(Codes8& r, const int8_t* p, int valid, bool vec) {
  if (valid >= 8 && vec) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    r.w[0] = v.x;
    r.w[1] = v.y;
  } else {
    r.w[0] = r.w[1] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid)
        r.w[i / 4] |= (uint32_t)__ldg(reinterpret_cast<const uint8_t*>(p) + i) << (8 * (i & 3));
  }
}
template <class T, int N>
__device__ __forceinline__ void row_pair(const Raw<T, 8>& r, int i, uint32_t (&p)[N]) {
  raw_pair(r, i, p);
}
// Two signed bytes as bf16: with s the sign bit and m the low 7 bits the value
// is m - 128 s = (128 + m) - (128 + 128 s).  In bf16, 0x4300 | m is 128 + m
// and 0x4300 | (s << 7) is 128 or 256, so one exact subtraction does it.
__device__ __forceinline__ void row_pair(const Codes8& r, int i, uint32_t (&p)[1]) {
  const uint32_t b = __byte_perm(r.w[i >> 1], 0, (i & 1) ? 0x4342 : 0x4140);
  const uint32_t lo = (b & 0x007f007fu) | 0x43004300u, hi = (b & 0x00800080u) | 0x43004300u;
  const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&lo),
                                   *reinterpret_cast<const __nv_bfloat162*>(&hi));
  p[0] = *reinterpret_cast<const uint32_t*>(&d);
}

template <class TX, int MR>
__device__ __forceinline__ void grad_body(const GradKernelArgs& k, const GradSide& p,
                                          const Piece& pc, int strip, int r0, uint4* frag) {
  constexpr int NX = Row8<TX>::parts;
  constexpr int kSteps = kBlockTok / 16;
  constexpr int kFrag = kSteps * MR * 3 * 32;  // uint4 per block of tokens
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int wc = p.wc, wtok = kWarps / wc;
  const int wcol = warp % wc, wt = warp / wc;
  const int C = (int)p.C;
  const int cs = strip * 32 * wc;  // the CTA's first column
  const int c = cs + 32 * wcol + 8 * q;
  const int rank = lora_rank(k.a, pc.slot);
  const float sc = p.scaled ? lora_scale(k.a, pc.slot) : 1.f;
  const int64_t G = p.xs ? (p.C + p.group - 1) / p.group : 0;
  const int grp = p.xs ? cs / p.group : 0;
  const bool vec = p.vec;

  // The matrix instruction cuts its fp32 sum off instead of rounding it, up to
  // 2^-23 of it each time and always towards zero, so long sums would drift:
  // every 8 steps or more the running sum moves to `total`, which is rounded.
  float acc[MR][4][4], total[MR][4][4];
#pragma unroll
  for (int i = 0; i < MR; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = total[i][j][e] = 0.f;
  auto flush = [&]() {
#pragma unroll
    for (int i = 0; i < MR; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          total[i][j][e] += acc[i][j][e];
          acc[i][j][e] = 0.f;
        }
  };
  const int flush_mask = (wc < 2 ? 8 : wc < 4 ? 4 : 2) - 1;  // blocks of 8 wc / 8 steps

  const int count = r0 < rank ? pc.count : 0;
  typename Row8<TX>::type row[2][2];  // [turn][token g, g + 8]
  auto load = [&](typename Row8<TX>::type (&r)[2], int step) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int t = piece_token(k.a, pc, step * 16 + 8 * h + g);
      row_load(r[h], static_cast<const TX*>(p.X) + (int64_t)max(t, 0) * p.ldx + c,
               t >= 0 ? C - c : 0, vec);
    }
  };
  // f of 128 tokens: [16 tokens][16 ranks][part][lane] in instruction order
  auto stage = [&](uint4* dst, int tok0) {
    for (int e = threadIdx.x; e < kSteps * MR * 32; e += kWarps * 32) {
      const int l = e & 31, i = (e >> 5) % MR, st = (e >> 5) / MR;
      const int gg = l >> 2, qq = l & 3;
      const int ra = r0 + 16 * i + gg, rb = ra + 8;
      float va[4], vb[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int t = piece_token(k.a, pc, tok0 + 16 * st + 2 * qq + (x & 1) + 8 * (x >> 1));
        float m = sc;
        if (t >= 0 && p.xs) m *= p.xs[(int64_t)t * G + grp];
        const float* f = p.f + (int64_t)max(t, 0) * p.ldf;
        va[x] = (t >= 0 && ra < rank) ? f[ra] * m : 0.f;
        vb[x] = (t >= 0 && rb < rank) ? f[rb] * m : 0.f;
      }
      uint32_t a[4][3];
      split_pair<3>(va[0], va[1], a[0]);
      split_pair<3>(vb[0], vb[1], a[1]);
      split_pair<3>(va[2], va[3], a[2]);
      split_pair<3>(vb[2], vb[3], a[3]);
#pragma unroll
      for (int x = 0; x < 3; ++x)
        dst[((st * MR + i) * 3 + x) * 32 + l] = make_uint4(a[0][x], a[1][x], a[2][x], a[3][x]);
    }
  };
  auto compute = [&](const typename Row8<TX>::type (&r)[2], const uint4* src) {
    uint32_t b[4][2][NX];  // [8 columns][token pairs]
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t t[NX];
        row_pair(r[h], j, t);
#pragma unroll
        for (int d = 0; d < NX; ++d) b[j][h][d] = transpose8x8(t[d]);
      }
#pragma unroll
    for (int i = 0; i < MR; ++i) {
      if (r0 + 16 * i >= rank) break;
#pragma unroll
      for (int x = 0; x < 3; ++x) {
        const uint4 f = src[(i * 3 + x) * 32 + lane];
        const uint32_t a[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
        for (int d = 0; d < NX; ++d) {
          if (x + d > 2) continue;
#pragma unroll
          for (int j = 0; j < 4; ++j) mma16816(acc[i][j], a, b[j][0][d], b[j][1][d]);
        }
      }
    }
  };
  const int steps = (count + 15) / 16;
  if (wt < steps) load(row[0], wt);
  bool odd = false;
  for (int b0 = 0; b0 * kSteps < steps; ++b0) {
    uint4* fr = frag + (b0 & 1) * kFrag;
    stage(fr, b0 * kBlockTok);
    __syncthreads();
    for (int st = wt; st < kSteps; st += wtok) {
      const int step = b0 * kSteps + st;
      if (step >= steps) break;
      const bool more = step + wtok < steps;
      if (odd) {
        if (more) load(row[0], step + wtok);
        compute(row[1], fr + st * MR * 96);
      } else {
        if (more) load(row[1], step + wtok);
        compute(row[0], fr + st * MR * 96);
      }
      odd = !odd;
    }
    if ((b0 & flush_mask) == flush_mask) flush();
  }
  flush();
  __syncthreads();
  // sums of the warps that took turns at the tokens
  constexpr int RL = 33;
  float* red = reinterpret_cast<float*>(frag);  // [warp][16 MR][RL]
#pragma unroll
  for (int i = 0; i < MR; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        // instruction j's column 2q + e' is column 8q' + 2j + .. of the 32
        const int n = 2 * q + (e & 1);
        red[(warp * 16 * MR + 16 * i + g + 8 * (e >> 1)) * RL + 8 * (n >> 1) + 2 * j + (n & 1)] =
            total[i][j][e];
      }
  __syncthreads();
  const bool whole = pc.pieces == 1;
  if (!whole && pc.multi + pc.index >= k.room) return;
  float* out = whole ? p.out + (int64_t)pc.slot * k.a.max_rank * p.C
                     : k.partial + (int64_t)(pc.multi + pc.index) * k.part_size + p.part;
  for (int e = threadIdx.x; e < 16 * MR * 32 * wc; e += kWarps * 32) {
    // the faster index runs along out's contiguous axis
    int r, cc;
    if (p.ld_c == 1) {
      cc = e % (32 * wc);
      r = e / (32 * wc);
    } else {
      r = e % (16 * MR);
      cc = e / (16 * MR);
    }
    if (r0 + r >= k.a.max_rank || cs + cc >= C) continue;
    float s = 0.f;
    for (int w = 0; w < wtok; ++w)
      s += red[((w * wc + cc / 32) * 16 * MR + r) * RL + cc % 32];
    out[(r0 + r) * p.ld_rank + (int64_t)(cs + cc) * p.ld_c] = s;
  }
}

// TA: x's type, TB: dy's type
template <class TA, class TB, int MR>
__global__ void __launch_bounds__(kWarps * 32) lora_grad_kernel(const GradKernelArgs k) {
  extern __shared__ uint4 frag[];
  dep_launch();
  const int strips = k.side[0].strips + k.side[1].strips;
  const Piece pc = find_piece(k.a, blockIdx.x / strips, k.piece, 1);
  dep_wait();
  if (pc.slot < 0) return;
  const int s = blockIdx.x % strips;
  const int r0 = blockIdx.y * 16 * MR;
  if (s < k.side[0].strips)
    grad_body<TA, MR>(k, k.side[0], pc, s, r0, frag);
  else
    grad_body<TB, MR>(k, k.side[1], pc, s - k.side[0].strips, r0, frag);
}

// The slots of several pieces: their pieces summed in order.
__global__ void __launch_bounds__(256) lora_grad_join_kernel(const GradKernelArgs k) {
  dep_launch();
  // the blockIdx.y-th slot of several pieces
  const int lane = threadIdx.x & 31;
  int nth = blockIdx.y, slot = -1, first = 0, pieces = 0;
  for (int a0 = 0; a0 < k.a.n_slots && slot < 0; a0 += 32) {
    const int a = a0 + lane;
    int pcs = 0;
    if (a < k.a.n_slots)
      pcs = (max(lora_start(k.a, a + 1) - lora_start(k.a, a), 0) + k.piece - 1) / k.piece;
    if (pcs < 2) pcs = 0;
    unsigned m = __ballot_sync(~0u, pcs > 0);
    while (m && slot < 0) {
      const int l = __ffs(m) - 1;
      m &= m - 1;
      const int n = __shfl_sync(~0u, pcs, l);
      if (nth-- == 0) {
        slot = a0 + l;
        pieces = n;
      } else {
        first += n;
      }
    }
  }
  dep_wait();
  if (slot < 0 || first + pieces > k.room) return;
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= k.part_size) return;
  const float* src = k.partial + (int64_t)first * k.part_size + e;
  float s = src[0];
  for (int i = 1; i < pieces; ++i) s += src[(int64_t)i * k.part_size];
  const GradSide& p = (k.side[1].out && e >= k.side[1].part) ? k.side[1] : k.side[0];
  p.out[(int64_t)slot * k.a.max_rank * p.C + (e - p.part)] = s;
}

constexpr int kMaxColWarps = 4;

// Tokens per piece.  Pieces multiply the CTAs of the columns; each costs its
// partial sums once more through memory.  About four turns of two CTAs per SM
// even out the last turn.
int grad_piece(const LoraArgs& a) {
  const int64_t strips = (a.n + 127) / 128 + (a.rows + 127) / 128;
  const int64_t want = (8 * 148 + strips - 1) / strips;
  int64_t piece = (a.ntok + want - 1) / want;
  piece = (piece + kBlockTok - 1) / kBlockTok * kBlockTok;
  return (int)(piece < 512 ? 512 : piece);
}

template <class TA, class TB, int MR>
cudaError_t launch(const GradKernelArgs& k, cudaStream_t s) {
  auto kern = lora_grad_kernel<TA, TB, MR>;
  constexpr size_t stage = 2 * (kBlockTok / 16) * MR * 3 * 32 * sizeof(uint4);
  constexpr size_t sums = (size_t)kWarps * 16 * MR * 33 * sizeof(float);
  constexpr size_t smem = stage > sums ? stage : sums;
  cudaError_t e;
  if (smem > 48 * 1024 &&
      (e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) !=
          cudaSuccess)
    return e;
  const int64_t pieces = (k.a.ntok + k.piece - 1) / k.piece + k.a.n_slots;
  cudaLaunchConfig_t c = {};
  const int64_t ctas = pieces * (k.side[0].strips + k.side[1].strips);
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  c.gridDim = dim3((unsigned)ctas, (k.a.max_rank + 16 * MR - 1) / (16 * MR));
  c.blockDim = dim3(kWarps * 32);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  if ((e = cudaLaunchKernelEx(&c, kern, k)) != cudaSuccess) return e;
  note_launch();
  if (k.a.ntok > k.piece) {
    c.gridDim = dim3((unsigned)((k.part_size + 255) / 256), (unsigned)(k.a.ntok / k.piece));
    c.blockDim = dim3(256);
    c.dynamicSmemBytes = 0;
    if ((e = cudaLaunchKernelEx(&c, lora_grad_join_kernel, k)) != cudaSuccess) return e;
    note_launch();
  }
  return cudaSuccess;
}

template <class TA, class TB>
cudaError_t by_rank(const GradKernelArgs& k, cudaStream_t s) {
  return k.a.max_rank <= 16 ? launch<TA, TB, 1>(k, s) : launch<TA, TB, 4>(k, s);
}
template <class TA>
cudaError_t by_dy(const GradKernelArgs& k, int dy_bf16, cudaStream_t s) {
  return dy_bf16 ? by_rank<TA, bf16>(k, s) : by_rank<TA, float>(k, s);
}

}  // namespace

// A slot of several pieces has fewer than twice its tokens' share of them.
static int grad_room(const LoraArgs& a) {
  const int piece = grad_piece(a);
  return a.ntok <= piece ? 0 : (int)(2 * a.ntok / piece);
}

size_t lora_grad_workspace_bytes(const LoraArgs& a) {
  return (size_t)grad_room(a) * (size_t)a.max_rank * (a.n + a.rows) * sizeof(float);
}

cudaError_t launch_lora_grad(const LoraArgs& a, const GradArgs& g, void* ws, cudaStream_t s) {
  GradKernelArgs k = {};
  k.a = a;
  k.piece = grad_piece(a);
  k.partial = static_cast<float*>(ws);
  k.room = grad_room(a);
  int64_t part = 0;
  if (g.dA) {
    GradSide& d = k.side[0];
    const int esz = g.x_kind == 0 ? 2 : g.x_kind == 1 ? 4 : 1;
    d.f = g.v;
    d.ldf = g.ldv;
    d.scaled = 0;
    d.X = g.x;
    d.ldx = g.ldx;
    d.C = a.n;
    d.wc = kMaxColWarps;
    if (g.x_kind == 2) {
      d.xs = g.code_scales;
      d.group = g.code_group > 0 ? g.code_group : (int)a.n;
      // a CTA's columns stay within one group
      if (g.code_group > 0 && g.code_group < 32 * kMaxColWarps) d.wc = g.code_group / 32;
    }
    d.out = g.dA;
    d.ld_rank = a.n;
    d.ld_c = 1;
    d.part = part;
    d.strips = (int)((a.n + 32 * d.wc - 1) / (32 * d.wc));
    d.vec = rows_aligned(g.x, g.ldx, 0, esz, esz == 1 ? 8 : 16);
    part += (int64_t)a.max_rank * a.n;
  }
  if (g.dB) {
    GradSide& d = k.side[1];
    d.f = g.u;
    d.ldf = g.ldu;
    d.scaled = 1;
    d.X = g.dy;
    d.ldx = g.lddy;
    d.C = a.rows;
    d.wc = kMaxColWarps;
    d.out = g.dB;
    d.ld_rank = 1;
    d.ld_c = a.max_rank;
    d.part = part;
    d.strips = (int)((a.rows + 32 * d.wc - 1) / (32 * d.wc));
    d.vec = rows_aligned(g.dy, g.lddy, 0, g.dy_bf16 ? 2 : 4, 16);
    part += (int64_t)a.max_rank * a.rows;
  }
  k.part_size = part;
  switch (g.x_kind) {
    case 0: return by_dy<bf16>(k, g.dy_bf16, s);
    case 1: return by_dy<float>(k, g.dy_bf16, s);
    default: return by_dy<int8_t>(k, g.dy_bf16, s);
  }
}

}  // namespace gptq
