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
// sums the pieces in order.  This kernel serves fp32, codes whose groups are
// narrower than 128 columns, and rows that are not 16-byte aligned; the others
// go to lora_grad_codes.cu and lora_grad_tc.cu.  Measured: 1500 tokens, 2048 +
// 2056 fp32 columns at rank 16 25 us (6 products of bf16 parts for each one),
// waiting for the rows' loads (issue 15 %, DRAM 8 %).  Calls that give v, dA and
// dB: 8192 tokens at 11008 columns of codes and 4096 of bf16, rank 16, 294 us with
// groups of 32 and 240 with groups of 64; 4096 tokens at 4097 + 4099 bf16 columns
// 141 us at rank 16, 240 at rank 64.
#include <cuda_runtime.h>

#include "lora_grad.cuh"

namespace gptq {
namespace {

constexpr int kWarps = 8;
constexpr int kBlockTok = 128;  // tokens of f staged at a time

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

  float acc[MR][4][4];
#pragma unroll
  for (int i = 0; i < MR; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.f;

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
    // The matrix instruction cuts its fp32 sum off instead of rounding it, always
    // towards zero, so long sums would drift (by 1.4e-6 after 24 instructions):
    // the products of a step are summed by themselves, the small ones first, and
    // added with rounding.
#pragma unroll
    for (int i = 0; i < MR; ++i) {
      if (r0 + 16 * i >= rank) break;
      uint4 f[3];
#pragma unroll
      for (int x = 0; x < 3; ++x) f[x] = src[(i * 3 + x) * 32 + lane];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int x = 2; x >= 0; --x) {
          const uint32_t a[4] = {f[x].x, f[x].y, f[x].z, f[x].w};
#pragma unroll
          for (int d = NX - 1; d >= 0; --d)
            if (x + d <= 2) mma16816(t, a, b[j][0][d], b[j][1][d]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] += t[e];
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
  }
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
            acc[i][j][e];
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
    out[(r0 + r) * p.ld_rank + (int64_t)(cs + cc) * p.ld_c] = r0 + r < rank ? s : 0.f;
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
  const int64_t e0 = (int64_t)blockIdx.x * 1024 + threadIdx.x;
  const float* src = k.partial + (int64_t)first * k.part_size;
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int i = 0; i < pieces; ++i)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int64_t e = e0 + 256 * x;
      if (e < k.part_size) sum[x] += src[(int64_t)i * k.part_size + e];
    }
#pragma unroll
  for (int x = 0; x < 4; ++x) {
    const int64_t e = e0 + 256 * x;
    if (e >= k.part_size) break;
    const GradSide& p = (k.side[1].out && e >= k.side[1].part) ? k.side[1] : k.side[0];
    p.out[(int64_t)slot * k.a.max_rank * p.C + (e - p.part)] = sum[x];
  }
}

constexpr int kMaxColWarps = 4;

// Tokens per piece.  Pieces multiply the CTAs of the columns; each costs its
// partial sums once more through memory.  Of 1, 2, ... pieces of at most
// kGradTcPiece tokens the number that fills its turns of one CTA of 256 columns
// per SM (two of 128) best is taken, a further piece having to gain 2 % of a
// turn.
int grad_piece(const LoraArgs& a) {
  if (a.ntok < kBlockTok) return kBlockTok;
  const int64_t strips = (a.n + kGradTcCols - 1) / kGradTcCols +
                         (a.rows + kGradTcCols - 1) / kGradTcCols;
  const int64_t slots = num_sms();
  const int64_t least = (a.ntok + kGradTcPiece - 1) / kGradTcPiece;
  int64_t best = least;
  double top = -1.;
  for (int64_t n = least; n < least + 16 && (n == least || a.ntok / n >= 256); ++n) {
    const int64_t turns = (n * strips + slots - 1) / slots;
    const double fill = (double)(n * strips) / (double)(turns * slots) - 0.02 * (double)(n - least);
    if (fill > top) {
      top = fill;
      best = n;
    }
  }
  const int64_t piece = (a.ntok + best - 1) / best;
  return (int)((piece + kBlockTok - 1) / kBlockTok * kBlockTok);
}

template <class TA, class TB, int MR>
cudaError_t launch(const GradKernelArgs& k, int64_t ctas, cudaStream_t s) {
  auto kern = lora_grad_kernel<TA, TB, MR>;
  constexpr size_t stage = 2 * (kBlockTok / 16) * MR * 3 * 32 * sizeof(uint4);
  constexpr size_t sums = (size_t)kWarps * 16 * MR * 33 * sizeof(float);
  constexpr size_t smem = stage > sums ? stage : sums;
  cudaError_t e;
  if (smem > 48 * 1024 &&
      (e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem)) !=
          cudaSuccess)
    return e;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)ctas, (k.a.max_rank + 16 * MR - 1) / (16 * MR));
  c.blockDim = dim3(kWarps * 32);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = k.behind ? 1 : 0;
  e = cudaLaunchKernelEx(&c, kern, k);
  note_launch();
  return e;
}

template <class TA, class TB>
cudaError_t by_rank(const GradKernelArgs& k, int64_t ctas, cudaStream_t s) {
  return k.a.max_rank <= 16 ? launch<TA, TB, 1>(k, ctas, s) : launch<TA, TB, 4>(k, ctas, s);
}
template <class TA>
cudaError_t by_dy(const GradKernelArgs& k, int dy_bf16, int64_t ctas, cudaStream_t s) {
  return dy_bf16 ? by_rank<TA, bf16>(k, ctas, s) : by_rank<TA, float>(k, ctas, s);
}

cudaError_t join(const GradKernelArgs& k, cudaStream_t s) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)((k.part_size + 1023) / 1024), (unsigned)(k.a.ntok / k.piece));
  c.blockDim = dim3(256);
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&c, lora_grad_join_kernel, k);
  note_launch();
  return e;
}

}  // namespace

// A slot of several pieces has fewer than twice its tokens' share of them.
static int grad_room(const LoraArgs& a) {
  const int piece = grad_piece(a);
  return a.ntok <= piece ? 0 : (int)(2 * a.ntok / piece);
}

// [partial sums | parts of f]
static size_t partial_bytes(const LoraArgs& a) {
  return ((size_t)grad_room(a) * (size_t)a.max_rank * (a.n + a.rows) * sizeof(float) + 255) /
         256 * 256;
}
size_t lora_grad_workspace_bytes(const LoraArgs& a) {
  return partial_bytes(a) + (a.ntok >= kGradTcTokens ? lora_grad_parts_bytes(a) : 0);
}

cudaError_t launch_lora_grad(const LoraArgs& a, const GradArgs& g, void* ws, cudaStream_t s) {
  GradKernelArgs k = {};
  k.a = a;
  k.piece = grad_piece(a);
  k.partial = static_cast<float*>(ws);
  k.room = grad_room(a);
  k.behind = g.behind;
  k.gate = current_wait_gate();
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
    d.vec_f = rows_aligned(d.f, d.ldf, 0, 4, 16);
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
    d.vec_f = rows_aligned(d.f, d.ldf, 0, 4, 16);
    part += (int64_t)a.max_rank * a.rows;
  }
  k.part_size = part;
  const int64_t pieces = (a.ntok + k.piece - 1) / k.piece + a.n_slots;
  // bf16 rows and codes whose scale is one for 128 columns, all 16-byte aligned
  const bool tc =
      (!g.dA || (g.x_kind != 1 && k.side[0].wc == kMaxColWarps &&
                 rows_aligned(g.x, g.ldx, 0, g.x_kind == 0 ? 2 : 1, 16))) &&
      (!g.dB || (g.dy_bf16 && k.side[1].vec));
  cudaError_t e = cudaSuccess;
  if (tc) {
    // Beside codes, dB stays in their launch: together the two fill the SMs
    // (8192 tokens, 11008 and 4096 columns, rank 16: 79 us, apart 68 + 24).
    const bool split_first = a.ntok >= kGradTcTokens && !(g.dA && g.x_kind == 2);
    for (int i = 0; i < 2; ++i) {
      GradSide& d = k.side[i];
      if (!split_first || !d.strips) continue;
      d.strips = 0;
      d.tc_strips = (int)((d.C + kGradTcCols - 1) / kGradTcCols);
    }
    if (k.side[0].strips || k.side[1].strips)
      e = launch_lora_grad_codes(k, k.side[0].strips && g.x_kind == 2, pieces, s);
    if (e == cudaSuccess && (k.side[0].tc_strips || k.side[1].tc_strips))
      e = launch_lora_grad_tc(k, static_cast<char*>(ws) + partial_bytes(a), s);
  } else {
    const int64_t ctas = pieces * (k.side[0].strips + k.side[1].strips);
    if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
    e = g.x_kind == 0   ? by_dy<bf16>(k, g.dy_bf16, ctas, s)
        : g.x_kind == 1 ? by_dy<float>(k, g.dy_bf16, ctas, s)
                        : by_dy<int8_t>(k, g.dy_bf16, ctas, s);
  }
  if (e != cudaSuccess || a.ntok <= k.piece) return e;
  return join(k, s);
}

}  // namespace gptq
