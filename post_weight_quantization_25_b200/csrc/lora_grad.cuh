// What the gradient kernels share: the description of a launch, the reading of
// 8 columns of a token, and the writing of a column's sums.
#pragma once
#include "lora_mma.cuh"

namespace gptq {

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
  int tc_strips;          // ... of the kernel for many tokens; 0: not its product
  int wc;                 // warps side by side in the columns
  int vec;
  int vec_f;              // f's rows are 16-byte aligned
};

struct GradKernelArgs {
  LoraArgs a;
  GradSide side[2];
  int piece;           // tokens per piece, a multiple of 128
  float* partial;      // [piece of a slot of several][part_size]
  int64_t part_size;
  int behind;          // the first launch is right behind a kernel of the same call
  int room;            // pieces that partial holds: enough for any real plan,
                       // checked for one that is not (slot_start not ascending)
  WaitGate gate;       // test gate and time limit of the tcgen05 kernels' waits
};

// Tokens of a piece of the tcgen05 kernels, at most
constexpr int kGradTcPiece = 2048;
// Few tokens, and 8-bit codes: f is split in the kernel (sides with strips).
cudaError_t launch_lora_grad_codes(const GradKernelArgs& k, bool codes, int64_t pieces,
                                   cudaStream_t s);
// Many tokens of bf16 X (sides with tc_strips): f is split beforehand, into
// `ws` of lora_grad_parts_bytes.
constexpr int kGradTcCols = 256;
// From this many tokens on.  4096 + 4096 columns, us beforehand / in the kernel:
// 1024 tokens at rank 16 18.7 / 18.6, rank 64 23.6 / 26.2; 4096 tokens 33.6 /
// 31.8 and 44.8 / 51.8: it pays with the rank, and from here on never loses much.
constexpr int kGradTcTokens = 1024;
size_t lora_grad_parts_bytes(const LoraArgs& a);
cudaError_t launch_lora_grad_tc(const GradKernelArgs& k, void* ws, cudaStream_t s);

namespace {

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

// Whole warps: whether 64 tokens are all there and consecutive rows.
__device__ __forceinline__ bool run_of_64(const int* toks) {
  const int lane = threadIdx.x & 31;
  const int a = toks[2 * lane], b = toks[2 * lane + 1], c = toks[min(2 * lane + 2, 63)];
  return __all_sync(~0u, a >= 0 && b == a + 1 && (lane == 31 || c == b + 1));
}

// R sums of column c, ranks r0 .., to the gradient or to the piece's partial
// sums; zeros from the slot's rank on.
template <int R>
__device__ __forceinline__ void store_column(const GradKernelArgs& k, const GradSide& p,
                                             const Piece& pc, int c, int r0, int rank,
                                             const float (&total)[R], bool bad) {
  const bool whole = pc.pieces == 1;
  if (!whole && pc.multi + pc.index >= k.room) return;
  float* out = whole ? p.out + (int64_t)pc.slot * k.a.max_rank * p.C
                     : k.partial + (int64_t)(pc.multi + pc.index) * k.part_size + p.part;
  float v[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    v[i] = r0 + i >= rank ? 0.f : bad ? __uint_as_float(0x7fffffffu) : total[i];
  if (p.ld_rank == 1 && (k.a.max_rank & 3) == 0 &&
      (reinterpret_cast<uintptr_t>(out) & 15) == 0) {  // dB: a thread's ranks are one stretch
    float* o = out + (int64_t)c * p.ld_c + r0;
#pragma unroll
    for (int i = 0; i < R; i += 4)
      if (r0 + i < k.a.max_rank)
        *reinterpret_cast<float4*>(o + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    return;
  }
#pragma unroll
  for (int i = 0; i < R; ++i)
    if (r0 + i < k.a.max_rank) out[(r0 + i) * p.ld_rank + (int64_t)c * p.ld_c] = v[i];
}

}  // namespace
}  // namespace gptq
