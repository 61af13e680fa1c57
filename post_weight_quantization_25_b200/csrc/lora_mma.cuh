// Building blocks of the adapter kernels: warp-level bf16 matrix
// instructions, fp32 values as sums of bf16 parts, row loads, and the search
// for a task's piece of the token plan.
//
// fp32 accuracy on bf16 matrix instructions.  An fp32 value has 24 significant
// bits, a bf16 value 8, so v = p0 + p1 + p2 exactly when each part takes the
// leading 8 bits of what is left (cutting off, not rounding: the next part
// has the same sign and the last one is exact).  So p1 is below 2^-7 and p2
// below 2^-15 of the value.  A product of two values is the sum of the part
// products; those with part numbers adding up to 3 or more are left out, p1 p2
// twice and p2 p2: less than 2^-21 of the product together, 2^-23 on average,
// and always with its sign.  bf16 values are their own single part, so products
// of bf16 data cost one instruction and are exact.
#pragma once
#include <cstdint>

#include "lora_internal.cuh"

namespace gptq {
namespace {

using bf16 = __nv_bfloat16;

// D += A B: A 16 x 16 (rows g, g + 8; column pairs 2q, 2q + 8), B 16 x 8
// (row pairs 2q, 2q + 8; column g), D fp32 (rows g, g + 8; columns 2q, 2q + 1)
// with g = lane / 4, q = lane % 4.
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Transposes an 8 x 8 matrix of 16-bit elements spread over the warp (lane
// holds row lane / 4, columns 2 (lane % 4) and the next).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

// bf16 parts that hold a value of type T exactly
template <class T>
struct Parts { static constexpr int n = 1; };
template <>
struct Parts<float> { static constexpr int n = 3; };

// (a, b) as N packed pairs of bf16 parts, a in the low half.  N = 3: exact.
// N = 2 (for bf16 results): both parts rounded to nearest, off by 2^-17.
template <int N>
__device__ __forceinline__ void split_pair(float a, float b, uint32_t (&p)[N]) {
  if (N == 3) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
      p[i] = __byte_perm(ua, ub, 0x7632);
      if (i + 1 < N) {
        a -= __uint_as_float(ua & 0xffff0000u);
        b -= __uint_as_float(ub & 0xffff0000u);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
      p[i] = *reinterpret_cast<const uint32_t*>(&h);
      if (i + 1 < N) {
        a -= __uint_as_float(p[i] << 16);
        b -= __uint_as_float(p[i] & 0xffff0000u);
      }
    }
  }
}

// E consecutive elements of a row, kept as loaded (bf16 pairs or floats)
template <class T, int E>
struct Raw;
template <int E>
struct Raw<bf16, E> { uint32_t w[E / 2]; };
template <int E>
struct Raw<float, E> { float w[E]; };

template <class T, int E>
__device__ __forceinline__ void raw_zero(Raw<T, E>& r) {
#pragma unroll
  for (int i = 0; i < (int)(sizeof(r.w) / 4); ++i) r.w[i] = 0;
}

// RO: memory that nothing writes while the kernel runs (read-only path)
template <bool RO, class V>
__device__ __forceinline__ V ld(const V* p) {
  if constexpr (RO) return __ldg(p);
  return *p;
}

// The first `valid` (any integer) of E elements at p, zeros for the others.
// vec: p is aligned to E elements (at most 16 bytes), so that all E load at
// once.  Nothing outside the valid elements is read.
template <bool RO = true, class T, int E>
__device__ __forceinline__ void raw_load(Raw<T, E>& r, const T* p, int valid, bool vec) {
  if (valid >= E && vec) {
    constexpr int bytes = E * (int)sizeof(T);
    if constexpr (bytes == 8) {
      const uint2 v = ld<RO>(reinterpret_cast<const uint2*>(p));
      memcpy(r.w, &v, 8);
    } else {
#pragma unroll
      for (int i = 0; i < bytes / 16; ++i) {
        const uint4 v = ld<RO>(reinterpret_cast<const uint4*>(p) + i);
        memcpy(r.w + 4 * i, &v, 16);
      }
    }
  } else {
    raw_zero(r);
    if constexpr (sizeof(T) == 2) {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (i < valid) r.w[i / 2] |= (uint32_t)ld<RO>(h + i) << (16 * (i & 1));
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (i < valid) r.w[i] = ld<RO>(reinterpret_cast<const float*>(p) + i);
    }
  }
}

// E aligned elements
template <bool RO, class T, int E>
__device__ __forceinline__ void raw_fetch(Raw<T, E>& r, const T* p) {
  constexpr int bytes = E * (int)sizeof(T);
  if constexpr (bytes == 8) {
    const uint2 v = ld<RO>(reinterpret_cast<const uint2*>(p));
    memcpy(r.w, &v, 8);
  } else {
    const uint4 v = ld<RO>(reinterpret_cast<const uint4*>(p));
    memcpy(r.w, &v, 16);
  }
}
// Zeros behind the first `valid` of 4 elements
template <class T>
__device__ __forceinline__ void raw_keep(Raw<T, 4>& r, int valid) {
  if constexpr (sizeof(T) == 2) {
    r.w[0] &= valid > 1 ? 0xffffffffu : valid > 0 ? 0x0000ffffu : 0u;
    r.w[1] &= valid > 3 ? 0xffffffffu : valid > 2 ? 0x0000ffffu : 0u;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i >= valid) r.w[i] = 0.f;
  }
}

// raw_load where `there` elements of the row may be read but only the first
// `valid` count: one load and a mask instead of one load per element.
template <class T>
__device__ __forceinline__ void raw_load_part(Raw<T, 4>& r, const T* p, int valid, int there,
                                              bool vec) {
  if (valid >= 4 || valid <= 0 || there < 4 || !vec) {
    raw_load(r, p, valid, vec);
    return;
  }
  raw_load(r, p, 4, true);
  raw_keep(r, valid);
}

// Pair i of the elements as packed parts
template <int E>
__device__ __forceinline__ void raw_pair(const Raw<bf16, E>& r, int i, uint32_t (&p)[1]) {
  p[0] = r.w[i];
}
template <int E>
__device__ __forceinline__ void raw_pair(const Raw<float, E>& r, int i, uint32_t (&p)[3]) {
  split_pair<3>(r.w[2 * i], r.w[2 * i + 1], p);
}

// 16 bytes global -> shared, the first `bytes` of them read, zeros behind
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}

// ---------------------------------------------------------------- the plan
// Piece `idx` of the plan, every slot's tokens cut into pieces of `size` (a
// slot without tokens has min_pieces).  Called by whole warps.
struct Piece {
  int slot;    // -1: there is no such piece
  int first;   // position of the piece's first token in `order`
  int count;   // its tokens (0..size)
  int index;   // its number within the slot
  int pieces;  // the slot's pieces
  int multi;   // pieces of earlier slots that have more than one
};

__device__ __forceinline__ Piece find_piece(const LoraArgs& p, int idx, int size, int min_pieces) {
  const int lane = threadIdx.x & 31;
  int before = 0, multi = 0;
  for (int a0 = 0; a0 < p.n_slots; a0 += 32) {
    const int a = a0 + lane;
    int s0 = 0, s1 = 0, pcs = 0;
    if (a < p.n_slots) {
      s0 = lora_start(p, a);
      s1 = max(lora_start(p, a + 1), s0);
      pcs = max((s1 - s0 + size - 1) / size, min_pieces);
    }
    int sum = pcs, msum = pcs > 1 ? pcs : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(~0u, sum, o), m = __shfl_up_sync(~0u, msum, o);
      if (lane >= o) {
        sum += u;
        msum += m;
      }
    }
    const unsigned hit = __ballot_sync(~0u, before + sum > idx);
    if (hit) {
      const int l = __ffs(hit) - 1;
      Piece r;
      const int mine = before + sum - pcs;  // pieces before slot a
      r.slot = a0 + l;
      r.pieces = __shfl_sync(~0u, pcs, l);
      r.index = idx - __shfl_sync(~0u, mine, l);
      const int start = __shfl_sync(~0u, s0, l), end = __shfl_sync(~0u, s1, l);
      r.first = start + r.index * size;
      r.count = min(size, end - r.first);
      r.multi = multi + __shfl_sync(~0u, msum - (pcs > 1 ? pcs : 0), l);
      return r;
    }
    before += __shfl_sync(~0u, sum, 31);
    multi += __shfl_sync(~0u, msum, 31);
  }
  return {-1, 0, 0, 0, 0, 0};
}

// Token at position first + i of a piece, or -1
__device__ __forceinline__ int piece_token(const LoraArgs& p, const Piece& pc, int i) {
  if (i >= pc.count) return -1;
  const int t = p.order[pc.first + i];
  return (t >= 0 && t < p.ntok) ? t : -1;
}

// Whole warps, lane i the i-th of 32 tokens (-1: none): whether a box of 32 rows
// from the first token's on brings them all, with few rows to spare.
__device__ __forceinline__ bool row_run(int t) {
  const int first = __shfl_sync(~0u, t, 0), lane = threadIdx.x & 31;
  const unsigned there = __ballot_sync(~0u, t >= 0);
  const bool fits = __all_sync(~0u, t < 0 || t == first + lane);
  return first >= 0 && fits && __popc(there) >= 24;
}

// ---------------------------------------------------------------- dependent launches
// The first kernel of a call is launched as any other; those behind it with
// programmatic stream serialization: they may start while the one before still
// runs, read what no kernel of the call writes before they do (the caller's
// earlier work is done, or the first kernel would not have started), and call
// dep_wait() before anything else.  Every CTA calls it, so a kernel never ends
// before its predecessors.
__device__ __forceinline__ void dep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void dep_launch() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

}  // namespace
}  // namespace gptq
