// The adapters' gradients on tcgen05 from 8-bit codes of x, and from few tokens
// of bf16 X: out(i, c) = sum over a slot's tokens of f[t][i] X[t][c].
//
// As in lora_grad_tc.cu, columns of X (128 a CTA) are the M of tcgen05.mma, the
// 3 RP rank parts of f its N, 64 tokens a stage its K.  Codes bring two
// things that keep threads at work: they are copied raw and widened to bf16
// (exactly) into the operand tile, and their scale belongs to a token and a
// group of columns, so it is multiplied onto f, which is split into its parts
// per CTA (a CTA's columns never leave a group).  For few tokens of bf16 the
// splitting in place saves a launch.
//
// Warps: 0-7 widen codes (bf16: split f) and drain, 8-11 copy (codes: and split
// f), 12 issues the instructions.  Two CTAs share an SM.  Measured: 77 us for
// both products of 8192 tokens at 11008 (codes) and 4096 (bf16 dy) columns and
// rank 16, 2.0 TB/s.  A stage of a CTA takes 2000 to 2700 cycles.  What it
// spends them on are threads, not memory: about 1700 warp instructions, and
// some 600 cycles of shared memory to write, read, widen and multiply 8 KB of
// codes; the copies are always there in time.
#include <cuda_runtime.h>

#include "lora_grad.cuh"
#include "sm100_ptx.cuh"

namespace gptq {
namespace {

constexpr int kWork = 256;           // threads of warps 0-7
constexpr int kCopy = 128;           // threads of warps 8-11
constexpr int kMmaWarp = (kWork + kCopy) / 32;
constexpr int kAll = kWork + kCopy + 32;
constexpr int kTok = 64;             // tokens per stage
constexpr int kCols = 128;           // columns of X per CTA
constexpr int kATile = kTok * kCols * 2;
constexpr int kRaw = kTok * kCols;   // codes of a stage
constexpr int kFlush = 8;            // stages between drains of TMEM

// Ring sizes: with the operand tiles of f, two CTAs fit an SM's shared memory.
template <class TX, int RP>
struct Plan {
  static constexpr bool kCodes = sizeof(TX) == 1;
  static constexpr int N = 3 * RP;
  static constexpr int kBTile = N * kTok * 2;
  static constexpr int kBPart = RP * kTok * 2;  // rows of RP ranks, swizzled over their width
  // tiles of X (of raw codes): as many as fit beside the tiles of f
  static constexpr int kARing = kCodes ? 2 : RP == 16 ? 5 : RP == 32 ? 4 : 3;
  static constexpr int kRawRing = !kCodes ? 0 : RP == 16 ? 5 : RP == 32 ? 4 : 2;
  static constexpr int kXRing = kCodes ? kRawRing : kARing;
  static constexpr int kXBytes = kCodes ? kRaw : kATile;
  static constexpr int kAhead = kXRing - 1;  // stages whose cp.async copies are under way
  static constexpr int kOffB = kARing * kATile;
  static constexpr int kOffRaw = kOffB + 2 * kBTile;
  static constexpr int kOffTok = kOffRaw + kRawRing * kRaw;
  static constexpr int kOffMul = kOffTok + kGradTcPiece * 4;
  static constexpr int kOffBar = kOffMul + kGradTcPiece * 4;
  static constexpr int kSmem = kOffBar + 128;
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs per SM");
};

// A operand, M contiguous: 64 columns of a token are 128 swizzled bytes, 8
// tokens 1024; the other 64 columns lie kATile / 2 further.  B operand, N
// contiguous: a block of RP ranks per part, rows of 2 RP bytes under the swizzle
// of that width, 8 tokens one after the other, the next part kBPart further.
// byte offset of 8 ranks of a token within a part's block
template <int RP>
__device__ __forceinline__ int n_major_at(int tok, int chunk) {
  const int x = RP == 64 ? tok & 7 : RP == 32 ? (tok >> 1) & 3 : (tok >> 2) & 1;
  return tok * (2 * RP) + ((chunk ^ x) << 4);
}
__host__ __device__ constexpr uint32_t idesc_mn_major(int N) {
  return ptx::idesc_bf16_f32(kCols, N) | (1u << 15) | (1u << 16);
}

template <class TX, int RP>
__device__ __forceinline__ void grad_body(const GradKernelArgs& k, const GradSide& p,
                                             const CUtensorMap* map, const Piece& pc, int strip,
                                             int r0, char* smem) {
  using L = Plan<TX, RP>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = ptx::smem_u32(smem);
  int* toks = reinterpret_cast<int*>(smem + L::kOffTok);
  float* mul = reinterpret_cast<float*>(smem + L::kOffMul);
  uint64_t* ready = reinterpret_cast<uint64_t*>(smem + L::kOffBar);  // threads' tiles are there
  uint64_t* done = ready + 2;       // the stage's instructions are
  uint64_t* xfull = done + 2;       // X's tile (the raw codes) is there
  uint64_t* xfree = xfull + 5;      // ... and has been used
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(xfree + 5);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int C = (int)p.C, cs = strip * kCols;
  const int rank = lora_rank(k.a, pc.slot);
  const int count = r0 < rank ? pc.count : 0;
  const int stages = (count + kTok - 1) / kTok;
  if (warp == 0) {
    ptx::tmem_alloc(tmem_slot, 256);
    ptx::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&ready[i], L::kCodes ? kWork + kCopy : kWork);
      ptx::mbar_init(&done[i], 1);
    }
    for (int i = 0; i < L::kXRing; ++i) {
      ptx::mbar_init(&xfull[i], kCopy);
      ptx::mbar_init(&xfree[i], L::kCodes ? kWork : 1);
    }
    ptx::fence_mbar_init();
    *abort = 0;
  }
  {
    const float sc = p.scaled ? lora_scale(k.a, pc.slot) : 1.f;
    const int64_t G = p.xs ? (p.C + p.group - 1) / p.group : 0;
    const int grp = p.xs ? cs / p.group : 0;
    // all the loads of a thread at once: first the tokens, then their scales
    constexpr int kEach = kGradTcPiece / kWork;
    if (tid < kWork) {
      int t[kEach];
      float m[kEach];
#pragma unroll
      for (int x = 0; x < kEach; ++x) {
        const int i = tid + x * kWork;
        t[x] = i < count ? piece_token(k.a, pc, i) : -1;
      }
#pragma unroll
      for (int x = 0; x < kEach; ++x)
        m[x] = p.xs && t[x] >= 0 ? p.xs[(int64_t)t[x] * G + grp] : 1.f;
#pragma unroll
      for (int x = 0; x < kEach; ++x) {
        const int i = tid + x * kWork;
        if (i < stages * kTok) {
          toks[i] = t[x];
          mul[i] = t[x] < 0 ? 0.f : sc * m[x];
        }
      }
    }
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // f of a stage: units of one token and 8 ranks
  constexpr int kChunks = RP / 8;
  constexpr int kUnits = kTok * kChunks;
  constexpr int kSplitters = L::kCodes ? kCopy : kWork;
  constexpr int kPer = (kUnits + kSplitters - 1) / kSplitters;
  const int ftid = L::kCodes ? tid - kWork : tid;
  float fv[kPer][8];
  auto load_f = [&](int s) {
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
      const int e = ftid + x * kSplitters;
      if (kUnits % kSplitters != 0 && e >= kUnits) break;
      const int r = r0 + 8 * (e % kChunks), t = toks[s * kTok + e / kChunks];
      const int left = t >= 0 ? rank - r : 0;
      const float* f = p.f + (int64_t)max(t, 0) * p.ldf + r;
      if (left >= 8 && p.vec_f) {
        const float4 lo = reinterpret_cast<const float4*>(f)[0];
        const float4 hi = reinterpret_cast<const float4*>(f)[1];
        fv[x][0] = lo.x, fv[x][1] = lo.y, fv[x][2] = lo.z, fv[x][3] = lo.w;
        fv[x][4] = hi.x, fv[x][5] = hi.y, fv[x][6] = hi.z, fv[x][7] = hi.w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) fv[x][i] = i < left ? f[i] : 0.f;
      }
    }
  };
  auto split_f = [&](int s) {
    char* dst = smem + L::kOffB + (s & 1) * L::kBTile;
#pragma unroll
    for (int x = 0; x < kPer; ++x) {
      const int e = ftid + x * kSplitters;
      if (kUnits % kSplitters != 0 && e >= kUnits) break;
      const int tok = e / kChunks;
      const float m = mul[s * kTok + tok];
      uint32_t w[3][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t q[3];
        split_pair<3>(fv[x][2 * i] * m, fv[x][2 * i + 1] * m, q);
#pragma unroll
        for (int c = 0; c < 3; ++c) w[c][i] = q[c];
      }
      char* d = dst + n_major_at<RP>(tok, e % kChunks);
#pragma unroll
      for (int c = 0; c < 3; ++c)
        *reinterpret_cast<uint4*>(d + c * L::kBPart) =
            make_uint4(w[c][0], w[c][1], w[c][2], w[c][3]);
    }
  };
  // 8-bit codes of a stage into the operand tile
  auto widen = [&](int s) {
    const char* src = smem + L::kOffRaw + (s % (L::kCodes ? L::kRawRing : 1)) * kRaw;
    char* dst = smem + (s & 1) * kATile;
    const int j = tid & 7;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = (tid >> 3) + 32 * i;
      const uint4 v = *reinterpret_cast<const uint4*>(src + row * 128 + (j << 4));
      const Codes8 lo = {{v.x, v.y}}, hi = {{v.z, v.w}};
      uint32_t o[8];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        uint32_t q[1];
        row_pair(lo, x, q);
        o[x] = q[0];
        row_pair(hi, x, q);
        o[4 + x] = q[0];
      }
      char* d = dst + (j >> 2) * (kATile / 2) + row * 128;
      // (the two halves of the columns in opposite order: 8 lanes, 8 bank groups)
      const int c = (2 * j) & 7, f = j >> 2;
      const uint4 v0 = make_uint4(o[0], o[1], o[2], o[3]), v1 = make_uint4(o[4], o[5], o[6], o[7]);
      *reinterpret_cast<uint4*>(d + (((c + f) ^ (row & 7)) << 4)) = f ? v1 : v0;
      *reinterpret_cast<uint4*>(d + (((c + 1 - f) ^ (row & 7)) << 4)) = f ? v0 : v1;
    }
  };
  // every wait has a limit; a CTA that met it gives NaN instead of sums
  bool bad = false;
  auto wait = [&](uint64_t* bars, int ring, int s) {
    if (!ptx::mbar_wait_bounded(&bars[s % ring], (s / ring) & 1, abort, k.gate.limit_ns)) {
      *abort = 1;
      bad = true;
    }
  };
  // totals: lane = column 32 (warp % 4) + lane, ranks RP / 2 (warp / 4) ..
  constexpr int kHalf = RP / 2;
  float total[kHalf];
#pragma unroll
  for (int i = 0; i < kHalf; ++i) total[i] = 0.f;
  auto drain = [&]() {
    ptx::tc_fence_after();
    const uint32_t at = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + (warp >> 2) * kHalf;
#pragma unroll
    for (int i = 0; i < kHalf; i += 8) {
      uint32_t v[3][8];
#pragma unroll
      for (int c = 0; c < 3; ++c) ptx::tmem_ld_32x32b_x8(at + c * RP + i, v[c]);
      ptx::tmem_ld_wait();
#pragma unroll
      for (int x = 0; x < 8; ++x)
        total[i + x] += (__uint_as_float(v[2][x]) + __uint_as_float(v[1][x])) +
                        __uint_as_float(v[0][x]);
    }
    ptx::tc_fence_before();
  };

  if (tid >= kWork && warp != kMmaWarp) {
    const int ctid = tid - kWork;
    // 16 bytes of a row a thread: 16 (codes: 8) threads side by side
    constexpr int kAcross = L::kXBytes / kTok / 16, kDown = kCopy / kAcross;
    constexpr int kEl = 16 / (int)sizeof(TX);
    const int j = ctid % kAcross, row0 = ctid / kAcross;
    const int left = (C - cs - kEl * j) * (int)sizeof(TX);
    const int bytes = left < 0 ? 0 : left > 16 ? 16 : left;
    const TX* X = static_cast<const TX*>(p.X) + (bytes > 0 ? cs + kEl * j : 0);
    uint32_t late = 0;  // bit i: the stage i iterations ago was copied by cp.async
    auto finish = [&](int s) {  // the copies of stage s are there
      ptx::cp_async_wait<L::kAhead>();
      if (s >= 0 && (late >> L::kAhead & 1)) {
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(&xfull[s % L::kXRing]);
      }
    };
    if (L::kCodes && stages > 0) load_f(0);
    if (ctid == 0 && !ptx::gate_wait_bounded(k.gate.gate, k.gate.limit_ns)) {
      *abort = 1;
      bad = true;
    }
    bad = __any_sync(~0u, bad);
    int s = 0;
    for (; s < stages + L::kAhead && !bad; ++s) {
      late <<= 1;
      if (s < stages) {
        if (s >= L::kXRing) wait(xfree, L::kXRing, s - L::kXRing);
        if ((bad = __any_sync(~0u, bad))) break;
        const int* t = toks + s * kTok;
        uint64_t* bar = &xfull[s % L::kXRing];
        const uint32_t dst =
            base + (L::kCodes ? L::kOffRaw : 0) + (s % L::kXRing) * L::kXBytes;
        if (run_of_64(t)) {
          if (ctid == 0) {
            ptx::mbar_arrive_expect_tx(bar, L::kXBytes);
            ptx::tma_load_2d(smem + (dst - base), map, bar, cs, t[0]);
            if (!L::kCodes) ptx::tma_load_2d(smem + (dst - base) + kATile / 2, map, bar, cs + 64, t[0]);
          } else {
            ptx::mbar_arrive(bar);
          }
        } else {
          late |= 1;
#pragma unroll
          for (int i = 0; i < kTok / kDown; ++i) {
            const int r = row0 + kDown * i;
            const int tok = t[r];
            const bool on = tok >= 0 && bytes > 0;
            const uint32_t at = L::kCodes ? r * kCols + (j << 4)
                                          : (j >> 3) * (kATile / 2) + r * 128 +
                                                (((j & 7) ^ (r & 7)) << 4);
            copy16(dst + at, X + (on ? (int64_t)tok * p.ldx : 0), on ? bytes : 0);
          }
        }
      }
      ptx::cp_async_commit();
      finish(s - L::kAhead);
      const int sf = s - L::kAhead;  // f of the stage whose copies are there
      if (L::kCodes && sf >= 0) {
        if (sf >= 2) wait(done, 2, sf - 2);  // the tile of f is free
        if ((bad = __any_sync(~0u, bad))) break;
        split_f(sf);
        if (sf + 1 < stages) load_f(sf + 1);
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(&ready[sf & 1]);
      }
    }
    ptx::cp_async_wait_all();
    // on an early end: wait for the boxes that are under way
    if (bad && ctid == 0) {
      const volatile int never = 0;
      for (int i = max(0, s - L::kXRing); i < min(s, stages); ++i)
        ptx::mbar_wait_bounded(&xfull[i % L::kXRing], (i / L::kXRing) & 1, &never, k.gate.limit_ns);
    }
  } else if (warp == kMmaWarp) {
    if (lane == 0) {
      int s = 0;
      for (; s < stages; ++s) {
        if (!L::kCodes) wait(xfull, L::kXRing, s);
        wait(ready, 2, s);
        if (bad) break;
        ptx::tc_fence_after();
        const uint32_t a = base + (s % L::kARing) * kATile;
        const uint32_t b = base + L::kOffB + (s & 1) * L::kBTile;
        const uint64_t da = ptx::smem_desc_rows(a, 128, kATile / 2);
        const uint64_t db = ptx::smem_desc_rows(b, 2 * RP, L::kBPart);
#pragma unroll
        for (int i = 0; i < kTok / 16; ++i)
          // 16 tokens on: 16 rows of either operand
          ptx::mma_bf16(tmem, da + i * (2048 >> 4), db + i * ((32 * RP) >> 4),
                        idesc_mn_major(L::N), (s % kFlush) | i);
        ptx::mma_commit(&done[s & 1]);
        if (!L::kCodes) ptx::mma_commit(&xfree[s % L::kXRing]);
      }
      // on an early end: TMEM is not given back under instructions that are under way
      const volatile int never = 0;
      if (bad && s > 0)
        ptx::mbar_wait_bounded(&done[(s - 1) & 1], ((s - 1) >> 1) & 1, &never, k.gate.limit_ns);
    }
  } else {
    if (!L::kCodes && stages > 0) load_f(0);
    for (int s = 0; s < stages; ++s) {
      // (lanes may learn of a timeout at different waits, and draining TMEM takes
      // whole warps: all leave, or none)
      if (s >= 2) wait(done, 2, s - 2);  // the tiles of f and of widened codes are free
      if ((bad = __any_sync(~0u, bad))) break;
      if (!L::kCodes) {
        split_f(s);
        if (s + 1 < stages) load_f(s + 1);
      } else {
        wait(xfull, L::kXRing, s);
        if ((bad = __any_sync(~0u, bad))) break;
        widen(s);
        ptx::mbar_arrive(&xfree[s % L::kXRing]);
      }
      ptx::fence_proxy_async_smem();
      ptx::mbar_arrive(&ready[s & 1]);
      if (s % kFlush == kFlush - 1 || s == stages - 1) {
        wait(done, 2, s);
        if ((bad = __any_sync(~0u, bad))) break;
        drain();  // before the next arrival, hence before the next instruction
      }
    }
  }
  __syncwarp();
  bad = __syncthreads_or(bad);
  if (warp == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 256);
  }
  if (tid >= kWork) return;
  const int c = cs + 32 * (warp & 3) + lane;
  if (c < C) store_column<kHalf>(k, p, pc, c, r0 + (warp >> 2) * kHalf, rank, total, bad);
}

template <class TA, int RP>
__global__ void __launch_bounds__(kAll, 2)
    lora_grad_codes_kernel(const GradKernelArgs k, const __grid_constant__ CUtensorMap map_a,
                        const __grid_constant__ CUtensorMap map_b) {
  extern __shared__ __align__(1024) char smem[];
  dep_launch();
  const int strips = k.side[0].strips + k.side[1].strips;
  const Piece pc = find_piece(k.a, blockIdx.x / strips, k.piece, 1);
  dep_wait();
  if (pc.slot < 0) return;
  const int s = blockIdx.x % strips;
  if (s < k.side[0].strips)
    grad_body<TA, RP>(k, k.side[0], &map_a, pc, s, blockIdx.y * RP, smem);
  else
    grad_body<bf16, RP>(k, k.side[1], &map_b, pc, s - k.side[0].strips, blockIdx.y * RP,
                           smem);
}

template <class TA, int RP>
cudaError_t launch(const GradKernelArgs& k, int64_t ctas, cudaStream_t s) {
  auto kern = lora_grad_codes_kernel<TA, RP>;
  constexpr int sa = Plan<TA, RP>::kSmem, sb = Plan<bf16, RP>::kSmem;
  constexpr int smem = sa > sb ? sa : sb;
  static std::atomic<uint64_t> raised{0};
  cudaError_t e =
      raise_limits(reinterpret_cast<const void*>(kern), smem, false, raised);
  if (e != cudaSuccess) return e;
  // (a product that is not asked for has no strips and no map)
  CUtensorMap map[2] = {};
  for (int i = 0; i < 2; ++i) {
    const GradSide& d = k.side[i];
    const int esz = i == 0 ? (int)sizeof(TA) : 2;
    if (d.strips && !make_tma_rows(&map[i], d.X, esz, 0, k.a.ntok, d.C, 0, d.ldx,
                                   esz == 1 ? kCols : kCols / 2, kTok, esz == 1 ? 0 : 128))
      return cudaErrorInvalidValue;
  }
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)ctas, (k.a.max_rank + RP - 1) / RP);
  c.blockDim = dim3(kAll);
  c.dynamicSmemBytes = smem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = k.behind ? 1 : 0;
  e = cudaLaunchKernelEx(&c, kern, k, map[0], map[1]);
  note_launch();
  return e;
}

}  // namespace

cudaError_t launch_lora_grad_codes(const GradKernelArgs& k, bool codes, int64_t pieces,
                                   cudaStream_t s) {
  const int64_t ctas = pieces * (k.side[0].strips + k.side[1].strips);
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  const int r = k.a.max_rank;
  if (codes)
    return r <= 16   ? launch<int8_t, 16>(k, ctas, s)
           : r <= 32 ? launch<int8_t, 32>(k, ctas, s)
                     : launch<int8_t, 64>(k, ctas, s);
  return r <= 16   ? launch<bf16, 16>(k, ctas, s)
         : r <= 32 ? launch<bf16, 32>(k, ctas, s)
                   : launch<bf16, 64>(k, ctas, s);
}

}  // namespace gptq
