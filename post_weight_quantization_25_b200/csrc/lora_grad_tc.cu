// The adapters' gradients on tcgen05 for many tokens of bf16 X (x or dy):
// out(i, c) = sum over a slot's tokens of f[t][i] X[t][c].
//
// What the warp-level kernel (lora_grad.cu) lacks is matrix throughput: f is
// fp32 and enters as 3 exact bf16 parts, so rank 64 costs 192 products for
// every element of X, more than twice the time that mma.sync has while X
// streams in.  Here 128 columns of X are the M of tcgen05.mma, the 3 RP rank
// parts its N (48, 96 or 192) and 64 tokens a stage its K:
//
//  * X's rows go to shared memory as they are ([token][column], 128-byte
//    swizzle), which is an A operand whose M axis is contiguous.  64 tokens in
//    a row are one TMA box per 64 columns; other tokens' rows are copied by
//    16-byte cp.async with the swizzle applied by hand (TMA's gather of 4 rows
//    takes about 80 cycles to issue: 2600 for 128 columns of a stage).
//  * f is split once for all columns by a kernel of its own, in the plan's
//    order, so a stage of it is one box, [part][token][rank].
//  * The sums of the parts lie in separate TMEM columns of the same lane, so
//    a thread adds the three parts of its column of X when it reads them.
//
// A CTA takes 256 columns, two products that share f's box, because f is read
// again for every strip of columns: at rank 64 a stage of f is 24 KB beside
// 32 KB of X.  The tensor core cuts its fp32 sums off instead of rounding
// them, so TMEM is emptied into rounded register totals every 512 tokens (32
// instructions).  One CTA per SM, 110 to 190 KB of it under way.  Measured at
// rank 64 and 4096 tokens, 4096 + 11008 columns: 40 us for 124 MB of X, and f's
// boxes (56 KB for 32 KB of X) from L2 beside them.  Nothing is at its limit:
// DRAM 37 %, L2 26 %, the tensor pipe 27 %; what the one CTA of an SM has under way
// does not cover the trip to memory.  With 128 columns a CTA it was 49 us.
#include <cuda_runtime.h>

#include "lora_grad.cuh"
#include "sm100_ptx.cuh"

namespace gptq {
namespace {

constexpr int kDrain = 256, kCopy = 128, kAll = kDrain + kCopy + 32;
constexpr int kMmaWarp = (kDrain + kCopy) / 32;
constexpr int kTok = 64;                   // tokens per stage
constexpr int kCols = kGradTcCols;         // columns of X per CTA
constexpr int kSub = kTok * 128;           // bytes of 64 columns
constexpr int kXTile = kTok * kCols * 2;
constexpr int kFlush = 8;                  // stages between drains of TMEM

template <int RP>
struct Plan {
  static constexpr int N = 3 * RP;
  static constexpr int kPart = kTok * RP * 2;
  static constexpr int kFTile = 3 * kPart;
  static constexpr int kRing = RP == 64 ? 3 : RP == 32 ? 4 : 5;
  static constexpr int kOffF = kRing * kXTile;
  static constexpr int kOffTok = kOffF + kRing * kFTile;
  static constexpr int kOffBar = kOffTok + kGradTcPiece * 4;
  static constexpr int kSmem = kOffBar + 16 * kRing + 48;
  static constexpr int kAhead = kRing - 1;
  static constexpr int kTmem = RP == 16 ? 128 : RP == 32 ? 256 : 512;  // >= 2 N
  static_assert(kSmem <= 227 * 1024, "shared memory");
};

// X: 64 columns of a token are 128 swizzled bytes, 8 tokens 1024; the next 64
// columns lie kSub further.  f: rows of RP ranks under the swizzle of their
// width, the next part kPart further.
template <int RP>
__global__ void __launch_bounds__(kAll, 1)
    lora_grad_tc_kernel(const GradKernelArgs k, const __grid_constant__ CUtensorMap map_x0,
                        const __grid_constant__ CUtensorMap map_x1,
                        const __grid_constant__ CUtensorMap map_f0,
                        const __grid_constant__ CUtensorMap map_f1) {
  using L = Plan<RP>;
  extern __shared__ __align__(1024) char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  dep_launch();
  const int strips = k.side[0].tc_strips + k.side[1].tc_strips;
  const Piece pc = find_piece(k.a, blockIdx.x / strips, k.piece, 1);
  if (pc.slot < 0) {
    dep_wait();
    return;
  }
  const int strip = blockIdx.x % strips;
  const bool second = strip >= k.side[0].tc_strips;
  const GradSide& p = second ? k.side[1] : k.side[0];
  const CUtensorMap* map_x = second ? &map_x1 : &map_x0;
  const CUtensorMap* map_f = second ? &map_f1 : &map_f0;
  const int cs = (strip - (second ? k.side[0].tc_strips : 0)) * kCols;
  const int r0 = blockIdx.y * RP;
  const int C = (int)p.C;
  const int rank = lora_rank(k.a, pc.slot);
  const int count = r0 < rank ? pc.count : 0;
  const int stages = (count + kTok - 1) / kTok;
  const int tail = count % kTok;  // tokens of a short last stage

  const uint32_t base = ptx::smem_u32(smem);
  int* toks = reinterpret_cast<int*>(smem + L::kOffTok);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* free_ = full + L::kRing;
  uint64_t* summed = free_ + L::kRing;  // the stages up to a drain are done
  uint64_t* drained = summed + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  if (warp == 0) {
    ptx::tmem_alloc(tmem_slot, L::kTmem);
    ptx::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < L::kRing; ++i) {
      ptx::mbar_init(&full[i], kCopy);
      ptx::mbar_init(&free_[i], 1);
    }
    ptx::mbar_init(summed, 1);
    ptx::mbar_init(drained, kDrain);
    ptx::fence_mbar_init();
    *abort = 0;
  }
  for (int i = tid; i < stages * kTok; i += kAll)
    toks[i] = i < count ? piece_token(k.a, pc, i) : -1;
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  dep_wait();  // f comes from the kernel before this one

  // every wait has a limit; a CTA that met it gives NaN instead of sums
  bool bad = false;
  auto wait = [&](uint64_t* bar, int phase) {
    if (!ptx::mbar_wait_bounded(bar, phase & 1, abort, k.gate.limit_ns)) {
      *abort = 1;
      bad = true;
    }
  };
  float total[RP];  // ranks of column 128 (warp / 4) + 32 (warp % 4) + lane
#pragma unroll
  for (int i = 0; i < RP; ++i) total[i] = 0.f;

  if (warp < kDrain / 32) {
    for (int s0 = 0, f = 0; s0 < stages; s0 += kFlush, ++f) {
      wait(summed, f);
      if ((bad = __any_sync(~0u, bad))) break;
      ptx::tc_fence_after();
      const uint32_t at = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) +
                          (warp >> 2) * L::N;
#pragma unroll
      for (int i = 0; i < RP; i += 8) {
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
      ptx::mbar_arrive(drained);
    }
  } else if (warp < kMmaWarp) {
    const int ctid = tid - kDrain;
    // 16 bytes of a row a thread, 32 threads side by side
    const int j = lane, row0 = ctid >> 5;
    const int left = (C - cs - 8 * j) * 2;
    const int bytes = left < 0 ? 0 : left > 16 ? 16 : left;
    const bf16* X = static_cast<const bf16*>(p.X) + (bytes > 0 ? cs + 8 * j : 0);
    uint32_t late = 0;  // bit i: the stage i iterations ago was copied by cp.async
    int s = 0;
    if (ctid == 0 && !ptx::gate_wait_bounded(k.gate.gate, k.gate.limit_ns)) {
      *abort = 1;
      bad = true;
    }
    bad = __any_sync(~0u, bad);
    for (; s < stages + L::kAhead && !bad; ++s) {
      late <<= 1;
      if (s < stages) {
        const int slot = s % L::kRing;
        if (s >= L::kRing) wait(&free_[slot], s / L::kRing - 1);
        if ((bad = __any_sync(~0u, bad))) break;
        const int* t = toks + s * kTok;
        const bool run = run_of_64(t);
        if (ctid == 0) {
          uint64_t* bar = &full[slot];
          if (run)
            ptx::mbar_arrive_expect_tx(bar, L::kFTile + kXTile);
          else  // (with copies of its own to wait for, this thread arrives late too)
            ptx::mbar_expect_tx(bar, L::kFTile);
          ptx::tma_load_3d(base + L::kOffF + slot * L::kFTile, map_f, bar, r0,
                           pc.first + s * kTok, 0);
          if (run)
#pragma unroll
            for (int x = 0; x < kCols / 64; ++x)
              ptx::tma_load_2d(smem + slot * kXTile + x * kSub, map_x, bar, cs + 64 * x, t[0]);
        } else if (run) {
          ptx::mbar_arrive(&full[slot]);
        }
        if (!run) {
          late |= 1;
          const uint32_t dst = base + slot * kXTile + (j >> 3) * kSub;
#pragma unroll 4
          for (int i = 0; i < kTok / 4; ++i) {
            const int r = row0 + 4 * i, tok = t[r];
            const bool on = tok >= 0 && bytes > 0;
            copy16(dst + r * 128 + (((j & 7) ^ (r & 7)) << 4), X + (on ? (int64_t)tok * p.ldx : 0),
                   on ? bytes : 0);
          }
        }
      }
      ptx::cp_async_commit();
      ptx::cp_async_wait<L::kAhead>();
      if (late >> L::kAhead & 1) {
        ptx::fence_proxy_async_smem();
        ptx::mbar_arrive(&full[(s - L::kAhead) % L::kRing]);
      }
    }
    ptx::cp_async_wait_all();
    // on an early end: wait for the boxes that are under way
    if (bad && ctid == 0) {
      const volatile int never = 0;
      for (int i = max(0, s - L::kRing); i < min(s, stages); ++i)
        ptx::mbar_wait_bounded(&full[i % L::kRing], (i / L::kRing) & 1, &never, k.gate.limit_ns);
    }
  } else {
    int s = 0;
    for (; s < stages; ++s) {
      const int slot = s % L::kRing;
      if (s && s % kFlush == 0) wait(drained, s / kFlush - 1);
      wait(&full[slot], s / L::kRing);
      if ((bad = __any_sync(~0u, bad))) break;
      if (tail && s == stages - 1) {
        // f's box goes on into the next slot's tokens: rows of zeros instead
        constexpr int kRow = 2 * RP / 16;
        const int each = (kTok - tail) * kRow;
        for (int e = lane; e < 3 * each; e += 32)
          *reinterpret_cast<uint4*>(smem + L::kOffF + slot * L::kFTile + (e / each) * L::kPart +
                                    tail * 2 * RP + 16 * (e % each)) = make_uint4(0, 0, 0, 0);
        ptx::fence_proxy_async_smem();
        __syncwarp();
      }
      if (lane == 0) {
        ptx::tc_fence_after();
        const uint32_t x = base + slot * kXTile;
        const uint64_t df = ptx::smem_desc_rows(base + L::kOffF + slot * L::kFTile, 2 * RP, L::kPart);
        constexpr uint32_t id = ptx::idesc_bf16_f32(128, L::N) | (1u << 15) | (1u << 16);
#pragma unroll
        for (int h = 0; h < kCols / 128; ++h) {
          if (cs + 128 * h >= C) break;
          const uint64_t dx = ptx::smem_desc_rows(x + 2 * h * kSub, 128, kSub);
#pragma unroll
          for (int i = 0; i < kTok / 16; ++i)
            // 16 tokens on: 16 rows of either operand
            ptx::mma_bf16(tmem + h * L::N, dx + i * (2048 >> 4), df + i * ((32 * RP) >> 4), id,
                          (s % kFlush) | i);
        }
        ptx::mma_commit(&free_[slot]);
        if (s % kFlush == kFlush - 1 || s == stages - 1) ptx::mma_commit(summed);
      }
      __syncwarp();
    }
    // on an early end: TMEM is not given back under instructions that are under way
    const volatile int never = 0;
    if (bad && s > 0)
      ptx::mbar_wait_bounded(&free_[(s - 1) % L::kRing], ((s - 1) / L::kRing) & 1, &never,
                             k.gate.limit_ns);
  }
  __syncwarp();
  bad = __syncthreads_or(bad);
  if (warp == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, L::kTmem);
  }
  const int c = cs + 128 * (warp >> 2) + 32 * (warp & 3) + lane;
  if (tid >= kDrain || c >= C) return;
  store_column<RP>(k, p, pc, c, r0, rank, total, bad);
}

// The three bf16 parts of f in the plan's order, [part][position][rank], zeros
// from a slot's rank on: 8 ranks of a position a thread.
struct PartsArgs {
  LoraArgs a;
  const float* f[2];
  int64_t ldf[2];
  int vec[2], scaled[2];
  bf16* out[2];
  int width;  // ranks of a row of the parts
};
__global__ void __launch_bounds__(256) lora_parts_kernel(const PartsArgs k) {
  dep_launch();
  const int chunks = k.width / 8;
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t pos = e / chunks;
  const int r = 8 * (int)(e % chunks);
  const int side = blockIdx.y;
  int slot = -1, t = -1;
  if (pos < lora_start(k.a, k.a.n_slots) && pos >= lora_start(k.a, 0)) {
    int lo = 0, hi = k.a.n_slots;  // start[lo] <= pos < start[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (lora_start(k.a, mid) <= pos) lo = mid; else hi = mid;
    }
    slot = lo;
    t = k.a.order[pos];
    if (t < 0 || t >= k.a.ntok) t = -1;
  }
  const int left = t < 0 ? 0 : lora_rank(k.a, slot) - r;
  const float sc = t >= 0 && k.scaled[side] ? lora_scale(k.a, slot) : 1.f;
  dep_wait();  // f comes from the kernel before this one
  if (pos >= k.a.ntok || !k.f[side]) return;
  const float* f = k.f[side] + (int64_t)max(t, 0) * k.ldf[side] + r;
  float v[8];
  if (left >= 8 && k.vec[side]) {
    const float4 lo = reinterpret_cast<const float4*>(f)[0];
    const float4 hi = reinterpret_cast<const float4*>(f)[1];
    v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w;
    v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = i < left ? f[i] : 0.f;
  }
  uint32_t w[3][4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t q[3];
    split_pair<3>(v[2 * i] * sc, v[2 * i + 1] * sc, q);
#pragma unroll
    for (int c = 0; c < 3; ++c) w[c][i] = q[c];
  }
  bf16* out = k.out[side] + pos * k.width + r;
#pragma unroll
  for (int c = 0; c < 3; ++c)
    *reinterpret_cast<uint4*>(out + (int64_t)c * k.a.ntok * k.width) =
        make_uint4(w[c][0], w[c][1], w[c][2], w[c][3]);
}

int block_of(int max_rank) { return max_rank <= 16 ? 16 : max_rank <= 32 ? 32 : 64; }
int width_of(int max_rank) {
  const int rp = block_of(max_rank);
  return (max_rank + rp - 1) / rp * rp;
}

template <int RP>
cudaError_t launch(const GradKernelArgs& k, void* const (&parts)[2], cudaLaunchConfig_t c) {
  auto kern = lora_grad_tc_kernel<RP>;
  static std::atomic<uint64_t> raised{0};
  cudaError_t e =
      raise_limits(reinterpret_cast<const void*>(kern), Plan<RP>::kSmem, false, raised);
  if (e != cudaSuccess) return e;
  const int width = width_of(k.a.max_rank);
  CUtensorMap x[2] = {}, f[2] = {};
  for (int i = 0; i < 2; ++i) {
    const GradSide& d = k.side[i];
    if (d.tc_strips &&
        (!make_tma_rows(&x[i], d.X, 2, 0, k.a.ntok, d.C, 0, d.ldx, 64, kTok, 128) ||
         !make_tma_rows(&f[i], parts[i], 2, 3, k.a.ntok, width, k.a.ntok * width, width, RP, kTok,
                        2 * RP, 3)))
      return cudaErrorInvalidValue;
  }
  const int64_t pieces = (k.a.ntok + k.piece - 1) / k.piece + k.a.n_slots;
  const int64_t ctas = pieces * (k.side[0].tc_strips + k.side[1].tc_strips);
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  c.gridDim = dim3((unsigned)ctas, width / RP);
  c.blockDim = dim3(kAll);
  c.dynamicSmemBytes = Plan<RP>::kSmem;
  e = cudaLaunchKernelEx(&c, kern, k, x[0], x[1], f[0], f[1]);
  note_launch();
  return e;
}

}  // namespace

size_t lora_grad_parts_bytes(const LoraArgs& a) {
  return 2 * (((size_t)3 * a.ntok * width_of(a.max_rank) * 2 + 255) / 256 * 256);
}

cudaError_t launch_lora_grad_tc(const GradKernelArgs& k, void* ws, cudaStream_t s) {
  void* parts[2] = {ws, static_cast<char*>(ws) + lora_grad_parts_bytes(k.a) / 2};
  PartsArgs pa = {};
  pa.a = k.a;
  pa.width = width_of(k.a.max_rank);
  int sides = 1;
  for (int i = 0; i < 2; ++i) {
    const GradSide& d = k.side[i];
    if (!d.tc_strips) continue;
    pa.f[i] = d.f;
    pa.ldf[i] = d.ldf;
    pa.vec[i] = d.vec_f;
    pa.scaled[i] = d.scaled;
    pa.out[i] = static_cast<bf16*>(parts[i]);
    sides = i + 1;
  }
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)((k.a.ntok * (pa.width / 8) + 255) / 256), sides);
  c.blockDim = dim3(256);
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = k.behind ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&c, lora_parts_kernel, pa);
  note_launch();
  c.numAttrs = 1;
  if (e != cudaSuccess) return e;
  const int rp = block_of(k.a.max_rank);
  return rp == 16 ? launch<16>(k, parts, c) : rp == 32 ? launch<32>(k, parts, c)
                                                       : launch<64>(k, parts, c);
}

}  // namespace gptq
