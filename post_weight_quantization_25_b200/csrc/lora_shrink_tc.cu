// The projection down to the rank (lora_shrink.cu) on tcgen05, for many bf16
// tokens: out[t] = scale (X[t] W_a).
//
// It is bound by reading X once, at ranks up to 64 with time to spare on any
// matrix path; what the register-fed kernel lacks is bytes in flight (a warp
// has two blocks of its own rows on the way, 30 KB per SM, and waits).  Here a
// CTA's 128 tokens are the M of tcgen05.mma, the ranks its N, and K runs in
// stages of 64 through a ring of tiles that no thread touches: X by TMA boxes
// of 32 tokens where those are consecutive rows (by cp.async of 16 bytes with
// the swizzle applied by hand where they are not), W by TMA boxes in either
// layout, K contiguous (A of the forward pass) or ranks contiguous (B of the
// backward pass).  About 90 KB per CTA are under way, two CTAs share an SM.
//
// Rows of X behind the piece's last token and ranks from the slot's rank on
// are computed with whatever they hold and not stored: they stay in their own
// rows and columns of the sums.  The tensor core cuts its sums off, so four
// sums in TMEM take turns and are moved to rounded totals every 32 stages.
// The CTAs of a cluster share K and add up through distributed shared memory.
// Measured: 8192 x 28672 at rank 32 74 us, 6.3 TB/s (the register-fed kernel:
// 250); 4096 x 4096 at rank 16 15 us, of which the first box takes 4 and the
// cluster's exchange 2.7.
#include <cuda_runtime.h>

#include "lora_shrink.cuh"
#include "sm100_ptx.cuh"

namespace gptq {
namespace {

constexpr int kTile = 128;            // tokens
constexpr int kK = 64;                // of K per stage
constexpr int kXTile = kTile * kK * 2;
constexpr int kSums = 4;              // accumulators that take turns
constexpr int kFlush = 8 * kSums;     // stages between drains
constexpr int kDrain = 128, kCopy = 128, kAll = kDrain + kCopy + 32;

template <int RP>
struct Plan {
  static constexpr int kWTile = RP * kK * 2;
  static constexpr int kRing = RP == 16 ? 6 : RP == 32 ? 5 : 4;
  static constexpr int kOffW = kRing * kXTile;
  static constexpr int kOffTok = kOffW + kRing * kWTile;
  static constexpr int kOffBar = kOffTok + kTile * 4;
  static constexpr int kSmem = kOffBar + 16 * kRing + 48;  // barriers, TMEM, abort, runs
  static constexpr int kAhead = kRing - 1;
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs per SM");
  static_assert(kTile * (RP + 4) * 4 <= kOffW, "the sums fit the ring");
};

template <bool RI, int RP>
__global__ void __launch_bounds__(kAll, 2)
    lora_shrink_tc_kernel(const ShrinkArgs p, const __grid_constant__ CUtensorMap map_x,
                          const __grid_constant__ CUtensorMap map_w) {
  using L = Plan<RP>;
  extern __shared__ __align__(1024) char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int splits = gridDim.y, split = blockIdx.y;
  dep_launch();
  const Piece pc = find_piece(p.a, blockIdx.x, kTile, 0);
  if (pc.slot < 0) return;  // the same in every CTA of the cluster
  const uint32_t base = ptx::smem_u32(smem);
  int* toks = reinterpret_cast<int*>(smem + L::kOffTok);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* free_ = full + L::kRing;
  uint64_t* summed = free_ + L::kRing;  // the stages up to a drain are done
  uint64_t* drained = summed + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drained + 1);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int r0 = blockIdx.z * RP;
  const int rank = lora_rank(p.a, pc.slot);
  const int K = (int)p.K;
  const int nk = (K + kK - 1) / kK;  // stage s of this CTA: block split + s splits
  const int stages = r0 < rank && split < nk ? (nk - split + splits - 1) / splits : 0;
  // groups of 32 tokens that are consecutive rows (or mostly there at all)
  uint32_t* runs = reinterpret_cast<uint32_t*>(smem + L::kOffBar + 16 * L::kRing + 32);
  if (tid < kTile) {
    const int t = piece_token(p.a, pc, tid);
    toks[tid] = t;
    const bool run = row_run(t);
    if (lane == 0) runs[warp] = run;
  }
  if (warp == 0) {
    ptx::tmem_alloc(tmem_slot, kSums * RP);
    ptx::tmem_relinquish();
  }
  __syncthreads();
  uint32_t boxes_of = 0;  // bit i: group i comes as a box
#pragma unroll
  for (int i = 0; i < kTile / 32; ++i) boxes_of |= runs[i] << i;
  const bool gap = boxes_of != (1u << (kTile / 32)) - 1;
  if (tid == 0) {
    for (int i = 0; i < L::kRing; ++i) {
      ptx::mbar_init(&full[i], gap ? 1 + kCopy : 1);
      ptx::mbar_init(&free_[i], 1);
    }
    ptx::mbar_init(summed, 1);
    ptx::mbar_init(drained, kDrain);
    ptx::fence_mbar_init();
    *abort = 0;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  // every wait has a limit; a CTA that met it gives NaN instead of sums, and so
  // does every CTA of its cluster, which adds its sums to its own
  bool bad = false;
  auto wait = [&](uint64_t* bar, int phase) {
    if (!ptx::mbar_wait_bounded(bar, phase & 1, abort, p.gate.limit_ns)) {
      *abort = 1;
      bad = true;
    }
  };
  float total[RP];
#pragma unroll
  for (int i = 0; i < RP; ++i) total[i] = 0.f;

  if (warp < kDrain / 32) {
    for (int s0 = 0, f = 0; s0 < stages; s0 += kFlush, ++f) {
      wait(summed, f);
      if ((bad = __any_sync(~0u, bad))) break;
      ptx::tc_fence_after();
      const int sums = min(kSums, stages - s0);
      const uint32_t at = tmem + (static_cast<uint32_t>(32 * warp) << 16);
#pragma unroll
      for (int i = 0; i < RP; i += 8)
        for (int a = 0; a < sums; ++a) {
          uint32_t v[8];
          ptx::tmem_ld_32x32b_x8(at + a * RP + i, v);
          ptx::tmem_ld_wait();
#pragma unroll
          for (int x = 0; x < 8; ++x) total[i + x] += __uint_as_float(v[x]);
        }
      ptx::tc_fence_before();
      ptx::mbar_arrive(drained);
    }
  } else if (warp < (kDrain + kCopy) / 32) {
    const int ctid = tid - kDrain;
    const int x_bytes = __popc(boxes_of) * (kXTile / (kTile / 32));
    auto boxes = [&](int s) {  // one thread
      const int k = (split + s * splits) * kK, slot = s % L::kRing;
      uint64_t* bar = &full[slot];
      ptx::mbar_arrive_expect_tx(bar, L::kWTile + x_bytes);
#pragma unroll
      for (int i = 0; i < kTile / 32; ++i)
        if (boxes_of >> i & 1)
          ptx::tma_load_2d(smem + slot * kXTile + i * 32 * 128, &map_x, bar, k, toks[32 * i]);
      const uint32_t w = base + L::kOffW + slot * L::kWTile;
      if (RI)
        ptx::tma_load_3d(w, &map_w, bar, r0, k, pc.slot);
      else
        ptx::tma_load_3d(w, &map_w, bar, k, r0, pc.slot);
    };
    int s = 0;
    // (the test gate: one CTA of a cluster waits for it)
    if (ctid == 0 && split == 0 && !ptx::gate_wait_bounded(p.gate.gate, p.gate.limit_ns)) {
      *abort = 1;
      bad = true;
    }
    if (!gap) {
      if (ctid == 0)
        for (; s < stages && !bad; ++s) {
          if (s >= L::kRing) wait(&free_[s % L::kRing], s / L::kRing - 1);
          if (bad) break;
          boxes(s);
        }
    } else {
      // a thread copies 16 bytes of 8 rows
      const int j = ctid & 7, row0 = ctid >> 3;
      const bf16* src[8];
      bool on[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int t = toks[row0 + 16 * i];
        on[i] = t >= 0;
        src[i] = static_cast<const bf16*>(p.X) + (int64_t)max(t, 0) * p.ldx;
      }
      auto finish = [&](int q) {  // the copies of stage q are there
        ptx::cp_async_wait<L::kAhead>();
        if (q >= 0) {
          ptx::fence_proxy_async_smem();
          ptx::mbar_arrive(&full[q % L::kRing]);
        }
      };
      for (; s < stages + L::kAhead && !bad; ++s) {
        if (s < stages) {
          if (s >= L::kRing) wait(&free_[s % L::kRing], s / L::kRing - 1);
          if (bad) break;
          if (ctid == 0) boxes(s);
          const int k = (split + s * splits) * kK + 8 * j;
          const int left = (K - k) * 2;
          const int bytes = left < 0 ? 0 : left > 16 ? 16 : left;
          const uint32_t dst = base + (s % L::kRing) * kXTile;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = row0 + 16 * i;
            if (boxes_of >> (i / 2) & 1) continue;  // r's group of 32
            copy16(dst + r * 128 + ((j ^ (r & 7)) << 4), src[i] + (bytes > 0 ? k : 0),
                   on[i] ? bytes : 0);
          }
        }
        ptx::cp_async_commit();
        finish(s - L::kAhead);
      }
      ptx::cp_async_wait_all();
    }
    // on an early end: wait for the boxes that are under way
    if (bad && ctid == 0) {
      const volatile int never = 0;
      for (int i = max(0, s - L::kRing); i < min(s, stages); ++i)
        ptx::mbar_wait_bounded(&full[i % L::kRing], (i / L::kRing) & 1, &never, p.gate.limit_ns);
    }
  } else if (lane == 0) {
    int s = 0;
    for (; s < stages; ++s) {
      if (s && s % kFlush == 0) wait(drained, s / kFlush - 1);
      wait(&full[s % L::kRing], s / L::kRing);
      if (bad) break;
      ptx::tc_fence_after();
      const uint32_t x = base + (s % L::kRing) * kXTile;
      const uint32_t w = base + L::kOffW + (s % L::kRing) * L::kWTile;
      const uint64_t dx = ptx::smem_desc_sw128(x);
      const uint64_t dw = RI ? ptx::smem_desc_rows(w, 2 * RP, L::kWTile) : ptx::smem_desc_sw128(w);
#pragma unroll
      for (int i = 0; i < kK / 16; ++i)
        ptx::mma_bf16(tmem + (s % kSums) * RP, dx + i * (32 >> 4),
                      dw + i * ((RI ? 32 * RP : 32) >> 4),
                      ptx::idesc_bf16_f32(kTile, RP) | (RI ? 1u << 16 : 0u),
                      (s % kFlush >= kSums) | i);
      ptx::mma_commit(&free_[s % L::kRing]);
      if (s % kFlush == kFlush - 1 || s == stages - 1) ptx::mma_commit(summed);
    }
    // on an early end: TMEM is not given back under instructions that are under way
    const volatile int never = 0;
    if (bad && s > 0)
      ptx::mbar_wait_bounded(&free_[(s - 1) % L::kRing], ((s - 1) / L::kRing) & 1, &never,
                             p.gate.limit_ns);
  }
  __syncwarp();
  bad = __syncthreads_or(bad);
  if (warp == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, kSums * RP);
  }
  if (bad) {
#pragma unroll
    for (int i = 0; i < RP; ++i) total[i] = __uint_as_float(0x7fffffffu);
  }
  const float sc = p.scaled ? lora_scale(p.a, pc.slot) : 1.f;
  const int rmax = p.a.max_rank;
  // 4 ranks of a token
  auto store = [&](int tok, int r, float4 v) {
    const int t = toks[tok];
    if (t < 0 || tok >= pc.count || r >= rmax) return;
    const float e[4] = {v.x, v.y, v.z, v.w};
    float o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = r + i < rank ? e[i] * sc : 0.f;
    float* at = p.out + (int64_t)t * p.ldo + r;
    if (p.vec_o && r + 4 <= rmax) {
      *reinterpret_cast<float4*>(at) = make_float4(o[0], o[1], o[2], o[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (r + i < rmax) at[i] = o[i];
    }
  };
  // The sums go through shared memory (the ring is used up): a thread has all
  // ranks of one token, the stores want the ranks side by side.
  constexpr int RL = RP + 4;
  float* red = reinterpret_cast<float*>(smem);
  if (tid < kDrain) {
#pragma unroll
    for (int i = 0; i < RP; i += 4)
      *reinterpret_cast<float4*>(red + tid * RL + i) =
          make_float4(total[i], total[i + 1], total[i + 2], total[i + 3]);
  }
  if (splits == 1) {
    __syncthreads();
    for (int e = tid; e < kTile * RP / 4; e += kAll) {
      const int tok = e / (RP / 4), r = 4 * (e % (RP / 4));
      store(tok, r0 + r, *reinterpret_cast<const float4*>(red + tok * RL + r));
    }
    return;
  }
  ptx::cluster_sync();
  for (int e = split * kAll + tid; e < kTile * RP / 4; e += splits * kAll) {
    const int tok = e / (RP / 4), r = 4 * (e % (RP / 4));
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int c = 0; c < splits; ++c) {
      float4 v;
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                   : "r"(ptx::mapa_shared(red + tok * RL + r, c)));
      s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
    }
    store(tok, r0 + r, s);
  }
  ptx::cluster_sync();  // no CTA leaves while its sums are read
}

template <bool RI, int RP>
cudaError_t launch(const ShrinkArgs& p, cudaStream_t s) {
  auto k = lora_shrink_tc_kernel<RI, RP>;
  static std::atomic<uint64_t> raised{0};
  cudaError_t e =
      raise_limits(reinterpret_cast<const void*>(k), Plan<RP>::kSmem, false, raised);
  if (e != cudaSuccess) return e;
  const LoraArgs& a = p.a;
  CUtensorMap mx, mw;
  const int64_t wrows = RI ? p.K : a.max_rank, wcols = RI ? a.max_rank : p.K;
  if (!make_tma_rows(&mx, p.X, 2, 0, a.ntok, p.K, 0, p.ldx, kK, 32, 128) ||
      !make_tma_rows(&mw, p.W, 2, a.n_slots, wrows, wcols,
                     a.n_slots > 1 ? p.stride_w : wrows * p.ldw, p.ldw, RI ? RP : kK, RI ? kK : RP,
                     RI ? 2 * RP : 128))
    return cudaErrorInvalidValue;
  const int64_t full = (a.ntok + kTile - 1) / kTile;
  const int64_t pieces = full + (a.n_slots < a.ntok ? a.n_slots : a.ntok);
  const int rblocks = (a.max_rank + RP - 1) / RP;
  // As many CTAs as two per SM hold at once, each with 4 stages or more
  int64_t splits = 2 * num_sms() / (full * rblocks);
  const int64_t most = p.K / (4 * kK);
  splits = splits > most ? most : splits;
  splits = splits > 8 ? 8 : splits < 1 ? 1 : splits;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)pieces, (unsigned)splits, rblocks);
  c.blockDim = dim3(kAll);
  c.dynamicSmemBytes = Plan<RP>::kSmem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = 1;
  at[0].val.clusterDim.y = (unsigned)splits;
  at[0].val.clusterDim.z = 1;
  c.attrs = at;
  c.numAttrs = splits > 1 ? 1 : 0;
  e = cudaLaunchKernelEx(&c, k, p, mx, mw);
  note_launch();
  return e;
}

}  // namespace

cudaError_t launch_lora_shrink_tc(const ShrinkArgs& p, bool ranks_inner, cudaStream_t s) {
  const int r = p.a.max_rank;
  if (ranks_inner)
    return r <= 16 ? launch<true, 16>(p, s) : r <= 32 ? launch<true, 32>(p, s)
                                                      : launch<true, 64>(p, s);
  return r <= 16 ? launch<false, 16>(p, s) : r <= 32 ? launch<false, 32>(p, s)
                                                     : launch<false, 64>(p, s);
}

}  // namespace gptq
