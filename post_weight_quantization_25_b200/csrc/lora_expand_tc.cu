// The projection back from the rank (lora_expand.cu) on tcgen05, for many
// tokens: Y[t] += scale (u[t] W_a).
//
// Bound by reading and writing Y once.  A CTA keeps the parts of 128 tokens' u
// as A operands and walks over Y in boxes of 128 tokens x 128 bytes: a ring of
// boxes of Y and of W is filled ahead (TMA boxes where the tokens are
// consecutive rows, 16-byte cp.async for Y where they are not), the product of
// a box appears in TMEM, and 8 warps add it to Y's box in shared memory, a row
// a thread, and store the box with rows side by side.  Loads, products and
// stores of different boxes overlap and no thread waits for memory.
//
// u is fp32 and enters as 3 exact bf16 parts towards an fp32 Y, as 2 (2^-17)
// towards a bf16 Y.  Ranks from the slot's rank on must not reach the sum: u
// is zero there, and W's entries, which may be NaN, are zeroed in shared
// memory if an instruction's 16 ranks hold any.  Measured: 8192 x 8192 bf16 at
// rank 32 51 us, 8192 x 11008 at rank 16 67 us, 5.3 TB/s of reading and writing
// (the register-fed kernel: 78 and 93).
#include <cuda_runtime.h>

#include "lora_expand.cuh"
#include "sm100_ptx.cuh"

namespace gptq {
namespace {

constexpr int kTile = 128;       // tokens
constexpr int kBox = kTile * 128;
constexpr int kWork = 256, kCopy = 128, kAll = kWork + kCopy + 32;
constexpr int kMmaWarp = (kWork + kCopy) / 32;

template <class TY, int RP>
struct Plan {
  static constexpr int NU = sizeof(TY) == 2 ? 2 : 3;
  static constexpr int N = 128 / (int)sizeof(TY);  // columns of a box
  static constexpr int kPart = kTile * RP * 2;
  static constexpr int kWBox = N * RP * 2;
  static constexpr int kRing = RP == 16 ? 5 : RP == 32 ? 4 : 3;
  static constexpr int kOffA = kRing * kBox;
  static constexpr int kOffW = kOffA + NU * kPart;
  static constexpr int kOffTok = kOffW + kRing * kWBox;
  static constexpr int kOffBar = kOffTok + kTile * 4;
  static constexpr int kSmem = kOffBar + 8 * (4 * kRing + 4) + 32;
  static constexpr int kAhead = kRing - 1;
  static_assert(kOffW % 1024 == 0 && kWBox % 1024 == 0, "swizzled tiles");
  static_assert(2 * (kSmem + 1024) <= 228 * 1024, "two CTAs per SM");
};

// byte offset of 16-byte piece `chunk` of a row
__device__ __forceinline__ int swizzled(int row, int chunk, int bytes) {
  const int x = bytes == 128 ? row & 7 : bytes == 64 ? (row >> 1) & 3 : (row >> 2) & 1;
  return row * bytes + ((chunk ^ x) << 4);
}

template <class TY, bool CI, int RP>
__global__ void __launch_bounds__(kAll, 2)
    lora_expand_tc_kernel(const ExpandArgs p, const __grid_constant__ CUtensorMap map_y,
                          const __grid_constant__ CUtensorMap map_w) {
  using L = Plan<TY, RP>;
  constexpr int N = L::N, NU = L::NU, E = 16 / (int)sizeof(TY);
  extern __shared__ __align__(1024) char smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  dep_launch();
  const Piece pc = find_piece(p.a, blockIdx.x / p.strips, kTile, 0);
  const int rank = pc.slot < 0 ? 0 : lora_rank(p.a, pc.slot);
  const int C = (int)p.C;
  const int first = (int)(blockIdx.x % p.strips) * p.turns;  // box
  const int boxes = min(p.turns, (C + N - 1) / N - first);
  if (rank == 0 || boxes <= 0) {
    dep_wait();
    return;
  }
  const uint32_t base = ptx::smem_u32(smem);
  int* toks = reinterpret_cast<int*>(smem + L::kOffTok);
  uint64_t* yfull = reinterpret_cast<uint64_t*>(smem + L::kOffBar);
  uint64_t* yfree = yfull + L::kRing;
  uint64_t* wfull = yfree + L::kRing;
  uint64_t* wfree = wfull + L::kRing;
  uint64_t* sfull = wfree + L::kRing;  // sums in TMEM
  uint64_t* sfree = sfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(sfree + 2);
  volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

  // groups of 32 tokens that are consecutive rows (or mostly there at all)
  uint32_t* runs = reinterpret_cast<uint32_t*>(smem + L::kOffBar + 8 * (4 * L::kRing + 4) + 8);
  if (tid < kTile) {
    const int t = piece_token(p.a, pc, tid);
    toks[tid] = t;
    const bool run = row_run(t);
    if (lane == 0) runs[warp] = run;
  }
  // ranks that an instruction reads but the slot does not have
  const int steps = (rank + 15) / 16;
  const bool mask = rank < min(16 * steps, p.a.max_rank);
  if (warp == 0) {
    ptx::tmem_alloc(tmem_slot, 2 * N);
    ptx::tmem_relinquish();
  }
  __syncthreads();
  uint32_t boxes_of = 0;  // bit i: group i comes as a box
#pragma unroll
  for (int i = 0; i < kTile / 32; ++i) boxes_of |= runs[i] << i;
  const bool gap = boxes_of != (1u << (kTile / 32)) - 1;
  if (tid == 0) {
    for (int i = 0; i < L::kRing; ++i) {
      ptx::mbar_init(&yfull[i], gap ? 1 + kCopy : 1);
      ptx::mbar_init(&yfree[i], kWork);
      ptx::mbar_init(&wfull[i], 1);
      ptx::mbar_init(&wfree[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&sfull[i], 1);
      ptx::mbar_init(&sfree[i], kWork);
    }
    ptx::fence_mbar_init();
    *abort = 0;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  TY* Y = static_cast<TY*>(p.Y);

  // every wait has a limit; a CTA that met it leaves NaN in its part of Y
  bool bad = false;
  auto wait = [&](uint64_t* bar, int phase) {
    if (!ptx::mbar_wait_bounded(bar, phase & 1, abort, p.gate.limit_ns)) {
      *abort = 1;
      bad = true;
    }
  };

  if (warp < kWork / 32) {
    // the parts of u, 8 ranks of a token a thread
    dep_wait();  // u comes from a kernel before this one
    const float sc = p.scaled ? lora_scale(p.a, pc.slot) : 1.f;
    constexpr int kChunks = RP / 8;
    for (int e = tid; e < kTile * kChunks; e += kWork) {
      const int row = e / kChunks, ch = e % kChunks;
      const int t = toks[row], left = t >= 0 ? rank - 8 * ch : 0;
      const float* u = p.u + (int64_t)max(t, 0) * p.ldu + 8 * ch;
      float v[8];
      if (left >= 8 && p.vec_u) {
        const float4 lo = reinterpret_cast<const float4*>(u)[0];
        const float4 hi = reinterpret_cast<const float4*>(u)[1];
        v[0] = lo.x, v[1] = lo.y, v[2] = lo.z, v[3] = lo.w;
        v[4] = hi.x, v[5] = hi.y, v[6] = hi.z, v[7] = hi.w;
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = i < left ? u[i] : 0.f;
      }
      uint32_t w[NU][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t q[NU];
        split_pair<NU>(v[2 * i] * sc, v[2 * i + 1] * sc, q);
#pragma unroll
        for (int c = 0; c < NU; ++c) w[c][i] = q[c];
      }
#pragma unroll
      for (int c = 0; c < NU; ++c)
        *reinterpret_cast<uint4*>(smem + L::kOffA + c * L::kPart + swizzled(row, ch, 2 * RP)) =
            make_uint4(w[c][0], w[c][1], w[c][2], w[c][3]);
    }
    ptx::fence_proxy_async_smem();
  }
  // the copies do not wait for u
  if (tid < kWork || warp == kMmaWarp) ptx::named_bar_sync(2, kWork + 32);

  if (warp < kWork / 32) {
    const int row = 32 * (warp & 3) + lane, half = warp >> 2;
    for (int s = 0; s < boxes; ++s) {
      const int slot = s % L::kRing;
      char* box = smem + slot * kBox;
      wait(&yfull[slot], s / L::kRing);
      wait(&sfull[s & 1], s >> 1);
      if ((bad = !ptx::named_bar_and(1, kWork, !bad))) break;
      ptx::tc_fence_after();
      // half of a row's columns a thread
#pragma unroll
      for (int i = 0; i < N / 2; i += 16) {
        uint32_t v[16];
        ptx::tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + (s & 1) * N +
                      half * (N / 2) + i, v);
        ptx::tmem_ld_wait();
#pragma unroll
        for (int x = 0; x < 16; x += E) {
          Raw<TY, E>* y = reinterpret_cast<Raw<TY, E>*>(
              box + swizzled(row, (half * (N / 2) + i + x) / E, 128));
          const uint4 old = *reinterpret_cast<const uint4*>(y);
          Raw<TY, E> r;
          memcpy(r.w, &old, 16);
          float d[E];
#pragma unroll
          for (int j = 0; j < E; ++j) d[j] = __uint_as_float(v[x + j]);
          add_row(d, r);
          r = round_row<TY, E>(d);
          uint4 now;
          memcpy(&now, r.w, 16);
          *reinterpret_cast<uint4*>(y) = now;
        }
      }
      ptx::tc_fence_before();
      ptx::mbar_arrive(&sfree[s & 1]);
      ptx::named_bar_sync(1, kWork);
      // out, 8 threads a row
      const int j = tid & 7, c = (first + s) * N + j * E;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = (tid >> 3) + 32 * i;
        const uint4 v = *reinterpret_cast<const uint4*>(box + swizzled(r, j, 128));
        const int t = toks[r];
        if (t < 0 || c >= C) continue;
        TY* at = Y + (int64_t)t * p.ldy + c;
        if (c + E <= C) {
          *reinterpret_cast<uint4*>(at) = v;
        } else {
          TY e[E];
          memcpy(e, &v, 16);
#pragma unroll
          for (int x = 0; x < E; ++x)
            if (c + x < C) at[x] = e[x];
        }
      }
      ptx::fence_proxy_async_smem();  // the next box comes through the async proxy
      ptx::mbar_arrive(&yfree[slot]);
    }
  } else if (warp < kMmaWarp) {
    const int ctid = tid - kWork;
    const int j = ctid & 7, row0 = ctid >> 3;
    auto finish = [&](int q) {  // cp.async: the copies of box q are there
      ptx::cp_async_wait<L::kAhead>();
      if (q >= 0) ptx::mbar_arrive(&yfull[q % L::kRing]);
    };
    int s = 0;
    const int end = gap ? boxes + L::kAhead : boxes;
    if (ctid == 0 && !ptx::gate_wait_bounded(p.gate.gate, p.gate.limit_ns)) {
      *abort = 1;
      bad = true;
    }
    if (gap || ctid == 0) {
      for (; s < end && !bad; ++s) {
        if (s < boxes) {
          const int slot = s % L::kRing, c0 = (first + s) * N;
          if (s == L::kRing) dep_wait();  // (no clock runs while u is awaited)
          if (s >= L::kRing) {
            wait(&yfree[slot], s / L::kRing - 1);
            wait(&wfree[slot], s / L::kRing - 1);
          }
          if (bad) break;
          if (ctid == 0) {
            ptx::mbar_arrive_expect_tx(&wfull[slot], L::kWBox);
            const uint32_t w = base + L::kOffW + slot * L::kWBox;
            if (CI)
              ptx::tma_load_3d(w, &map_w, &wfull[slot], c0, 0, pc.slot);
            else
              ptx::tma_load_3d(w, &map_w, &wfull[slot], 0, c0, pc.slot);
          }
          if (ctid == 0) {
            ptx::mbar_arrive_expect_tx(&yfull[slot], __popc(boxes_of) * (kBox / (kTile / 32)));
#pragma unroll
            for (int i = 0; i < kTile / 32; ++i)
              if (boxes_of >> i & 1)
                ptx::tma_load_2d(smem + slot * kBox + i * 32 * 128, &map_y, &yfull[slot], c0,
                                 toks[32 * i]);
          }
          if (gap) {
            const int c = c0 + E * j;
            const int left = (C - c) * (int)sizeof(TY);
            const int bytes = left < 0 ? 0 : left > 16 ? 16 : left;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              if (boxes_of >> (i / 2) & 1) continue;  // the row's group of 32
              const int r = row0 + 16 * i, t = toks[r];
              const bool on = t >= 0 && bytes > 0;
              copy16(base + slot * kBox + swizzled(r, j, 128),
                     Y + (on ? (int64_t)t * p.ldy + c : 0), on ? bytes : 0);
            }
          }
        }
        if (gap) {
          ptx::cp_async_commit();
          finish(s - L::kAhead);
        }
      }
    }
    ptx::cp_async_wait_all();
    // on an early end: wait for the boxes that are under way
    if (bad && ctid == 0) {
      const volatile int never = 0;
      for (int i = max(0, s - L::kRing); i < min(s, boxes); ++i) {
        ptx::mbar_wait_bounded(&wfull[i % L::kRing], (i / L::kRing) & 1, &never, p.gate.limit_ns);
        ptx::mbar_wait_bounded(&yfull[i % L::kRing], (i / L::kRing) & 1, &never, p.gate.limit_ns);
      }
    }
  } else {
    int s = 0;
    for (; s < boxes; ++s) {
      const int slot = s % L::kRing;
      wait(&wfull[slot], s / L::kRing);
      if (s >= 2) wait(&sfree[s & 1], (s >> 1) - 1);
      if ((bad = __any_sync(~0u, bad))) break;
      char* wbox = smem + L::kOffW + slot * L::kWBox;
      if (mask) {
        if (CI) {  // whole rows
          constexpr int kRow = 2 * N / 16;
          for (int e = lane; e < (16 * steps - rank) * kRow; e += 32)
            *reinterpret_cast<uint4*>(wbox + (rank + e / kRow) * (2 * N) + 16 * (e % kRow)) =
                make_uint4(0, 0, 0, 0);
        } else {  // the ends of the rows
          for (int n = lane; n < N; n += 32)
            for (int r = rank; r < 16 * steps; ++r)
              *reinterpret_cast<uint16_t*>(wbox + swizzled(n, r / 8, 2 * RP) + 2 * (r % 8)) = 0;
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
      }
      if (lane == 0) {
        ptx::tc_fence_after();
        const uint64_t dw = ptx::smem_desc_rows(ptx::smem_u32(wbox), CI ? 2 * N : 2 * RP);
        const uint32_t d = tmem + (s & 1) * N;
        constexpr uint32_t id = ptx::idesc_bf16_f32(kTile, N) | (CI ? 1u << 16 : 0u);
        // the small parts first
#pragma unroll
        for (int c = NU - 1; c >= 0; --c) {
          const uint64_t da = ptx::smem_desc_rows(base + L::kOffA + c * L::kPart, 2 * RP);
          for (int i = 0; i < steps; ++i)
            ptx::mma_bf16(d, da + i * (32 >> 4), dw + i * ((CI ? 32 * N : 32) >> 4), id,
                          c < NU - 1 || i > 0);
        }
        ptx::mma_commit(&wfree[slot]);
        ptx::mma_commit(&sfull[s & 1]);
      }
      __syncwarp();
    }
    // on an early end: TMEM is not given back under instructions that are under way
    const volatile int never = 0;
    if (bad && s > 0)
      ptx::mbar_wait_bounded(&wfree[(s - 1) % L::kRing], ((s - 1) / L::kRing) & 1, &never,
                             p.gate.limit_ns);
  }
  __syncwarp();
  bad = __syncthreads_or(bad);
  if (warp == 0) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, 2 * N);
  }
  if (bad)
    for (int r = warp; r < pc.count; r += kAll / 32)
      for (int c = first * N + lane; c < min((first + boxes) * N, C); c += 32)
        if (toks[r] >= 0) Y[(int64_t)toks[r] * p.ldy + c] = from_f32<TY>(__uint_as_float(0x7fffffffu));
}

template <class TY, bool CI, int RP>
cudaError_t launch(ExpandArgs p, cudaStream_t s) {
  using L = Plan<TY, RP>;
  auto k = lora_expand_tc_kernel<TY, CI, RP>;
  static std::atomic<uint64_t> raised{0};
  cudaError_t e =
      raise_limits(reinterpret_cast<const void*>(k), L::kSmem, false, raised);
  if (e != cudaSuccess) return e;
  const LoraArgs& a = p.a;
  CUtensorMap my, mw;
  const int64_t wrows = CI ? a.max_rank : p.C, wcols = CI ? p.C : a.max_rank;
  if (!make_tma_rows(&my, p.Y, sizeof(TY), 0, a.ntok, p.C, 0, p.ldy, L::N, 32, 128) ||
      !make_tma_rows(&mw, p.W, 2, a.n_slots, wrows, wcols,
                     a.n_slots > 1 ? p.stride_w : wrows * p.ldw, p.ldw, CI ? L::N : RP,
                     CI ? RP : L::N, CI ? 2 * L::N : 2 * RP))
    return cudaErrorInvalidValue;
  const int64_t full = (a.ntok + kTile - 1) / kTile;
  const int64_t pieces = full + (a.n_slots < a.ntok ? a.n_slots : a.ntok);
  // One round of two CTAs per SM; two where a CTA still has 16 boxes then
  const int64_t boxes = (p.C + L::N - 1) / L::N, slots = 2 * num_sms();
  const int64_t rounds = full * boxes >= 32 * slots ? 2 : 1;
  int64_t across = slots * rounds / full;
  across = across < 1 ? 1 : across > boxes ? boxes : across;
  p.turns = (int)((boxes + across - 1) / across);
  p.strips = (int)((boxes + p.turns - 1) / p.turns);
  if (pieces * p.strips > INT32_MAX) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)(pieces * p.strips));
  c.blockDim = dim3(kAll);
  c.dynamicSmemBytes = L::kSmem;
  c.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  c.attrs = at;
  c.numAttrs = 1;
  e = cudaLaunchKernelEx(&c, k, p, my, mw);
  note_launch();
  return e;
}

template <class TY, bool CI>
cudaError_t by_rank(const ExpandArgs& p, cudaStream_t s) {
  const int r = p.a.max_rank;
  return r <= 16 ? launch<TY, CI, 16>(p, s) : r <= 32 ? launch<TY, CI, 32>(p, s)
                                                      : launch<TY, CI, 64>(p, s);
}

}  // namespace

cudaError_t launch_lora_expand_tc(const ExpandArgs& p, bool columns_inner, int y_bf16,
                                  cudaStream_t s) {
  if (y_bf16) return columns_inner ? by_rank<bf16, true>(p, s) : by_rank<bf16, false>(p, s);
  return columns_inner ? by_rank<float, true>(p, s) : by_rank<float, false>(p, s);
}

}  // namespace gptq
