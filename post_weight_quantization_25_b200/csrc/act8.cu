// Activations in 8 bits with one scale per row or per group of columns.
//
// Quantizing reads x once and writes a byte per element, so it is bound by
// HBM as long as the arithmetic stays near 5 instructions an element.  The
// definition rounds the exact quotient x / scale, ties to even.  With
// y = RN(1 / scale) the value fma(x, y, 1.5 2^23) is x y rounded to an
// integer, its low byte is the code, and x y is within 127 2^-23 of the
// quotient.  So only a quotient that seems to lie within 1e-4 of a tie can be
// on the wrong side; those are decided by the remainder x - r scale, which a
// fused multiply-add gives exactly (|x| < 1.01 (r + 1/2) scale, so it has at
// most 24 bits).
//
// Measured on 8192 x 28672 bf16: quantizing 186 us, 3.8 TB/s, half of it the ten
// instructions an element; restoring 123 us, 5.8 TB/s.
//
// A group of 32 .. 1024 columns is held by 4 .. 32 lanes in registers (8
// columns a lane and step), wider groups and whole rows by a CTA that reads
// them a second time from the caches.
#include <cuda_runtime.h>

#include "lora_mma.cuh"

namespace gptq {
namespace {

constexpr float kMagic = 12582912.f;  // 1.5 * 2^23

__device__ __forceinline__ void raw_floats(const Raw<bf16, 8>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(r.w[i] << 16);
    v[2 * i + 1] = __uint_as_float(r.w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ void raw_floats(const Raw<float, 8>& r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = r.w[i];
}

// max |x| as the bits of a float: bits of magnitudes order like the values,
// infinity and NaN above every finite one.
template <class TX>
__device__ __forceinline__ uint32_t max_bits(const Raw<TX, 8>& r, uint32_t m) {
  float v[8];
  raw_floats(r, v);
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
  return m;
}
__device__ __forceinline__ float scale_of(uint32_t bits) {
  return bits >= 0x7f800000u ? __uint_as_float(0x7fffffffu)
                             : fmaxf(__fdiv_rn(__uint_as_float(bits), 127.f), 0x1p-126f);
}

// The exactly rounded quotient where q = r + d seems next to a tie
__device__ __noinline__ float resolve(float x, float sc, float r) {
  // exact, and so is its double (half of a scale next to 2^-126 may not be a
  // value)
  const float e = 2.f * fmaf(-r, sc, x);
  if (fabsf(e) > sc || (fabsf(e) == sc && ((int)r & 1))) r += e > 0.f ? 1.f : -1.f;
  return r;
}

template <class TX>
__device__ __forceinline__ void quantize8(const Raw<TX, 8>& r, float sc, float inv, int8_t* out,
                                          int valid, bool vec) {
  float v[8];
  raw_floats(r, v);
  uint32_t t[8];
  bool near = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float s = fmaf(v[i], inv, kMagic);
    t[i] = __float_as_uint(s);
    near |= fabsf(fmaf(v[i], inv, kMagic - s)) > 0.4999f;
  }
  if (near) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float n = __uint_as_float(t[i]) - kMagic;
      if (fabsf(fmaf(v[i], inv, -n)) > 0.4999f)
        t[i] = __float_as_uint(resolve(v[i], sc, n) + kMagic);
    }
  }
  if (!(sc < INFINITY)) {  // NaN scale: codes 0
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = 0;
  }
  uint2 o;
  o.x = __byte_perm(__byte_perm(t[0], t[1], 0x0040), __byte_perm(t[2], t[3], 0x0040), 0x5410);
  o.y = __byte_perm(__byte_perm(t[4], t[5], 0x0040), __byte_perm(t[6], t[7], 0x0040), 0x5410);
  if (valid >= 8 && vec) {
    *reinterpret_cast<uint2*>(out) = o;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < valid) out[i] = (int8_t)((i < 4 ? o.x : o.y) >> (8 * (i & 3)));
  }
}

struct Act8Args {
  const void* x;
  int64_t rows, ldx;
  int n, group, G;
  int8_t* codes;
  int64_t ldc;
  float* scales;
  int vec_x, vec_c;
};

// Columns 1024 w .. of a row belong to warp w of it, four loads of 256 columns
// in flight.  A group is LG lanes of S of the loads: S = 1 and 32 / LG groups a
// load, or one group of 256 S columns.
constexpr int kLoads = 4;
template <class TX, int LG, int S>
__global__ void __launch_bounds__(256) act8_quantize_kernel(const Act8Args p, int warps_per_row) {
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int64_t row = w / warps_per_row;
  if (row >= p.rows) return;
  const int lane = threadIdx.x & 31;
  const int c0 = (int)(w - row * warps_per_row) * 256 * kLoads;
  const TX* x = static_cast<const TX*>(p.x) + row * p.ldx;
  Raw<TX, 8> r[kLoads];
#pragma unroll
  for (int s = 0; s < kLoads; ++s) {
    const int c = c0 + 256 * s + 8 * lane;
    raw_load(r[s], x + c, p.n - c, p.vec_x);
  }
  int8_t* out = p.codes + row * p.ldc;
#pragma unroll
  for (int g = 0; g < kLoads; g += S) {
    const int first = c0 + 256 * g + 8 * lane;
    uint32_t m = 0;
#pragma unroll
    for (int s = 0; s < S; ++s) m = max_bits(r[g + s], m);
    if constexpr (LG == 32) {
      m = __reduce_max_sync(~0u, m);
    } else {
#pragma unroll
      for (int o = LG / 2; o; o >>= 1) m = max(m, __shfl_xor_sync(~0u, m, o));
    }
    const float sc = scale_of(m);
    const float inv = __frcp_rn(sc);
    if (lane % LG == 0 && first < p.n) p.scales[row * p.G + first / (S * 8 * LG)] = sc;
#pragma unroll
    for (int s = 0; s < S; ++s) {
      const int c = first + 256 * s;
      quantize8(r[g + s], sc, inv, out + c, p.n - c, p.vec_c);
    }
  }
}

// One CTA per row and group of any width.
template <class TX>
__global__ void __launch_bounds__(256) act8_quantize_wide_kernel(const Act8Args p) {
  const int64_t row = blockIdx.x / p.G;
  const int g = (int)(blockIdx.x - row * p.G);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c0 = g * p.group, c1 = min(c0 + p.group, p.n);
  const TX* x = static_cast<const TX*>(p.x) + row * p.ldx;
  uint32_t m = 0;
#pragma unroll 4
  for (int c = c0 + 8 * threadIdx.x; c < c1; c += 2048) {
    Raw<TX, 8> r;
    raw_load(r, x + c, c1 - c, p.vec_x);
    m = max_bits(r, m);
  }
  m = __reduce_max_sync(~0u, m);
  __shared__ uint32_t s_m[8];
  if (lane == 0) s_m[warp] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, s_m[i]);
  const float sc = scale_of(m);
  const float inv = __frcp_rn(sc);
  if (threadIdx.x == 0) p.scales[row * p.G + g] = sc;
#pragma unroll 2
  for (int c = c0 + 8 * threadIdx.x; c < c1; c += 2048) {
    Raw<TX, 8> r;
    raw_load(r, x + c, c1 - c, p.vec_x);
    quantize8(r, sc, inv, p.codes + row * p.ldc + c, c1 - c, p.vec_c);
  }
}

// out = scale code: 8 columns a thread and step, U steps in flight.  A signed
// byte b as a float: the bits 0x4b000000 | (b ^ 0x80) are 2^23 + 128 + b.
template <class TO, int U>
__global__ void __launch_bounds__(256)
    act8_dequant_kernel(const int8_t* __restrict__ codes, int64_t rows, int n, int64_t ldc,
                        const float* __restrict__ scales, int group, int G, TO* __restrict__ out,
                        int64_t ldo, int vec_c, int vec_o, int chunks) {
  const int64_t b = blockIdx.x;
  const int64_t row = b / chunks;
  const int c0 = (int)(b - row * chunks) * 2048 * U + 8 * threadIdx.x;
  uint2 w[U];
  float sc[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = c0 + 2048 * u;
    w[u] = make_uint2(0, 0);
    sc[u] = 0.f;
    if (c >= n) continue;
    sc[u] = __ldg(scales + row * G + c / group);
    const int8_t* p = codes + row * ldc + c;
    if (vec_c && c + 8 <= n) {
      w[u] = __ldg(reinterpret_cast<const uint2*>(p));
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < n) {
          const uint32_t v = (uint32_t)(uint8_t)__ldg(p + i) << (8 * (i & 3));
          if (i < 4) w[u].x |= v; else w[u].y |= v;
        }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int c = c0 + 2048 * u;
    if (c >= n) continue;
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t word = (i < 4 ? w[u].x : w[u].y) ^ 0x80808080u;
      v[i] = (__uint_as_float(__byte_perm(word, 0x4b000000u, 0x7540 | (i & 3))) - 8388736.f) *
             sc[u];
    }
    TO* o = out + row * ldo + c;
    if (vec_o && c + 8 <= n) {
      if constexpr (sizeof(TO) == 2) {
        uint4 h;
        uint32_t* hw = reinterpret_cast<uint32_t*>(&h);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
          memcpy(hw + i, &t, 4);
        }
        *reinterpret_cast<uint4*>(o) = h;
      } else {
        reinterpret_cast<float4*>(o)[0] = make_float4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<float4*>(o)[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < n) o[i] = from_f32<TO>(v[i]);
    }
  }
}

template <class TX, int LG, int S>
cudaError_t quantize(const Act8Args& p, cudaStream_t s) {
  const int wpr = (p.n + 256 * kLoads - 1) / (256 * kLoads);
  const int64_t blocks = (p.rows * wpr + 7) / 8;
  if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
  act8_quantize_kernel<TX, LG, S><<<(unsigned)blocks, 256, 0, s>>>(p, wpr);
  note_launch();
  return cudaGetLastError();
}

template <class TX>
cudaError_t quantize_any(const Act8Args& p, cudaStream_t s) {
  switch (p.group) {
    case 32: return quantize<TX, 4, 1>(p, s);
    case 64: return quantize<TX, 8, 1>(p, s);
    case 128: return quantize<TX, 16, 1>(p, s);
    case 256: return quantize<TX, 32, 1>(p, s);
    case 512: return quantize<TX, 32, 2>(p, s);
    case 1024: return quantize<TX, 32, 4>(p, s);
    default: break;
  }
  if (p.rows * p.G > INT32_MAX) return cudaErrorInvalidConfiguration;
  act8_quantize_wide_kernel<TX><<<(unsigned)(p.rows * p.G), 256, 0, s>>>(p);
  note_launch();
  return cudaGetLastError();
}

template <class TO, int U>
cudaError_t dequant(const int8_t* codes, int64_t rows, int64_t n, int64_t ldc, const float* scales,
                    int64_t gs, int64_t G, TO* out, int64_t ldo, cudaStream_t s) {
  const int64_t chunks = (n + 2048 * U - 1) / (2048 * U);
  if (rows * chunks > INT32_MAX) return cudaErrorInvalidConfiguration;
  act8_dequant_kernel<TO, U><<<(unsigned)(rows * chunks), 256, 0, s>>>(
      codes, rows, (int)n, ldc, scales, (int)gs, (int)G, out, ldo, rows_aligned(codes, ldc, 0, 1, 8),
      rows_aligned(out, ldo, 0, sizeof(TO), 16), (int)chunks);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_quantize_act8(const void* x, int x_bf16, int64_t rows, int64_t n, int64_t ldx,
                                 int group, int8_t* codes, int64_t ldc, float* scales,
                                 cudaStream_t s) {
  const int64_t gs = group > 0 ? group : n;
  const Act8Args p = {x, rows, ldx, (int)n, (int)gs, (int)((n + gs - 1) / gs), codes, ldc, scales,
                      rows_aligned(x, ldx, 0, x_bf16 ? 2 : 4, 16), rows_aligned(codes, ldc, 0, 1, 8)};
  return x_bf16 ? quantize_any<bf16>(p, s) : quantize_any<float>(p, s);
}

cudaError_t launch_dequant_act8(const int8_t* codes, int64_t rows, int64_t n, int64_t ldc,
                                const float* scales, int group, void* out, int out_bf16,
                                int64_t ldo, cudaStream_t s) {
  const int64_t gs = group > 0 ? group : n, G = (n + gs - 1) / gs;
  if (out_bf16)
    return dequant<bf16, 2>(codes, rows, n, ldc, scales, gs, G, static_cast<bf16*>(out), ldo, s);
  return dequant<float, 2>(codes, rows, n, ldc, scales, gs, G, static_cast<float*>(out), ldo, s);
}

}  // namespace gptq
