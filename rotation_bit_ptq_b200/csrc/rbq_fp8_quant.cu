// The block-scaled FP8 quantisers and the GELU's backward pass from an 8-bit
// checkpoint (format: rbq_fp8.cuh).
//
//   quantize_fp8:          codes[t, k] = E4M3(h[t, k] / s[t, k / 128]), h = x or GELU(x)
//   quantize_weights_fp8:  codes[n, k] = E4M3(w[n, k] / s[n / 128, k / 128])
//   gelu_backward_fp8:     dx = dh * (Phi(x) + x phi(x)), x = code * s
//
// All three are bound by HBM: one pass over their inputs, each value held in
// registers between the block's maximum and its rounding.

#include <cuda_runtime.h>

#include "rbq_fp8.cuh"
#include "rbq_internal.h"

namespace rbq {
namespace fp8 {
namespace {

// A thread holds 16 consecutive values of a row (d is a multiple of 16); the
// 8 threads of a block of 128 find its maximum by shuffles.
constexpr int kVals = 16;
constexpr int kLanesPerBlock = kBlock / kVals;
constexpr int kThreads = 256;
constexpr int kBlocksPerCta = kThreads / kLanesPerBlock;

// Eight / sixteen values of `src` (16-byte aligned) as fp32.
__device__ __forceinline__ void load16(const uint16_t* src, float (&x)[kVals]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const uint4 v = reinterpret_cast<const uint4*>(src)[j];
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[8 * j + 2 * i] = __uint_as_float(w[i] << 16);
      x[8 * j + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
}
__device__ __forceinline__ void load16(const float* src, float (&x)[kVals]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 v = reinterpret_cast<const float4*>(src)[j];
    x[4 * j] = v.x;
    x[4 * j + 1] = v.y;
    x[4 * j + 2] = v.z;
    x[4 * j + 3] = v.w;
  }
}

__device__ __forceinline__ float amax16(const float (&x)[kVals]) {
  float m = fabsf(x[0]);
#pragma unroll
  for (int i = 1; i < kVals; ++i) m = fmaxf(m, fabsf(x[i]));     // NaN is passed over
  return m;
}
// Maximum over the 8 threads of a block (every lane of the warp takes part).
__device__ __forceinline__ float block_max(float m) {
#pragma unroll
  for (int o = kLanesPerBlock / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// The scale byte of the block this thread's 16 values belong to.  An infinity
// has no E4M3 value: it becomes NaN (and so reaches the result) and does not
// count for the maximum, which would otherwise flush its 127 neighbours.
__device__ __forceinline__ uint32_t block_scale(float (&x)[kVals]) {
  float m = block_max(amax16(x));
  if (__any_sync(0xffffffffu, m == INFINITY)) {
#pragma unroll
    for (int i = 0; i < kVals; ++i)
      if (fabsf(x[i]) == INFINITY) x[i] = __uint_as_float(0x7FFFFFFFu);
    m = block_max(amax16(x));
    if (!(m >= 0.f)) m = 0.f;                                     // nothing but NaN
  }
  return scale_byte(m >= 0.f ? m : 0.f);
}

__device__ __forceinline__ uint4 encode16(const float (&x)[kVals], float inv) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = encode4(x[4 * j] * inv, x[4 * j + 1] * inv, x[4 * j + 2] * inv, x[4 * j + 3] * inv);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Phi(x) and exp(-x^2 / 2): the normal CDF from Abramowitz & Stegun (1964),
// formula 7.1.26 (Hastings' approximation of erf, |error| <= 1.5e-7), which
// shares its exponential with the density.
__device__ __forceinline__ void normal_cdf(float x, float& cdf, float& e) {
  const float z = fabsf(x) * 0.70710678118654752f;
  const float t = __fdividef(1.0f, fmaf(0.3275911f, z, 1.0f));
  float p = fmaf(t, 1.061405429f, -1.453152027f);
  p = fmaf(t, p, 1.421413741f);
  p = fmaf(t, p, -0.284496736f);
  p = fmaf(t, p, 0.254829592f);
  e = __expf(-z * z);
  const float tail = 0.5f * t * p * e;
  cdf = x >= 0.f ? 1.0f - tail : tail;
}
__device__ __forceinline__ float gelu(float x) {
  float cdf, e;
  normal_cdf(x, cdf, e);
  return x * cdf;
}
// d/dx x Phi(x) = Phi(x) + x phi(x), phi(x) = exp(-x^2 / 2) / sqrt(2 pi).
__device__ __forceinline__ float gelu_slope(float x) {
  float cdf, e;
  normal_cdf(x, cdf, e);
  return fmaf(x * 0.39894228040143268f, e, cdf);
}

// Where a group of 8 threads works: row, block of the row, this thread's
// first column.
struct Place {
  long long row;
  int kb, col;
  bool in;
};
__device__ __forceinline__ Place place(long long total, int d, int kbs) {
  const long long b = static_cast<long long>(blockIdx.x) * kBlocksPerCta + threadIdx.x / kLanesPerBlock;
  Place p;
  p.row = b <= 0xFFFFFFFFll ? static_cast<uint32_t>(b) / static_cast<uint32_t>(kbs) : b / kbs;
  p.kb = static_cast<int>(b - p.row * kbs);
  p.col = p.kb * kBlock + (threadIdx.x % kLanesPerBlock) * kVals;
  p.in = b < total && p.col < d;                    // the last block of a row may be short
  return p;
}

template <typename T, bool GELU, bool CKPT>
__global__ void __launch_bounds__(kThreads) quantize_fp8_kernel(const T* X, long long total, int d, int kbs,
                                                                uint8_t* codes, uint8_t* scales, uint8_t* xcodes,
                                                                uint8_t* xscales) {
  const Place p = place(total, d, kbs);
  const long long off = p.row * d + p.col, so = p.row * kbs + p.kb;
  const bool lead = threadIdx.x % kLanesPerBlock == 0 && p.in;
  float x[kVals] = {};
  if (p.in) load16(X + off, x);
  if constexpr (CKPT) {
    float y[kVals];
#pragma unroll
    for (int i = 0; i < kVals; ++i) y[i] = x[i];
    const uint32_t s = block_scale(y);
    if (p.in) *reinterpret_cast<uint4*>(xcodes + off) = encode16(y, inv_scale(s));
    if (lead) xscales[so] = static_cast<uint8_t>(s);
  }
  if constexpr (GELU) {
#pragma unroll
    for (int i = 0; i < kVals; ++i) x[i] = gelu(x[i]);
  }
  const uint32_t s = block_scale(x);
  if (p.in) *reinterpret_cast<uint4*>(codes + off) = encode16(x, inv_scale(s));
  if (lead) scales[so] = static_cast<uint8_t>(s);
}

template <bool QUANT>
__global__ void __launch_bounds__(kThreads) gelu_backward_fp8_kernel(const uint16_t* dH, const uint8_t* xcodes,
                                                                     const uint8_t* xscales, long long total, int d,
                                                                     int kbs, uint16_t* dX, uint8_t* codes,
                                                                     uint8_t* scales) {
  const Place p = place(total, d, kbs);
  const long long off = p.row * d + p.col, so = p.row * kbs + p.kb;
  float g[kVals] = {};
  if (p.in) {
    load16(dH + off, g);
    const uint4 c = __ldg(reinterpret_cast<const uint4*>(xcodes + off));
    const float s = scale_value(xscales[so]);
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t o[kVals / 2];
#pragma unroll
    for (int i = 0; i < kVals / 2; ++i) {
      const float2 v = decode2(w[i / 2] >> (16 * (i & 1)));
      const __nv_bfloat162 r = __floats2bfloat162_rn(g[2 * i] * gelu_slope(v.x * s), g[2 * i + 1] * gelu_slope(v.y * s));
      o[i] = *reinterpret_cast<const uint32_t*>(&r);
      g[2 * i] = __uint_as_float(o[i] << 16);              // the codes are those of the BF16 gradient
      g[2 * i + 1] = __uint_as_float(o[i] & 0xFFFF0000u);
    }
    uint4* dst = reinterpret_cast<uint4*>(dX + off);
    dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
    dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
  if constexpr (QUANT) {
    const uint32_t s = block_scale(g);
    if (p.in) {
      *reinterpret_cast<uint4*>(codes + off) = encode16(g, inv_scale(s));
      if (threadIdx.x % kLanesPerBlock == 0) scales[so] = static_cast<uint8_t>(s);
    }
  }
}

// One CTA per 128 x 128 block: thread (row t / 8 + 32 i, columns 16 (t % 8))
// holds 4 x 16 values.  The transposed codes go through shared memory: row n's
// 16-byte piece c is kept at piece c ^ (n / 16), so that both the 16-byte
// writes (a row per 8 lanes) and the word reads of the transposition (8 row
// groups x 4 words per warp) touch all 32 banks once.
template <typename T, bool TRANS>
__global__ void __launch_bounds__(kThreads) quantize_weights_fp8_kernel(const T* W, int N, int K, int nbs, int kbs,
                                                                        uint8_t* codes, uint8_t* scales,
                                                                        uint8_t* codes_t, uint8_t* scales_t) {
  __shared__ float wmax[kThreads / 32];
  __shared__ __align__(16) uint32_t tile[TRANS ? kBlock * kBlock / 4 : 4];
  const int kb = blockIdx.x % kbs, nb = blockIdx.x / kbs;
  const int sub = threadIdx.x % kLanesPerBlock, r0 = threadIdx.x / kLanesPerBlock;
  const int col = kb * kBlock + sub * kVals;
  float x[4][kVals];
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = nb * kBlock + r0 + 32 * i;
#pragma unroll
    for (int j = 0; j < kVals; ++j) x[i][j] = 0.f;
    if (row < N && col < K) load16(W + static_cast<long long>(row) * K + col, x[i]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int j = 0; j < kVals; ++j) {
      if (fabsf(x[i][j]) == INFINITY) x[i][j] = __uint_as_float(0x7FFFFFFFu);   // as block_scale
      m = fmaxf(m, fabsf(x[i][j]));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) m = fmaxf(m, wmax[i]);
  const uint32_t s = scale_byte(m);
  const float inv = inv_scale(s);
  if (threadIdx.x == 0) {
    scales[static_cast<long long>(nb) * kbs + kb] = static_cast<uint8_t>(s);
    if constexpr (TRANS) scales_t[static_cast<long long>(kb) * nbs + nb] = static_cast<uint8_t>(s);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = r0 + 32 * i, row = nb * kBlock + n;
    const uint4 q = encode16(x[i], inv);
    if (row < N && col < K) *reinterpret_cast<uint4*>(codes + static_cast<long long>(row) * K + col) = q;
    if constexpr (TRANS) *reinterpret_cast<uint4*>(&tile[n * 32 + 4 * (sub ^ (n >> 4))]) = q;
  }
  if constexpr (TRANS) {
    __syncthreads();
    const int pc = threadIdx.x & 7, w = threadIdx.x >> 3;       // rows 16 pc .. 16 pc + 15, columns 4 w .. 4 w + 3
    const int n0 = nb * kBlock + 16 * pc, k0 = kb * kBlock + 4 * w;
    uint32_t o[4][4];                                            // [column][word of 4 rows]
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      uint32_t a[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = tile[(16 * pc + 4 * q + i) * 32 + ((w & 3) | (4 * ((w >> 2) ^ pc)))];
      const uint32_t t0 = __byte_perm(a[0], a[1], 0x5140), t1 = __byte_perm(a[2], a[3], 0x5140);
      const uint32_t t2 = __byte_perm(a[0], a[1], 0x7362), t3 = __byte_perm(a[2], a[3], 0x7362);
      o[0][q] = __byte_perm(t0, t1, 0x5410);
      o[1][q] = __byte_perm(t0, t1, 0x7632);
      o[2][q] = __byte_perm(t2, t3, 0x5410);
      o[3][q] = __byte_perm(t2, t3, 0x7632);
    }
    if (n0 < N) {                                                // N is a multiple of 16 here
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (k0 + i < K)
          *reinterpret_cast<uint4*>(codes_t + static_cast<long long>(k0 + i) * N + n0) =
              make_uint4(o[i][0], o[i][1], o[i][2], o[i][3]);
    }
  }
}

int launched() {
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? RBQ_OK : cuda_fail(e);
}

// CTAs for `total` blocks, 0 when the grid cannot hold them.
unsigned grid_of(long long total) {
  const long long g = (total + kBlocksPerCta - 1) / kBlocksPerCta;
  return g <= 0x7FFFFFFFll ? static_cast<unsigned>(g) : 0u;
}

template <typename T>
int launch_quantize(const void* X, long long total, int d, bool gelu, uint8_t* codes, uint8_t* scales,
                    uint8_t* xcodes, uint8_t* xscales, cudaStream_t st) {
  const unsigned grid = grid_of(total);
  if (!grid) return RBQ_EINVAL;
  const T* x = static_cast<const T*>(X);
  const int kbs = blocks(d);
  if (gelu && xcodes)
    quantize_fp8_kernel<T, true, true><<<grid, kThreads, 0, st>>>(x, total, d, kbs, codes, scales, xcodes, xscales);
  else if (gelu)
    quantize_fp8_kernel<T, true, false><<<grid, kThreads, 0, st>>>(x, total, d, kbs, codes, scales, nullptr, nullptr);
  else
    quantize_fp8_kernel<T, false, false><<<grid, kThreads, 0, st>>>(x, total, d, kbs, codes, scales, nullptr, nullptr);
  return launched();
}

template <typename T>
int launch_weights(const void* W, int N, int K, uint8_t* codes, uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t,
                   cudaStream_t st) {
  const int nbs = blocks(N), kbs = blocks(K);
  const long long grid = static_cast<long long>(nbs) * kbs;
  if (grid > 0x7FFFFFFFll) return RBQ_EINVAL;
  const T* w = static_cast<const T*>(W);
  const unsigned g = static_cast<unsigned>(grid);
  if (codes_t)
    quantize_weights_fp8_kernel<T, true><<<g, kThreads, 0, st>>>(w, N, K, nbs, kbs, codes, scales, codes_t, scales_t);
  else
    quantize_weights_fp8_kernel<T, false><<<g, kThreads, 0, st>>>(w, N, K, nbs, kbs, codes, scales, nullptr, nullptr);
  return launched();
}

}  // namespace
}  // namespace fp8
}  // namespace rbq

using namespace rbq;

extern "C" int quantize_fp8(const void* X, int dtype, int T, int d, int activation, uint8_t* codes, uint8_t* scales,
                            uint8_t* x_codes, uint8_t* x_scales, void* stream) {
  if ((dtype != RBQ_BF16 && dtype != RBQ_F32) || T < 0 || d <= 0 || d % 16) return RBQ_EINVAL;
  if (activation != RBQ_ACT_NONE && activation != RBQ_ACT_GELU) return RBQ_EINVAL;
  if (!x_codes != !x_scales || (x_codes && activation == RBQ_ACT_NONE)) return RBQ_EINVAL;
  if (T == 0) return RBQ_OK;
  if (!X || !codes || !scales) return RBQ_EINVAL;
  if (!aligned(X, 16) || !aligned(codes, 16) || (x_codes && !aligned(x_codes, 16))) return RBQ_EALIGN;
  const long long total = static_cast<long long>(T) * fp8::blocks(d);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool gelu = activation == RBQ_ACT_GELU;
  return dtype == RBQ_BF16
             ? fp8::launch_quantize<uint16_t>(X, total, d, gelu, codes, scales, x_codes, x_scales, st)
             : fp8::launch_quantize<float>(X, total, d, gelu, codes, scales, x_codes, x_scales, st);
}

extern "C" int quantize_weights_fp8(const void* W, int dtype, int N, int K, uint8_t* codes, uint8_t* scales,
                                    uint8_t* codes_t, uint8_t* scales_t, void* stream) {
  if ((dtype != RBQ_BF16 && dtype != RBQ_F32) || N < 0 || K <= 0 || K % 16) return RBQ_EINVAL;
  if (!codes_t != !scales_t || (codes_t && N % 16)) return RBQ_EINVAL;
  if (N == 0) return RBQ_OK;
  if (!W || !codes || !scales) return RBQ_EINVAL;
  if (!aligned(W, 16) || !aligned(codes, 16) || (codes_t && !aligned(codes_t, 16))) return RBQ_EALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == RBQ_BF16 ? fp8::launch_weights<uint16_t>(W, N, K, codes, scales, codes_t, scales_t, st)
                           : fp8::launch_weights<float>(W, N, K, codes, scales, codes_t, scales_t, st);
}

extern "C" int gelu_backward_fp8(const uint16_t* dH, const uint8_t* x_codes, const uint8_t* x_scales, int T, int d,
                                 uint16_t* dX, uint8_t* codes, uint8_t* scales, void* stream) {
  if (T < 0 || d <= 0 || d % 16 || !codes != !scales) return RBQ_EINVAL;
  if (T == 0) return RBQ_OK;
  if (!dH || !x_codes || !x_scales || !dX) return RBQ_EINVAL;
  if (!aligned(dH, 16) || !aligned(x_codes, 16) || !aligned(dX, 16) || (codes && !aligned(codes, 16)))
    return RBQ_EALIGN;
  const long long total = static_cast<long long>(T) * fp8::blocks(d);
  const unsigned grid = fp8::grid_of(total);
  if (!grid) return RBQ_EINVAL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int kbs = fp8::blocks(d);
  if (codes)
    fp8::gelu_backward_fp8_kernel<true>
        <<<grid, fp8::kThreads, 0, st>>>(dH, x_codes, x_scales, total, d, kbs, dX, codes, scales);
  else
    fp8::gelu_backward_fp8_kernel<false>
        <<<grid, fp8::kThreads, 0, st>>>(dH, x_codes, x_scales, total, d, kbs, dX, nullptr, nullptr);
  return fp8::launched();
}
