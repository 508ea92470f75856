// The block-scaled FP8 quantisers and the GELU's backward pass from an 8-bit
// checkpoint (format: rbq_fp8.cuh).
//
//   quantize_fp8:          codes[t, k] = E4M3(h[t, k] / s[t, k / 128]), h = x or GELU(x)
//   quantize_weights_fp8:  codes[n, k] = E4M3(w[n, k] / s[n / 128, k / 128])
//   gelu_backward_fp8:     dx = dh * (Phi(x) + x phi(x)), x = code * s
//
// One pass over the inputs, each value held in registers between the block's
// maximum and its rounding.  Of the copy rate (6.57 TB/s): plain rows of 16384
// BF16 0.99 (4096 of them 30 us), weights in both layouts 0.94 (16384 x 4096
// 43 us), the GELU's backward pass with codes 0.99 (4096 x 16384 62 us); GELU and
// checkpoint 0.87 (32760 x 8960 207 us), bound by instructions: 17 a value, 68 %
// of the issue slots.

#include <cuda_runtime.h>

#include <utility>

#include "rbq_fp8.cuh"
#include "rbq_internal.h"
#include "rbq_sm100.cuh"

namespace rbq {
namespace fp8 {
namespace {

using sm100::griddep_launch_dependents;
using sm100::griddep_wait;

// The row kernels: a thread holds 32 consecutive values of a row (of which the
// second 16 may lie behind its end: d is a multiple of 16), and the 4 threads
// of a block of 128 find its maximum by shuffles.  What a thread does besides
// its values (its place, shuffles, scales) is paid half as often as with 16
// values: 32760 x 8960 with GELU and checkpoint took 243 us with 16 values, 223
// with 32 in CTAs of 256 threads and 207 in CTAs of 128, eight to an SM.
constexpr int kVals = 32;
constexpr int kRowThreads = 128, kRowCtas = 8;
constexpr int kLanesPerBlock = kBlock / kVals;
constexpr int kBlocksPerCta = kRowThreads / kLanesPerBlock;
constexpr int kWeightThreads = 256;
// CTAs of the weights' kernel to an SM: as many as its registers allow without
// spilling (fp32, both layouts, 16384 x 4096: 62 us with three, 65 with two, 88
// with four; BF16 44 with four or five, 49 with six).
template <typename T>
constexpr int kWeightCtas = sizeof(T) == 2 ? 4 : 3;
constexpr uint32_t kNaN = 0x7FFFFFFFu;

// ---- pairs of fp32 in one 64-bit register, for the packed FMA ------------------
using f2 = unsigned long long;
__device__ __forceinline__ f2 pack(float lo, float hi) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack(f2 v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f2 both(float v) { return pack(v, v); }
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// ---- loads and stores -----------------------------------------------------------
// 32 bytes in one instruction where the address allows it (`wide`), two of 16 elsewhere.
__device__ __forceinline__ void load32(const void* src, bool wide, uint32_t* w) {
  if (wide) {
    asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
                 : "l"(src));
  } else {
    const uint4 a = static_cast<const uint4*>(src)[0], b = static_cast<const uint4*>(src)[1];
    w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w;
    w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
  }
}
__device__ __forceinline__ void store32(void* dst, bool wide, const uint32_t* w) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]),
                 "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    static_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
    static_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

// V values of a row as they are stored: words of two BF16 or of one fp32.
template <typename T, int V>
struct Piece {
  static constexpr bool kF32 = sizeof(T) == 4;
  static constexpr int kPairs = V / 2, kHalfWords = kF32 ? 16 : 8, kWords = V / 16 * kHalfWords;
  uint32_t w[kWords];

  // The first `n` values (a multiple of 16); the others are 0.
  __device__ __forceinline__ void load(const T* src, int n, bool wide) {
#pragma unroll
    for (int h = 0; h < V / 16; ++h) {
      uint32_t* u = w + h * kHalfWords;
      if (16 * h < n) {
        load32(src + 16 * h, wide, u);
        if constexpr (kF32) load32(src + 16 * h + 8, wide, u + 8);
      } else {
#pragma unroll
        for (int i = 0; i < kHalfWords; ++i) u[i] = 0u;
      }
    }
  }
  __device__ __forceinline__ f2 pair(int i) const {
    if constexpr (kF32)
      return pack(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    else
      return pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
  }
  // Largest magnitude; NaN is passed over.
  __device__ __forceinline__ float amax() const {
    if constexpr (kF32) {
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < V; i += 2)
        m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[i])), fabsf(__uint_as_float(w[i + 1]))));
      return m;
    } else {
      __nv_bfloat162 m = __habs2(two(0));
#pragma unroll
      for (int i = 1; i < kWords; ++i) m = __hmax2(m, __habs2(two(i)));
      return fmaxf(fmaxf(__low2float(m), __high2float(m)), 0.f);
    }
  }
  __device__ __forceinline__ void drop_infinities() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (kF32) {
        if ((w[i] & 0x7FFFFFFFu) == 0x7F800000u) w[i] = kNaN;
      } else {
        if ((w[i] & 0x7FFFu) == 0x7F80u) w[i] |= 0x7Fu;
        if ((w[i] & 0x7FFF0000u) == 0x7F800000u) w[i] |= 0x7F0000u;
      }
    }
  }

 private:
  __device__ __forceinline__ __nv_bfloat162 two(int i) const { return *reinterpret_cast<const __nv_bfloat162*>(&w[i]); }
};
// V values as pairs of fp32.
template <int V>
struct Pairs {
  static constexpr int kPairs = V / 2;
  f2 v[kPairs];
  __device__ __forceinline__ f2 pair(int i) const { return v[i]; }
  __device__ __forceinline__ float amax() const {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      float a, b;
      unpack(v[i], a, b);
      m = fmaxf(m, fmaxf(fabsf(a), fabsf(b)));
    }
    return m;
  }
  __device__ __forceinline__ void drop_infinities() {
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      float a, b;
      unpack(v[i], a, b);
      if (fabsf(a) == INFINITY) a = __uint_as_float(kNaN);
      if (fabsf(b) == INFINITY) b = __uint_as_float(kNaN);
      v[i] = pack(a, b);
    }
  }
};

// Maximum over the threads of a block (every lane of the warp takes part).
__device__ __forceinline__ float block_max(float m) {
#pragma unroll
  for (int o = kLanesPerBlock / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// The scale byte of the block this thread's values belong to.  An infinity
// has no E4M3 value: it becomes NaN (and so reaches the result) and does not
// count for the maximum, which would otherwise flush its 127 neighbours.
template <typename V>
__device__ __forceinline__ uint32_t block_scale(V& x) {
  float m = block_max(x.amax());
  if (__any_sync(0xffffffffu, m == INFINITY)) {
    x.drop_infinities();
    m = block_max(x.amax());
  }
  return scale_byte(m);
}

template <typename V>
__device__ __forceinline__ void encode(const V& x, float inv, uint32_t (&w)[V::kPairs / 2]) {
  const f2 k = both(inv);
#pragma unroll
  for (int j = 0; j < V::kPairs / 2; ++j) {
    float a, b, c, d;
    unpack(mul2(x.pair(2 * j), k), a, b);
    unpack(mul2(x.pair(2 * j + 1), k), c, d);
    w[j] = encode4(a, b, c, d);
  }
}

// ---- the GELU --------------------------------------------------------------------
// Phi(-z) = 2^Q(z), z = |x|: Q is a polynomial of degree 8, fitted here to
// log2 Phi(-z) on [0, 7] by iteratively reweighted least squares so that the
// largest of |error| / max(Phi(-z), 1e-5) is least.  With q evaluated in fp32
// and an exact exponential, |error of Phi| <= 8e-8 everywhere, and 9e-4 of
// Phi(-z) itself to z = 5, 4.2e-3 to z = 7 (an E4M3 code's half step is 6e-2);
// beyond, it falls below 2e-12 and on to 0.  ex2.approx adds 2^-22 of Phi(-z),
// the last FMA of the GELU 2^-24 of the result: in all at most 2.2e-7 |x| for x
// Phi(x), and with the second exponential 3.3e-7 for its slope while |x| <= 16.
// One exponential and no reciprocal: with erf's usual rational
// approximation the kernel was bound by its instructions (38 a value).
//
// Everything works on n = -|x| (so the odd coefficients' signs are turned),
// two values to an instruction.
__device__ __forceinline__ f2 normal_tail(f2 n) {
  f2 q = fma2(both(-8.438778991e-07f), n, both(-1.533665090e-05f));
  q = fma2(q, n, both(-7.393999113e-05f));
  q = fma2(q, n, both(3.969362006e-04f));
  q = fma2(q, n, both(7.381424308e-03f));
  q = fma2(q, n, both(5.269747227e-02f));
  q = fma2(q, n, both(-4.591485262e-01f));
  q = fma2(q, n, both(1.151111722e+00f));
  q = fma2(q, n, both(-9.999998808e-01f));
  float a, b;
  unpack(q, a, b);
  return pack(ex2(a), ex2(b));
}
__device__ __forceinline__ float minus_abs(float x) { return __uint_as_float(__float_as_uint(x) | 0x80000000u); }
// x Phi(x) = max(x, 0) - |x| Phi(-|x|)
__device__ __forceinline__ f2 gelu(f2 x) {
  float a, b;
  unpack(x, a, b);
  const f2 n = pack(minus_abs(a), minus_abs(b));
  return fma2(n, normal_tail(n), pack(fmaxf(a, 0.f), fmaxf(b, 0.f)));
}
// d/dx x Phi(x) = Phi(x) + x phi(x), phi(x) = exp(-x^2 / 2) / sqrt(2 pi):
// g = Phi(-|x|) - |x| phi(x) for x < 0, 1 - g for x >= 0.
__device__ __forceinline__ f2 gelu_slope(f2 x) {
  float a, b;
  unpack(x, a, b);
  const f2 n = pack(minus_abs(a), minus_abs(b));
  // log2 phi = -x^2 log2(e) / 2 - log2(2 pi) / 2
  float u, v;
  unpack(fma2(mul2(x, both(-0.72134752044f)), x, both(-1.32574806473f)), u, v);
  const f2 g = fma2(n, pack(ex2(u), ex2(v)), normal_tail(n));
  float g0, g1, h0, h1;
  unpack(g, g0, g1);
  unpack(fma2(g, both(-1.0f), both(1.0f)), h0, h1);
  return pack(a >= 0.f ? h0 : g0, b >= 0.f ? h1 : g1);
}

// ---- where a block's threads work ----------------------------------------------------
struct Rows {
  long long total;        // blocks of 128 in all
  int d, kbs;
  uint32_t mul;           // b / kbs = (b mul) >> shift for b < 2^31
  int shift;
  int wide;               // 32-byte accesses to the 16-bit (or fp32) rows
  int wide_codes;         // ... and to the codes
};
struct Place {
  long long off, so;      // this thread's first value, the block's scale
  int n;                  // its values: 32, 16 or none
  bool lead;
};
__device__ __forceinline__ Place place(const Rows& r) {
  const long long b = static_cast<long long>(blockIdx.x) * kBlocksPerCta + threadIdx.x / kLanesPerBlock;
  const long long row = r.total <= 0x7FFFFFFFll - kBlocksPerCta
                            ? static_cast<long long>((static_cast<unsigned long long>(b) * r.mul) >> r.shift)
                            : b / r.kbs;
  const int sub = threadIdx.x % kLanesPerBlock;
  const int col = static_cast<int>(b - row * r.kbs) * kBlock + sub * kVals;
  Place p;
  p.n = b < r.total ? min(max(r.d - col, 0), kVals) : 0;          // the last block of a row may be short
  p.lead = sub == 0 && b < r.total;
  p.off = row * r.d + col;
  p.so = b;
  return p;
}
__device__ __forceinline__ void store_codes(uint8_t* dst, const Place& p, const Rows& r, const uint32_t (&w)[8]) {
  if (p.n == kVals)
    store32(dst + p.off, r.wide_codes, w);
  else if (p.n)
    *reinterpret_cast<uint4*>(dst + p.off) = make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T, bool GELU, bool CKPT>
__global__ void __launch_bounds__(kRowThreads, sizeof(T) == 2 ? kRowCtas : kRowCtas - 2)
    quantize_fp8_kernel(const T* X, const Rows r, uint8_t* codes, uint8_t* scales, uint8_t* xcodes, uint8_t* xscales) {
  griddep_wait();
  griddep_launch_dependents();
  const Place p = place(r);
  Piece<T, kVals> x;
  x.load(X + p.off, p.n, r.wide);
  Pairs<kVals> h;
  if constexpr (GELU) {
#pragma unroll
    for (int i = 0; i < kVals / 2; ++i) h.v[i] = gelu(x.pair(i));
  }
  uint32_t w[kVals / 4];
  if constexpr (CKPT || !GELU) {
    const uint32_t s = block_scale(x);
    encode(x, inv_scale(s), w);
    store_codes(GELU ? xcodes : codes, p, r, w);
    if (p.lead) (GELU ? xscales : scales)[p.so] = static_cast<uint8_t>(s);
  }
  if constexpr (GELU) {
    const uint32_t s = block_scale(h);
    encode(h, inv_scale(s), w);
    store_codes(codes, p, r, w);
    if (p.lead) scales[p.so] = static_cast<uint8_t>(s);
  }
}

template <bool QUANT>
__global__ void __launch_bounds__(kRowThreads)
    gelu_backward_fp8_kernel(const uint16_t* dH, const uint8_t* xcodes, const uint8_t* xscales, const Rows r,
                             uint16_t* dX, uint8_t* codes, uint8_t* scales) {
  griddep_wait();
  griddep_launch_dependents();
  const Place p = place(r);
  Piece<uint16_t, kVals> g;
  g.load(dH + p.off, p.n, r.wide);
  uint32_t w[kVals / 4] = {};
  if (p.n == kVals) {
    load32(xcodes + p.off, r.wide_codes, w);
  } else if (p.n) {
    const uint4 c = *reinterpret_cast<const uint4*>(xcodes + p.off);
    w[0] = c.x, w[1] = c.y, w[2] = c.z, w[3] = c.w;
  }
  // From 2^-9 * 2^100 on the slope is 0 or 1: larger scales count as 2^100, under
  // which no code overflows (256 * 2^120, of an |x| above 3.29e38, does).
  const uint32_t xb = p.n ? xscales[p.so] : kMinScale;
  const f2 xs = both(scale_value(xb == 255u ? xb : min(xb, 227u)));
#pragma unroll
  for (int i = 0; i < kVals / 2; ++i) {
    const float2 v = decode2(w[i / 2] >> (16 * (i & 1)));
    float a, b;
    unpack(mul2(g.pair(i), gelu_slope(mul2(pack(v.x, v.y), xs))), a, b);
    const __nv_bfloat162 o = __floats2bfloat162_rn(a, b);
    g.w[i] = *reinterpret_cast<const uint32_t*>(&o);        // the codes are those of the BF16 gradient
  }
  if (p.n) store32(dX + p.off, r.wide, g.w);
  if (p.n == kVals) store32(dX + p.off + 16, r.wide, g.w + 8);
  if constexpr (QUANT) {
    const uint32_t s = block_scale(g);
    encode(g, inv_scale(s), w);
    store_codes(codes, p, r, w);
    if (p.lead) scales[p.so] = static_cast<uint8_t>(s);
  }
}

// One CTA per 128 x 128 block: thread (row t / 8 + 32 i, columns 16 (t % 8))
// holds 4 x 16 values as they were loaded.  The transposed codes go through
// shared memory: row n's 16-byte piece c is kept at piece c ^ (n / 16), so that
// both the 16-byte writes (a row per 8 lanes) and the word reads of the
// transposition (8 row groups x 4 words per warp) touch all 32 banks once.
template <typename T, bool TRANS>
__global__ void __launch_bounds__(kWeightThreads, kWeightCtas<T>)
    quantize_weights_fp8_kernel(const T* W, int N, int K, int nbs, int kbs, int wide, uint8_t* codes, uint8_t* scales,
                                uint8_t* codes_t, uint8_t* scales_t) {
  __shared__ float wmax[2][kWeightThreads / 32];
  __shared__ __align__(16) uint32_t tile[TRANS ? kBlock * kBlock / 4 : 4];
  griddep_wait();
  griddep_launch_dependents();
  const int kb = blockIdx.x % kbs, nb = blockIdx.x / kbs;
  const int sub = threadIdx.x & 7, r0 = threadIdx.x >> 3;
  const int col = kb * kBlock + sub * 16;
  Piece<T, 16> x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = nb * kBlock + r0 + 32 * i;
    x[i].load(W + static_cast<long long>(row) * K + col, row < N && col < K ? 16 : 0, wide);
  }
  float m = 0.f;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    m = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, x[i].amax());
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    if ((threadIdx.x & 31) == 0) wmax[pass][threadIdx.x >> 5] = m;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kWeightThreads / 32; ++i) m = fmaxf(m, wmax[pass][i]);
    if (m != INFINITY) break;                                    // the same in every thread
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i].drop_infinities();          // as block_scale
  }
  const uint32_t s = scale_byte(m);
  const float inv = inv_scale(s);
  if (threadIdx.x == 0) {
    scales[static_cast<long long>(nb) * kbs + kb] = static_cast<uint8_t>(s);
    if constexpr (TRANS) scales_t[static_cast<long long>(kb) * nbs + nb] = static_cast<uint8_t>(s);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int n = r0 + 32 * i, row = nb * kBlock + n;
    uint32_t w[4];
    encode(x[i], inv, w);
    const uint4 q = make_uint4(w[0], w[1], w[2], w[3]);
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

// The next kernel of the stream may set itself up while this one runs (each
// waits for the one before it to end before it touches memory).
template <typename... P, typename... A>
int launch(void (*kernel)(P...), unsigned grid, int threads, cudaStream_t st, A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? RBQ_OK : cuda_fail(e);
}

Rows make_rows(int T, int d, bool wide, bool wide_codes) {
  Rows r{};
  r.d = d;
  r.kbs = blocks(d);
  r.total = static_cast<long long>(T) * r.kbs;
  // With 2^s >= kbs and mul = ceil(2^(31 + s) / kbs), mul kbs = 2^(31 + s) + e,
  // e < kbs <= 2^s, so for b < 2^31 the quotient's error b e / (kbs 2^(31 + s)) is
  // below 1 / kbs: the shift gives floor(b / kbs).
  int s = 0;
  while ((1ll << s) < r.kbs) ++s;
  r.mul = static_cast<uint32_t>(((1ull << (31 + s)) + r.kbs - 1) / r.kbs);
  r.shift = 31 + s;
  r.wide = wide;
  r.wide_codes = wide_codes && d % 32 == 0;
  return r;
}
// CTAs for `total` blocks, 0 when the grid cannot hold them.
unsigned grid_of(long long total) {
  const long long g = (total + kBlocksPerCta - 1) / kBlocksPerCta;
  return g <= 0x7FFFFFFFll ? static_cast<unsigned>(g) : 0u;
}

template <typename T>
int launch_quantize(const void* X, const Rows& r, bool gelu, uint8_t* codes, uint8_t* scales, uint8_t* xcodes,
                    uint8_t* xscales, cudaStream_t st) {
  const unsigned grid = grid_of(r.total);
  if (!grid) return RBQ_EINVAL;
  const T* x = static_cast<const T*>(X);
  const auto kernel = !gelu    ? quantize_fp8_kernel<T, false, false>
                      : xcodes ? quantize_fp8_kernel<T, true, true>
                               : quantize_fp8_kernel<T, true, false>;
  return launch(kernel, grid, kRowThreads, st, x, r, codes, scales, xcodes, xscales);
}

template <typename T>
int launch_weights(const void* W, int N, int K, uint8_t* codes, uint8_t* scales, uint8_t* codes_t, uint8_t* scales_t,
                   cudaStream_t st) {
  const int nbs = blocks(N), kbs = blocks(K);
  const long long grid = static_cast<long long>(nbs) * kbs;
  if (grid > 0x7FFFFFFFll) return RBQ_EINVAL;
  const T* w = static_cast<const T*>(W);
  const unsigned g = static_cast<unsigned>(grid);
  const int wide = aligned(W, 32);                 // rows are multiples of 32 bytes
  const auto kernel = codes_t ? quantize_weights_fp8_kernel<T, true> : quantize_weights_fp8_kernel<T, false>;
  return launch(kernel, g, kWeightThreads, st, w, N, K, nbs, kbs, wide, codes, scales, codes_t, scales_t);
}

}  // namespace
}  // namespace fp8
}  // namespace rbq

using namespace rbq;

extern "C" int quantize_fp8(const void* X, int dtype, int T, int d, int activation, uint8_t* codes, uint8_t* scales,
                            uint8_t* x_codes, uint8_t* x_scales, void* stream) {
  if ((dtype != RBQ_BF16 && dtype != RBQ_F32) || T < 0 || d <= 0 || d > fp8::kMaxSize || d % 16)
    return RBQ_EINVAL;
  if (activation != RBQ_ACT_NONE && activation != RBQ_ACT_GELU) return RBQ_EINVAL;
  if (!x_codes != !x_scales || (x_codes && activation == RBQ_ACT_NONE)) return RBQ_EINVAL;
  if (T == 0) return RBQ_OK;
  if (!X || !codes || !scales) return RBQ_EINVAL;
  if (!aligned(X, 16) || !aligned(codes, 16) || (x_codes && !aligned(x_codes, 16))) return RBQ_EALIGN;
  const fp8::Rows r = fp8::make_rows(T, d, aligned(X, 32), aligned(codes, 32) && (!x_codes || aligned(x_codes, 32)));
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const bool gelu = activation == RBQ_ACT_GELU;
  return dtype == RBQ_BF16
             ? fp8::launch_quantize<uint16_t>(X, r, gelu, codes, scales, x_codes, x_scales, st)
             : fp8::launch_quantize<float>(X, r, gelu, codes, scales, x_codes, x_scales, st);
}

extern "C" int quantize_weights_fp8(const void* W, int dtype, int N, int K, uint8_t* codes, uint8_t* scales,
                                    uint8_t* codes_t, uint8_t* scales_t, void* stream) {
  if ((dtype != RBQ_BF16 && dtype != RBQ_F32) || N < 0 || N > fp8::kMaxSize || K <= 0 || K > fp8::kMaxSize || K % 16)
    return RBQ_EINVAL;
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
  if (T < 0 || d <= 0 || d > fp8::kMaxSize || d % 16 || !codes != !scales) return RBQ_EINVAL;
  if (T == 0) return RBQ_OK;
  if (!dH || !x_codes || !x_scales || !dX) return RBQ_EINVAL;
  if (!aligned(dH, 16) || !aligned(x_codes, 16) || !aligned(dX, 16) || (codes && !aligned(codes, 16)))
    return RBQ_EALIGN;
  const fp8::Rows r = fp8::make_rows(T, d, aligned(dH, 32) && aligned(dX, 32),
                                     aligned(x_codes, 32) && (!codes || aligned(codes, 32)));
  const unsigned grid = fp8::grid_of(r.total);
  if (!grid) return RBQ_EINVAL;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const auto kernel = codes ? fp8::gelu_backward_fp8_kernel<true> : fp8::gelu_backward_fp8_kernel<false>;
  return fp8::launch(kernel, grid, fp8::kRowThreads, st, dH, x_codes, x_scales, r, dX, codes, scales);
}
