// qlinear_fp8_wgrad: the weight gradient of a linear layer from the 8-bit
// codes kept of its input (format: rbq_fp8.cuh).
//
//   dW[n, k] = sum_m dY[m, n] x[m, k],   x[m, k] = code[m, k] 2^(b[m, k/128] - 127)
//
// The sum runs over tokens, and the scales change from token to token along
// it, so they cannot be taken out of the product; but code * scale is exact in
// BF16, so the product runs on BF16 operands (tcgen05 kind::f16, fp32 sums)
// with no rounding besides dY's own.
//
// Two kernels per call (three when the tokens are split):
// 1. decode_rows_kernel: codes and scales -> BF16 [M, K] in a stream-ordered
//    workspace; above 2 GiB, a panel of columns after the other.
// 2. wgrad_kernel: persistent, on CTA pairs, tiles of 256 x 256 or 256 x 128
//    values of dW (cta_group::2), slices of 64 tokens.  Both operands lie with
//    the token as their row, so they are "MN-major": a TMA box of 64 tokens x
//    64 columns (128 bytes, 128B swizzle) is one column of swizzle atoms.
//    Warps 0..3 epilogue, 4 MMA issuer, 5 TMA producer.
// 3. With too few tiles to fill the GPU the tokens are split: each part's sums
//    go to the workspace in fp32 and sum_parts_kernel adds them in order.
//
// 4096 x 16384 x 4096 takes 329 us in a burst (1.67 PFLOP/s, what the library's
// BF16 product reaches; 9 of them the decoding) and 386 us in a row, under the
// power cap; 1560 x 1536 x 1536 11.8 us, bound by L2 and by the two launches.
// (Decoding inside wgrad_kernel, by eight warps from codes that TMA brought, gave
// 14.2 us and 449: they do not keep up with the MMAs.)

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>
#include <utility>

#include "rbq_fp8.cuh"
#include "rbq_internal.h"
#include "rbq_qcodes.cuh"
#include "rbq_sm100.cuh"
#include "rbq_tiles.cuh"

namespace rbq {
namespace fp8 {
namespace {

using namespace sm100;

constexpr int kTok = 64;                   // tokens per slice
constexpr int kTileN = 256;                // rows of dW per tile
constexpr int kHalf = kTileN / 2;          // of them per CTA
constexpr int kBox = 64;                   // columns per TMA box (128 bytes)
constexpr int kBoxBytes = kBox * 2 * kTok; // 8 KB
constexpr int kWThreads = 192;
constexpr int kWMmaWarp = 4, kWTmaWarp = 5;

// Tiles of 256 x BK (256 or 128) values of dW.
template <int BK>
struct Wg {
  static constexpr int kA = kHalf / kBox * kBoxBytes;         // dY: 16 KB per CTA
  static constexpr int kB = BK / 2 / kBox * kBoxBytes;        // x: 16 or 8 KB
  static constexpr int kStage = kA + kB;
  static constexpr int kStages = BK == 256 ? 6 : 8;
  static constexpr uint32_t kTmemCols = 2 * BK;
  // Instruction descriptor: BF16 A and B, both MN-major (bits 15 and 16), fp32 sums.
  static constexpr uint32_t kIdesc = idesc_f16(kTileN, BK, true) | (1u << 15) | (1u << 16);
};
constexpr int kWMaxStages = 8;

// Shared-memory descriptor of an MN-major operand in the 128-byte swizzle
// layout: 64 columns x 8 tokens per swizzle atom; the next 8 tokens 1024
// bytes on (stride offset), the next 64 columns one box on (leading offset).
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(kBoxBytes >> 4) << 16) |
         (static_cast<uint64_t>(1024u >> 4) << 32) | (static_cast<uint64_t>(1u) << 46) |
         (static_cast<uint64_t>(2u) << 61);
}

struct WParams {
  int M, N, K;
  int f32;                    // of the output, [parts, N, K]
  int parts;                  // token ranges, each summed apart
  int order;
  unsigned int* err;
};

struct __align__(8) WTail {
  uint64_t full[kWMaxStages];
  uint64_t empty[kWMaxStages];
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t drain;
  uint32_t tmem_slot;
  volatile uint32_t abort;
};

constexpr int kPiece = 32 * 128;          // bytes of a warp's piece of the output: 32 rows x 64 BF16 or 32 fp32
template <int BK>
constexpr size_t kWSmem = 1024 + Wg<BK>::kStages * Wg<BK>::kStage + 8 * kPiece + sizeof(WTail) + 64;
static_assert(kWSmem<256> <= 227 * 1024 && kWSmem<128> <= 227 * 1024, "fits an SM");

__device__ __forceinline__ void st_v8(void* dst, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Slices [first, last) of part `part`.
__device__ __forceinline__ void part_range(int slices, int parts, int part, int& first, int& last) {
  first = static_cast<int>(static_cast<long long>(slices) * part / parts);
  last = static_cast<int>(static_cast<long long>(slices) * (part + 1) / parts);
}

template <int BK>
__global__ void __launch_bounds__(kWThreads, 1)
    wgrad_kernel(const __grid_constant__ CUtensorMap tmY, const __grid_constant__ CUtensorMap tmX,
                 const __grid_constant__ CUtensorMap tmW, const WParams p) {
  using G = Wg<BK>;
  constexpr int kWStages = G::kStages, kWStage = G::kStage;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* ops = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* pieces = ops + kWStages * kWStage;
  WTail* tl = reinterpret_cast<WTail*>(pieces + 8 * kPiece);
  const int tid = threadIdx.x, warp = warp_number(), lane = tid & 31;
  // clusters are pairs of neighbouring blocks; the compiler knows that these are the same in all threads
  const uint32_t rank = blockIdx.x & 1u;
  const int work0 = static_cast<int>(blockIdx.x >> 1), wstep = static_cast<int>(gridDim.x >> 1);
  const int ntiles_n = (p.N + kTileN - 1) / kTileN, ntiles_k = (p.K + BK - 1) / BK;
  const int ntiles = ntiles_n * ntiles_k, nwork = ntiles * p.parts;
  const int slices = (p.M + kTok - 1) / kTok;
  volatile uint32_t* abort = &tl->abort;
  bool issuer = false;                     // the thread that issues the MMAs

  if (tid == 0) {
    for (int s = 0; s < kWStages; ++s) {
      mbar_init(&tl->full[s], 1);
      mbar_init(&tl->empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tl->acc_full[a], 1);
      mbar_init(&tl->acc_empty[a], 8);
    }
    mbar_init(&tl->drain, 1);
    tl->abort = 0u;
    mbar_fence_init();
  }
  if (warp == kWMmaWarp) {
    tmem_alloc_pair(&tl->tmem_slot, G::kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tl->tmem_slot, 0);
  griddep_wait();
  griddep_launch_dependents();

  if (warp == kWMmaWarp) {
    if (rank == 0) {       // the warp goes through the loop together, one thread issues
      const uint64_t desc0 = sdesc_mn_sw128(smem_u32(ops));
      uint32_t s = 0, ph = 0, it = 0;
      bool ok = true;
      for (int w = work0; w < nwork && ok; w += wstep, ++it) {
        const uint32_t a = it & 1u, use = it >> 1;
        if (use >= 1 && !mbar_warp_wait_cl(&tl->acc_empty[a], (use - 1) & 1, abort)) { ok = false; break; }
        tc_fence_after();
        const uint32_t acc = tmem + a * BK;
        int first, last;
        part_range(slices, p.parts, w / ntiles, first, last);
        for (int t = first; t < last; ++t) {
          if (!mbar_warp_wait(&tl->full[s], ph, abort)) { ok = false; break; }
          tc_fence_after();
          const uint64_t ad = desc0 + ((s * static_cast<uint32_t>(kWStage)) >> 4);
          const uint64_t bd = ad + (G::kA >> 4);
          const uint32_t add = t != first;
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kTok / 16; ++k)          // 16 tokens = two atoms of 8
              umma_f16_pair(acc, ad + k * (2048 >> 4), bd + k * (2048 >> 4), G::kIdesc, k != 0 ? 1u : add);
            umma_commit_pair(&tl->empty[s], 3);
          }
          if (++s == kWStages) { s = 0; ph ^= 1u; }
        }
        if (ok && elect_one()) umma_commit_pair(&tl->acc_full[a], 3);
      }
      if (!ok && lane == 0) atomicOr(p.err, 2u);
      issuer = elect_one();
    }
  } else if (warp == kWTmaWarp) {
    if (elect_one()) {
      tma_prefetch_desc(&tmY);
      tma_prefetch_desc(&tmX);
      uint32_t s = 0, ph = 0;
      bool wrapped = false, ok = true;
      for (int w = work0; w < nwork && ok; w += wstep) {
        int nt, kt, first, last;
        tiles::tile_coords(w % ntiles, ntiles_n, ntiles_k, p.order, nt, kt);
        part_range(slices, p.parts, w / ntiles, first, last);
        const int n0 = nt * kTileN + static_cast<int>(rank) * kHalf, k0 = kt * BK + static_cast<int>(rank) * (BK / 2);
        for (int t = first; t < last; ++t) {
          if (wrapped && !mbar_wait_or_abort(&tl->empty[s], ph ^ 1u, abort)) { ok = false; break; }
          uint8_t* st = ops + s * kWStage;
          if (rank == 0) mbar_arrive_expect_tx(&tl->full[s], 2 * kWStage);
          const uint32_t bar = mapa_shared(&tl->full[s], 0);
#pragma unroll
          for (int b = 0; b < kHalf / kBox; ++b)
            tma_load_2d_pair(st + b * kBoxBytes, &tmY, n0 + b * kBox, t * kTok, bar);
#pragma unroll
          for (int b = 0; b < BK / 2 / kBox; ++b)
            tma_load_2d_pair(st + G::kA + b * kBoxBytes, &tmX, k0 + b * kBox, t * kTok, bar);
          if (++s == kWStages) { s = 0; ph ^= 1u; wrapped = true; }
        }
      }
      if (!ok) atomicOr(p.err, 16u);
    }
  } else {
    // The output leaves by TMA, which writes whole lines and cuts what lies
    // outside: a warp's 32 rows in pieces of 128 bytes, two of them in turn.
    // (Row by lane in 32-byte stores, the 4096 x 16384 gradient of 64 tokens
    // took 48 us in place of 29.)
    uint32_t it = 0, pieces_out = 0;
    const auto put = [&](const uint32_t (&o)[32], int x, int y, int z) {
      uint8_t* piece = pieces + (2 * warp + (pieces_out++ & 1u)) * kPiece;
      if (lane == 0) bulk_wait_read<1>();               // the piece before the last has left
      __syncwarp();
#pragma unroll
      for (int j = 0; j < 8; ++j)
        *reinterpret_cast<uint4*>(piece + sw128_offset(lane, j)) =
            make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tma_store_3d(&tmW, x, y, z, piece);
    };
    for (int w = work0; w < nwork; w += wstep, ++it) {
      const uint32_t a = it & 1u, use = it >> 1;
      if (!mbar_warp_wait(&tl->acc_full[a], use & 1, abort)) {
        if (lane == 0) atomicOr(p.err, 4u);
        break;
      }
      tc_fence_after();
      int nt, kt;
      tiles::tile_coords(w % ntiles, ntiles_n, ntiles_k, p.order, nt, kt);
      const int n0 = nt * kTileN + static_cast<int>(rank) * kHalf + 32 * warp, part = w / ntiles;
#pragma unroll 1
      for (int c = 0; c < BK / 64; ++c) {
        uint32_t u[32], v[32];
        const uint32_t t = tmem + (static_cast<uint32_t>(32 * warp) << 16) + a * BK + 64 * c;
        tmem_ld32(t, u);
        tmem_ld32(t + 32, v);
        tmem_wait_ld();
        const int kc = kt * BK + 64 * c;
        if (n0 >= p.N || kc >= p.K) continue;           // the same in the whole warp
        if (p.f32) {
          put(u, kc, n0, part);
          if (kc + 32 < p.K) put(v, kc + 32, n0, part);
        } else {
          uint32_t o[32];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            o[j] = bf16x2(u[2 * j], u[2 * j + 1]);
            o[16 + j] = bf16x2(v[2 * j], v[2 * j + 1]);
          }
          put(o, kc, n0, part);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_relaxed(mapa_shared(&tl->acc_empty[a], 0));
    }
    if (lane == 0) bulk_wait();
  }

  tc_fence_before();
  __syncthreads();
  if (tl->abort) {
    drain_after_abort(issuer, &tl->drain, true);
    __syncthreads();
  }
  cluster_sync();
  if (warp == kWMmaWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, G::kTmemCols);
  }
}

// Codes and scales -> BF16 values [M, cols], 16 per thread (K and cols are
// multiples of 16); CTA (x, y): 4096 values of each of `rows` rows from row
// `rows` y on.
__global__ void __launch_bounds__(256) decode_rows_kernel(const uint8_t* codes, const uint8_t* scales, int M, int K,
                                                          int kbs, int cols, int rows, uint16_t* out) {
  griddep_wait();
  griddep_launch_dependents();
  const int col = (blockIdx.x * 256 + threadIdx.x) * 16, row0 = blockIdx.y * rows, row1 = min(M, row0 + rows);
  if (col >= cols) return;
#pragma unroll 4
  for (int row = row0; row < row1; ++row) {
    const uint4 c = *reinterpret_cast<const uint4*>(codes + static_cast<long long>(row) * K + col);
    const float s = scale_value(scales[static_cast<long long>(row) * kbs + col / kBlock]);
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
    uint32_t o[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 v = decode2(w[j / 2] >> (16 * (j & 1)));
      const __nv_bfloat162 h = __floats2bfloat162_rn(v.x * s, v.y * s);      // exact
      o[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
    st_v8(out + static_cast<long long>(row) * cols + col, o);       // the workspace and its rows are 32-byte aligned
  }
}

// out = the sum of the parts, n4 groups of four values each (cols4 to a row; a
// row of out is pitch4 long): G groups of threads take every G-th part each, in
// their order, and the groups' sums are added in theirs.  One group where the
// parts are few; eight where they are many and the gradient small, so that
// their loads do not wait for one another (256 x 256 in 27 parts: 9.7 us with
// one group).
template <int G>
__global__ void __launch_bounds__(256) sum_parts_kernel(const float4* parts, int nparts, long long n4,
                                                        unsigned cols4, unsigned pitch4, void* out, int f32) {
  constexpr int kOut = 256 / G;
  __shared__ float4 sums[G > 1 ? 256 : 1];
  griddep_wait();
  griddep_launch_dependents();
  const int g = threadIdx.x / kOut, l = threadIdx.x % kOut;
  const long long i = blockIdx.x * static_cast<long long>(kOut) + l;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  const auto add = [&](const float4& v) {
    s.x += v.x;
    s.y += v.y;
    s.z += v.z;
    s.w += v.w;
  };
  if (i < n4) {
#pragma unroll 8
    for (int q = g; q < nparts; q += G) add(parts[q * n4 + i]);
  }
  if constexpr (G > 1) {
    sums[threadIdx.x] = s;
    __syncthreads();
    if (g) return;
#pragma unroll
    for (int q = 1; q < G; ++q) add(sums[q * kOut + l]);
  }
  if (i >= n4) return;
  long long o = i;
  if (cols4 != pitch4) {                    // i < 2^32: the tiles of all parts fit the GPU at once
    const unsigned r = static_cast<unsigned>(i) / cols4;
    o = static_cast<long long>(r) * pitch4 + (static_cast<unsigned>(i) - r * cols4);
  }
  if (f32) {
    static_cast<float4*>(out)[o] = s;
  } else {
    static_cast<uint2*>(out)[o] = make_uint2(bf16x2(__float_as_uint(s.x), __float_as_uint(s.y)),
                                             bf16x2(__float_as_uint(s.z), __float_as_uint(s.w)));
  }
}

// BF16 [rows, cols] row-major, boxes of 64 rows (tokens) x 64 columns, 128B swizzle.
int encode_tokens_map(CUtensorMap* map, const uint16_t* base, int rows, int cols) {
  auto fn = qfast::encode_fn();
  if (!fn) return RBQ_ECUDA;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {2 * static_cast<cuuint64_t>(cols)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(kBox), static_cast<cuuint32_t>(kTok)};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<uint16_t*>(base), dims, strides, box,
                        estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? RBQ_OK : RBQ_ECUDA;
}

// [parts, N, K] of BF16 or fp32 with rows `pitch` values apart, boxes of 32 rows x 128 bytes, 128B swizzle.
int encode_out_map(CUtensorMap* map, void* base, int parts, int N, int K, int pitch, bool f32) {
  auto fn = qfast::encode_fn();
  if (!fn) return RBQ_ECUDA;
  const cuuint64_t row = (f32 ? 4 : 2) * static_cast<cuuint64_t>(pitch);
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(parts)};
  const cuuint64_t strides[2] = {row, row * static_cast<cuuint64_t>(N)};
  const cuuint32_t box[3] = {f32 ? 32u : 64u, 32, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = fn(map, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims,
                        strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? RBQ_OK : RBQ_ECUDA;
}

// Pairs of wgrad_kernel that can be resident on device `dev`, asked once per device (0: none).
template <int BK>
int wgrad_pairs(int dev) {
  static int cached[kMaxDevices] = {};        // 0 = not yet asked; else pairs + 1
  if (cached[dev]) return cached[dev] - 1;
  if (cudaFuncSetAttribute(wgrad_kernel<BK>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           static_cast<int>(kWSmem<BK>)) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(kWThreads, 1, 1);
  cfg.dynamicSmemBytes = kWSmem<BK>;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, wgrad_kernel<BK>, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  cached[dev] = n + 1;
  return n;
}

// Launches that may set themselves up while the one before them runs (each
// waits for its end before it touches memory); `pair`: clusters of two CTAs.
template <typename... P, typename... A>
int launch(void (*kernel)(P...), dim3 grid, int threads, size_t smem, bool pair, cudaStream_t st, A&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = 2;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pair ? 2 : 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? RBQ_OK : cuda_fail(e);
}

// The width of a tile and the parts the tokens are split into: what takes least
// by a linear model, in ns: `start` a launch, `slice` each 64 tokens or what 17
// TB/s take from L2 for all of them, `wave` each further wave of tiles, and for
// the joint sum 2300, 110 a part and 0.3 per thousand fp32 values moved.  Narrow
// tiles are twice as many, wide ones read dY half as often: 1560 x 1536 x 1536
// takes 12.5 us with 128 (no parts), 15.3 with 256 and 16.8 with 256 in two
// parts; 4096 x 16384 x 4096 320 us with 256, 376 with 128; 4096 x 64 x 128 10.2
// us in 8 parts, 18.3 in one.
// The constants were fitted before the output left by TMA and the parts were
// summed in groups: the model's times are too long where the result's bytes
// count (it says 43 us for 64 x 16384 x 4096, which takes 34), its choice holds.
// Measured on 62 gradients of 16 to 32760 tokens and eight weights of 64 x 128
// to 16384 x 4096, BF16 and fp32, every choice in each: the best or within 7 % of
// it in 118 of 124.  It loses most where the rows of dY and of x both begin off
// 128-byte lines, which it does not count (8000 x 1000 x 1552: 50 us, 40 to 46 with
// 256 in two parts; 8000 x 1024 x 1552 34, 8000 x 1000 x 1536 33).
struct WPlan {
  int BK, parts;
};
WPlan make_wplan(int M, int N, int K, int pairs) {
  const auto up = [](double a, double b) { return std::ceil(a / b); };
  constexpr struct {
    int BK, start, wave, slice;
  } kinds[] = {{256, 4700, 2600, 310}, {128, 3600, 1300, 165}};
  const int slices = (M + kTok - 1) / kTok;
  WPlan best{256, 1};
  double least = -1;
  for (const auto& k : kinds) {
    const double tiles = up(N, 256) * up(K, k.BK), l2 = tiles * slices * ((256 + k.BK) * 2 * kTok) / 17000;
    for (int parts = 1; parts <= slices && (parts == 1 || tiles * parts <= pairs); ++parts) {
      const double waves = up(tiles * parts, pairs);
      const double t = k.start + k.wave * (waves - 1) + std::max(waves * up(slices, parts) * k.slice, l2) +
                       (parts > 1 ? 2300 + 110 * parts + (parts + 1.) * N * K * 3 / 10000 : 0);
      if (least < 0 || t < least) {
        least = t;
        best = {k.BK, parts};
      }
    }
  }
  return best;
}

// dW[:, k0 : k0 + cols] (k0 a multiple of kBlock): the values of those columns of x go through the workspace.
int wgrad_panel(const uint16_t* dY, const uint8_t* codes, const uint8_t* scales, int M, int N, int K, int k0, int cols,
                void* dW, bool f32, unsigned int* err, int dev, cudaStream_t st) {
  codes += k0;
  scales += k0 / kBlock;
  dW = static_cast<uint8_t*>(dW) + static_cast<size_t>(k0) * (f32 ? 4 : 2);
  const int pairs256 = wgrad_pairs<256>(dev), pairs128 = wgrad_pairs<128>(dev);
  if (pairs256 < 1 || pairs128 < 1) return RBQ_ECUDA;
  const WPlan plan = make_wplan(M, N, cols, pairs256);
  const int parts = plan.parts, pairs = plan.BK == 256 ? pairs256 : pairs128;
  const long long ntiles = ((N + kTileN - 1LL) / kTileN) * ((cols + plan.BK - 1LL) / plan.BK);
  if (ntiles * parts > (1 << 28)) return RBQ_EINVAL;

  cudaMemPool_t pool = qfast::workspace_pool(dev);
  if (!pool) return RBQ_ECUDA;
  const size_t x_bytes = (static_cast<size_t>(M) * cols * 2 + 255) / 256 * 256;
  const size_t part_bytes = parts > 1 ? static_cast<size_t>(parts) * N * cols * 4 : 0;
  void* ws = nullptr;
  cudaError_t e = cudaMallocFromPoolAsync(&ws, x_bytes + part_bytes, pool, st);
  if (e != cudaSuccess) return cuda_fail(e);
  uint16_t* x = static_cast<uint16_t*>(ws);
  float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + x_bytes);

  // rows per CTA: while eight CTAs to an SM remain, at most 65535 along y
  const int xs = (cols + 4095) / 4096;
  int rows = 1, sms = 148;
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  while (rows < 8 && static_cast<long long>(xs) * M / (2 * rows) >= 8 * sms) rows *= 2;
  while ((M + rows - 1) / rows > 65535) rows *= 2;
  int rc = launch(decode_rows_kernel, dim3(xs, (M + rows - 1) / rows, 1), 256, 0, false, st, codes, scales, M, K,
                  blocks(K), cols, rows, x);

  WParams p{};
  p.M = M;
  p.N = N;
  p.K = cols;
  p.parts = parts;
  p.f32 = parts > 1 || f32;
  p.order = tiles::tile_order(dev, 2LL * M * N, 2LL * M * cols);
  p.err = err;
  CUtensorMap mY, mX, mW;
  if (rc == RBQ_OK) rc = encode_tokens_map(&mY, dY, M, N);
  if (rc == RBQ_OK) rc = encode_tokens_map(&mX, x, M, cols);
  if (rc == RBQ_OK)
    rc = parts > 1 ? encode_out_map(&mW, part, parts, N, cols, cols, true) : encode_out_map(&mW, dW, 1, N, cols, K, f32);
  if (rc == RBQ_OK) {
    const long long nwork = ntiles * parts;
    const dim3 grid(2 * static_cast<unsigned>(nwork < pairs ? nwork : pairs), 1, 1);
    rc = plan.BK == 256 ? launch(wgrad_kernel<256>, grid, kWThreads, kWSmem<256>, true, st, mY, mX, mW, p)
                        : launch(wgrad_kernel<128>, grid, kWThreads, kWSmem<128>, true, st, mY, mX, mW, p);
  }
  if (rc == RBQ_OK && parts > 1) {
    const long long n4 = static_cast<long long>(N) * cols / 4, per = parts > 4 ? 32 : 256, grid = (n4 + per - 1) / per;
    rc = grid > 0x7FFFFFFFll
             ? RBQ_EINVAL
             : launch(parts > 4 ? sum_parts_kernel<8> : sum_parts_kernel<1>, dim3(static_cast<unsigned>(grid), 1, 1),
                      256, 0, false, st, reinterpret_cast<const float4*>(part), parts, n4,
                      static_cast<unsigned>(cols / 4), static_cast<unsigned>(K / 4), dW, static_cast<int>(f32));
  }
  e = cudaFreeAsync(ws, st);
  if (rc == RBQ_OK && e != cudaSuccess) rc = cuda_fail(e);
  return rc;
}

// x takes twice the room of its codes in the workspace, and the pool keeps what
// it once had: so at most 2 GiB of it at a time, a panel of columns after the
// other.  (131072 x 1024 x 16384 takes 3.9 ms in two panels and 4.1 in one, 70000
// x 1024 x 16384 2.2 and 2.1: within what the power cap's clock moves them.)
constexpr long long kPanelBytes = 2ll << 30;
constexpr int kPanelStep = 256;           // columns of the widest tile, whole scale blocks

int wgrad(const uint16_t* dY, const uint8_t* codes, const uint8_t* scales, int M, int N, int K, void* dW, bool f32,
          unsigned int* err, cudaStream_t st) {
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= kMaxDevices) return RBQ_EINVAL;
  const long long fits = kPanelBytes / (2ll * M) / kPanelStep * kPanelStep;
  const int panel = static_cast<int>(std::min<long long>(K, std::max<long long>(fits, kPanelStep)));
  for (int k0 = 0; k0 < K; k0 += panel) {
    const int rc = wgrad_panel(dY, codes, scales, M, N, K, k0, std::min(panel, K - k0), dW, f32, err, dev, st);
    if (rc != RBQ_OK) return rc;
  }
  return RBQ_OK;
}

}  // namespace
}  // namespace fp8
}  // namespace rbq

using namespace rbq;

extern "C" int qlinear_fp8_wgrad(const uint16_t* dY, const uint8_t* a_codes, const uint8_t* a_scales, int M, int N,
                                 int K, void* dW, int dtype, void* stream) {
  if (M < 0 || M > fp8::kMaxSize || N < 0 || N > fp8::kMaxSize || N % 8 || K <= 0 || K > fp8::kMaxSize || K % 16)
    return RBQ_EINVAL;
  if (dtype != RBQ_BF16 && dtype != RBQ_F32) return RBQ_EINVAL;
  if (N == 0) return RBQ_OK;
  if (!dW) return RBQ_EINVAL;
  if (!aligned(dW, 16)) return RBQ_EALIGN;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (M == 0) {                                   // no tokens: a gradient of zeros
    const cudaError_t e = cudaMemsetAsync(dW, 0, static_cast<size_t>(N) * K * (dtype == RBQ_F32 ? 4 : 2), st);
    return e == cudaSuccess ? RBQ_OK : cuda_fail(e);
  }
  if (!dY || !a_codes || !a_scales) return RBQ_EINVAL;
  if (!aligned(dY, 16) || !aligned(a_codes, 16)) return RBQ_EALIGN;
  unsigned int* err = nullptr;
  const int rc = device_error_word_ptr(&err);
  if (rc != RBQ_OK) return rc;
  return fp8::wgrad(dY, a_codes, a_scales, M, N, K, dW, dtype == RBQ_F32, err, st);
}
