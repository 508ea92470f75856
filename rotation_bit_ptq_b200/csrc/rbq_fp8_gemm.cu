// qlinear_fp8: the linear layer on block-scaled FP8 codes (format: rbq_fp8.cuh).
//
//   Y[m, n] = bf16( sum_k (sa[m, k/128] qa[m, k]) (sw[n/128, k/128] qw[n, k]) )
//
// on tcgen05 kind::mxf8f6f4 with block scales: the tensor core multiplies each
// 32-value slice of K by the two operands' E8M0 scales, held in tensor memory,
// and sums in fp32.  The hardware's block is 32 values, ours 128: the four MMAs
// of a 128-value K slice use the same scale byte, and the four bytes of a
// scale word hold four consecutive K slices (the instruction descriptor picks
// the byte).  The product so runs at the rate of an unscaled FP8 product;
// general fp32 scales would need every partial sum of 128 read back and
// rescaled on the CUDA cores.
//
// Scales reach tensor memory through shared memory: four loader warps gather
// the bytes (a row per thread; four K slices per 32-bit word, four words per
// hand-over) into the 32 x 16 byte blocks tcgen05.cp replicates over the four
// lane quadrants: the word of row r at 16 (r % 32) + 4 (r / 32).
//
// Three kernels, chosen by make_plan.
// 1. fp8_pair_kernel (many tokens): persistent, on CTA pairs, 256 x 256 tiles
//    (cta_group::2), K slices of 128, 6 stages of 32 KB per CTA.  Warps 0..3
//    epilogue, 4 MMA issuer, 5 TMA producer, 6..9 scale loaders.  Two
//    accumulators of 256 columns and the scales' 24 do not fit in the 512
//    columns of tensor memory, so the accumulators overlap in 32 columns,
//    which the epilogue reads first; the next tile's MMAs wait for that read
//    only (800 of a 4096-deep tile's 18050 cycles; 16384 are the MMAs' own).
//    4096 x 16384 x 4096 takes 186 us (2.96 PFLOP/s) in a burst, 219 us in
//    a row, where power sets the pace (1.2 GHz).
// 2. fp8_few_kernel (few tokens): bound by reading the weights.  The weights
//    take the MMA's M side (128 rows), the tokens its N side, and the CTAs of
//    a cluster split K, each summing its part; the partial sums meet through
//    distributed shared memory in a fixed order.  8 x 4096 x 4096 takes 4.9 us
//    with the weights in L2 and 6.4 from HBM, 1 x 16384 x 4096 8.2 and 12.8 us
//    (5.3 TB/s).
// 3. fp8_dot_kernel (one to four tokens and not too many weights): CUDA cores.
//
// Every mbarrier wait is bounded; a thread whose wait runs out raises a shared
// abort flag, records an error in the library's device error word, and the
// CTA still frees its TMEM.

#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <algorithm>
#include <cmath>

#include "rbq_fp8.cuh"
#include "rbq_internal.h"
#include "rbq_qcodes.cuh"
#include "rbq_sm100.cuh"
#include "rbq_tiles.cuh"

namespace rbq {
namespace fp8 {
namespace {

using namespace sm100;

constexpr int kBK = 128;                  // K values (= bytes) per slice
constexpr int kThreads = 320;             // 4 epilogue warps, MMA, TMA, 4 scale loader warps
constexpr int kMmaWarp = 4, kTmaWarp = 5, kScaleWarp = 6;
constexpr int kGroup = 4;                 // K slices per scale word
constexpr int kSfBlock = 512;             // shared-memory bytes of 128 rows' scale words
constexpr int kGroups = 4;                // scale words per row and slot: the scales of up to 16 K slices
constexpr int kSlotSlices = kGroup * kGroups;
constexpr int kSfSlots = 2;               // ring of those slots in shared memory

// Instruction descriptor of kind::mxf8f6f4: E4M3 A and B (format 0), both
// K-major, E8M0 scales (bit 23), N>>3 at bit 17, M>>4 at bit 24; bits 4-5 and
// 29-30 pick the byte of B's and A's scale words.
__host__ __device__ constexpr uint32_t idesc_mx(int M, int N) {
  return (static_cast<uint32_t>(N >> 3) << 17) | (1u << 23) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ uint32_t idesc_byte(uint32_t b) { return (b << 4) | (b << 29); }

// D[tmem] (+)= (A scaled by sfa) (B scaled by sfb)^T.
template <bool PAIR>
__device__ __forceinline__ void umma_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                        uint32_t accumulate) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(accumulate)
        : "memory");
}
// 32 rows x 16 bytes of shared memory -> 4 columns of tensor memory, in every
// lane quadrant (of both CTAs of a pair, each from its own shared memory).
template <bool PAIR>
__device__ __forceinline__ void cp_scales(uint32_t taddr, uint64_t sdesc) {
  if constexpr (PAIR)
    asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
  else
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}
// Shared-memory descriptor of a 32 x 16 byte scale block: no swizzle, groups
// of 8 rows 128 bytes apart (stride offset), version 1.
__device__ __forceinline__ uint64_t sdesc_scales(uint32_t saddr) {
  return static_cast<uint64_t>((saddr >> 4) & 0x3FFFu) | (static_cast<uint64_t>(1u) << 16) |
         (static_cast<uint64_t>(128u >> 4) << 32) | (static_cast<uint64_t>(1u) << 46);
}

// The scales of 16 consecutive K slices of a row, four words, loaded without
// waiting for them and put together when they are stored.  ALIGN: what the
// first byte's address and the row's length are multiples of.  16: one load; 4:
// a load per word; 1: the row may start at any address, and a word is put
// together from two aligned ones.  (Byte by byte, the 512 x 1536 x 8960 layer,
// whose rows have 70 scales, took 38 us by pairs in place of 31.)  Loaded words
// may hold bytes of the rows beside it, but never of anything outside the
// matrix of scales [lo, hi); what follows the row's last slice is not
// multiplied.  Plain loads, not read-only ones: the kernel before may still be
// writing the scales when this one is launched.
template <int ALIGN>
struct ScaleRow {
  static constexpr int kWords = ALIGN == 1 ? kGroups + 1 : kGroups;
  const uint8_t *row = nullptr, *lo, *hi;        // null: a row outside the matrix, all its scales 0
  int left = 0;                                  // the row's slices from `row` on
  uint32_t w[kWords];
  __device__ __forceinline__ void start(const uint8_t* at, int slices, const uint8_t* matrix, long long bytes) {
    row = at;
    left = slices;
    lo = matrix;
    hi = matrix + bytes;
  }
  __device__ __forceinline__ void none() { row = nullptr; }
  // The next 16 slices' words.
  __device__ __forceinline__ void load() {
#pragma unroll
    for (int q = 0; q < kWords; ++q) w[q] = 0u;
    if (!row) return;
    if constexpr (ALIGN == 16) {
      const uint4 v = *reinterpret_cast<const uint4*>(row);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (ALIGN == 4) {
#pragma unroll
      for (int q = 0; q < kGroups; ++q)
        if (kGroup * q < left) w[q] = reinterpret_cast<const uint32_t*>(row)[q];
    } else {
      const uint8_t* p = row - offset();
#pragma unroll
      for (int q = 0; q < kWords; ++q, p += kGroup) {
        if (kGroup * q >= left + static_cast<int>(offset())) break;
        if (p >= lo && p + kGroup <= hi) {
          w[q] = *reinterpret_cast<const uint32_t*>(p);
        } else {
#pragma unroll
          for (int j = 0; j < kGroup; ++j)
            if (p + j >= lo && p + j < hi) w[q] |= static_cast<uint32_t>(p[j]) << (8 * j);
        }
      }
    }
  }
  // Word q of those that were loaded.
  __device__ __forceinline__ uint32_t word(int q) const {
    if constexpr (ALIGN == 1) return __funnelshift_r(w[q], w[q + 1], 8u * offset());
    return w[q];
  }
  __device__ __forceinline__ void step() {       // on to the 16 slices after these
    if (row) row += kSlotSlices;
    left -= kSlotSlices;
  }

 private:
  __device__ __forceinline__ uint32_t offset() const {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(row)) & 3u;
  }
};
__device__ __forceinline__ void put_scale_word(uint8_t* block, int r, uint32_t w) {
  *reinterpret_cast<uint32_t*>(block + 16 * (r & 31) + 4 * (r >> 5)) = w;
}

// One thread (row r) of the scale loaders: the words of its W rows, slot after
// slot of the ring `sf`.  `next(rows)` goes on to the next slices (false: there
// are no more), `slot_free(slot, use)` waits until the MMAs are done with the
// slot's last contents (false: gave up), `filled(slot)` reports.  The next
// slot's loads are in flight while the MMAs work on the last one's.  A slot
// holds the scales of 16 slices: with four, each hand-over (its wait acquires
// at cluster scope, which costs the L1 its lines) came four times as often, and
// a slice of 128 took 760 cycles in place of ~600.
template <int W, int ALIGN, typename Next, typename Free, typename Filled>
__device__ __forceinline__ bool feed_scales(ScaleRow<ALIGN> (&rows)[W], Next next, uint8_t* sf, int r, Free slot_free,
                                            Filled filled) {
  bool more = next(rows);
  for (uint32_t n = 0; more; ++n) {
    const uint32_t slot = n % kSfSlots;
    if (!slot_free(slot, n / kSfSlots)) return false;
    uint8_t* block = sf + slot * (kGroups * W * kSfBlock);
#pragma unroll
    for (int q = 0; q < kGroups; ++q)
#pragma unroll
      for (int j = 0; j < W; ++j) put_scale_word(block + (q * W + j) * kSfBlock, r, rows[j].word(q));
    fence_proxy_async_smem();
    __syncwarp();
    filled(slot);
    more = next(rows);
  }
  return true;
}

struct Params {
  int M, N, K, kbs;
  const uint8_t* sa;          // [M, kbs]
  const uint8_t* sw;          // [blocks(N), kbs]
  uint16_t* Y;
  unsigned int* err;
  int order;                  // tile order (tiles::TileOrder)
  int sf_align;               // 16, 4 or 1: as ScaleRow, of every part of a scale row that a CTA reads
  int y_four;                 // rows of Y 8-byte aligned
  int y_tma;                  // rows of Y 16-byte aligned: they go out by TMA
};

// ---- many tokens --------------------------------------------------------------
constexpr int kBM = 128;                  // rows of A per CTA
constexpr int kBN = 256;
constexpr int kATile = kBM * kBK;         // 16 KB
constexpr int kBTile = kBN / 2 * kBK;     // 16 KB: half of the tile's weight rows
constexpr int kStage = kATile + kBTile;
constexpr int kStages = 6;
constexpr int kSfWord = 3 * kSfBlock;     // a scale word of 128 rows of A and 256 of B
constexpr int kSfSlot = kGroups * kSfWord;
// Tensor memory: accumulator 0 in columns 0..255, accumulator 1 in 224..479,
// two buffers of scales (4 columns of A, 8 of B) from 480.
constexpr uint32_t kAcc1 = 224, kSfCol = 480, kSfCols = 12;

struct __align__(8) Tail {
  uint64_t full[kStages];
  uint64_t empty[kStages];
  uint64_t sf_full[kSfSlots];
  uint64_t sf_empty[kSfSlots];
  uint64_t sf_used[2];           // a tensor-memory buffer of scales
  uint64_t acc_full[2];
  uint64_t acc_empty[2];
  uint64_t overlap;              // the shared columns of the last tile's accumulator have been read
  uint64_t drain;                // abort path only: completion of the MMAs issued
  uint32_t tmem_slot;
  volatile uint32_t abort;
};

constexpr int kPiece = 32 * 128;          // bytes of a warp's 32 rows x 64 columns of the output
constexpr size_t kSmem = 1024 + kStages * kStage + kSfSlots * kSfSlot + 4 * kPiece + sizeof(Tail) + 64;
static_assert(kSfSlots * kSfSlot % 1024 == 0, "pieces are swizzle atoms");

// A warp's 32 rows x 64 columns of the output (row m0 + lane in each lane, 32
// words of two BF16) to rows whose length or address TMA does not take (N no
// multiple of 8).  Row by lane, each 2-byte store of the warp falls into 32
// sectors (a 333 x 1001 x 1552 layer took 44 us by pairs in place of 14), so the
// rows go through shared memory, word j of row r at j ^ r, and the warp writes
// one after the other with 4-byte stores.  A row that begins in the middle of a
// word is shifted by a half while it is still in its lane's registers; the lane writes
// the halves that are left at its ends.  One warp of the scheduler does all
// this, a few cycles an instruction: what counts is how many a row takes.
__device__ __forceinline__ void put_rows(uint32_t* turn, int lane, const uint32_t (&o)[32], const Params& p, int m0,
                                         int nb) {
  const int rows = min(32, p.M - m0), cols = min(64, p.N - nb);
  uint16_t* first = p.Y + static_cast<long long>(m0) * p.N + nb;      // of row 0
  const auto half_of = [&](int r) {                // row r begins in the middle of a word
    return static_cast<int>((reinterpret_cast<uintptr_t>(first) >> 1) + static_cast<uintptr_t>(r) * p.N) & 1;
  };
  const int h = half_of(lane);
#pragma unroll
  for (int j = 0; j < 32; ++j)
    turn[32 * lane + (j ^ lane)] = __byte_perm(o[j], o[min(j + 1, 31)], h ? 0x5432u : 0x3210u);
  if (lane < rows) {
    uint16_t* row = first + static_cast<long long>(lane) * p.N;
    const int words = (cols - h) >> 1;
    if (h) row[0] = static_cast<uint16_t>(o[0]);
    if ((cols - h) & 1) row[cols - 1] = static_cast<uint16_t>(turn[32 * lane + (words ^ lane)]);
  }
  __syncwarp();
  // rows r and r + 1 alternate between two alignments (or share one)
  const int h0 = half_of(0), h1 = half_of(1);
  uint32_t* even = reinterpret_cast<uint32_t*>(first + h0) + lane;
  uint32_t* odd = reinterpret_cast<uint32_t*>(first + p.N + h1) + lane;
  const bool in0 = lane < (cols - h0) >> 1, in1 = lane < (cols - h1) >> 1;
#pragma unroll
  for (int r = 0; r < 32; r += 2, even += p.N, odd += p.N) {        // two rows on: 2 N halves
    const uint32_t a = turn[32 * r + (lane ^ r)], b = turn[32 * (r + 1) + (lane ^ (r + 1))];
    if (in0 && r < rows) *even = a;
    if (in1 && r + 1 < rows) *odd = b;
  }
  __syncwarp();
}

// The scale loaders of one CTA of a pair: its 128 rows of A, all 256 of B.
template <int ALIGN>
__device__ __forceinline__ bool load_pair_scales(const Params& p, Tail& tl, uint8_t* sf, uint32_t rank, int tile,
                                                 int tstep) {
  const int r = threadIdx.x - 32 * kScaleWarp, lane = threadIdx.x & 31;
  const int ntiles_m = (p.M + 2 * kBM - 1) / (2 * kBM), ntiles_n = (p.N + kBN - 1) / kBN;
  const int ntiles = ntiles_m * ntiles_n, last_nb = blocks(p.N) - 1;
  const long long sa_bytes = static_cast<long long>(p.M) * p.kbs, sw_bytes = (last_nb + 1ll) * p.kbs;
  int kb = 0;
  ScaleRow<ALIGN> rows[3];
  // the next slices of this tile, or the first of the next
  const auto next = [&](ScaleRow<ALIGN> (&row)[3]) {
    if (tile >= ntiles) return false;
    if (kb == 0) {
      int mt, nt;
      tiles::tile_coords(tile, ntiles_m, ntiles_n, p.order, mt, nt);
      const int m = mt * 2 * kBM + static_cast<int>(rank) * kBM + r, nb = nt * (kBN / kBlock);
      if (m < p.M)
        row[0].start(p.sa + static_cast<long long>(m) * p.kbs, p.kbs, p.sa, sa_bytes);
      else
        row[0].none();
      row[1].start(p.sw + static_cast<long long>(nb) * p.kbs, p.kbs, p.sw, sw_bytes);
      row[2].start(p.sw + static_cast<long long>(min(nb + 1, last_nb)) * p.kbs, p.kbs, p.sw, sw_bytes);
    } else {
#pragma unroll
      for (int j = 0; j < 3; ++j) row[j].step();
    }
#pragma unroll
    for (int j = 0; j < 3; ++j) row[j].load();
    if ((kb += kSlotSlices) >= p.kbs) {
      kb = 0;
      tile += tstep;
    }
    return true;
  };
  return feed_scales(
      rows, next, sf, r,
      [&](uint32_t slot, uint32_t use) {
        return use < 1 || mbar_warp_wait(&tl.sf_empty[slot], (use - 1) & 1, &tl.abort);
      },
      [&](uint32_t slot) {
        if (lane == 0) mbar_arrive_cluster(mapa_shared(&tl.sf_full[slot], 0));
      });
}

__global__ void __launch_bounds__(kThreads, 1)
    fp8_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmY, const Params p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* ops = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* sf = ops + kStages * kStage;
  Tail* tl = reinterpret_cast<Tail*>(sf + kSfSlots * kSfSlot + 4 * kPiece);
  const int tid = threadIdx.x, warp = warp_number(), lane = tid & 31;
  // clusters are pairs of neighbouring blocks; the compiler knows that these are the same in all threads
  const uint32_t rank = blockIdx.x & 1u;
  const int tile0 = static_cast<int>(blockIdx.x >> 1), tstep = static_cast<int>(gridDim.x >> 1);
  const int ntiles_m = (p.M + 2 * kBM - 1) / (2 * kBM), ntiles_n = (p.N + kBN - 1) / kBN;
  const int ntiles = ntiles_m * ntiles_n;
  const int KS = p.kbs;
  volatile uint32_t* abort = &tl->abort;
  bool issuer = false;                     // the thread that issues the MMAs

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&tl->full[s], 1);
      mbar_init(&tl->empty[s], 1);
    }
    for (int s = 0; s < kSfSlots; ++s) {
      mbar_init(&tl->sf_full[s], 8);       // one arrival per loader warp of both CTAs
      mbar_init(&tl->sf_empty[s], 1);
    }
    mbar_init(&tl->sf_used[0], 1);
    mbar_init(&tl->sf_used[1], 1);
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tl->acc_full[a], 1);
      mbar_init(&tl->acc_empty[a], 8);     // one arrival per epilogue warp of both CTAs
    }
    mbar_init(&tl->overlap, 8);
    mbar_init(&tl->drain, 1);
    tl->abort = 0u;
    mbar_fence_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc_pair(&tl->tmem_slot, 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();                          // a pair's barriers are signalled from both CTAs
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, tl->tmem_slot, 0);
  griddep_wait();
  griddep_launch_dependents();

  if (warp == kMmaWarp) {
    // ---------------- MMA issuer (the even CTA's) ----------------
    // The warp goes through the loop together and one thread issues.  With one
    // thread in the whole loop a slice took 532 to 620 cycles, another number
    // after every change to the kernel; 4096 x 16384 x 4096 went from 198 to 186 us
    // together with the output by TMA.  (fp8_few_kernel's loop is short, and the
    // joint waits cost it more: 5.2 us in place of 4.9 for 1 x 4096 x 4096.)
    if (rank == 0) {
      constexpr uint32_t kIdesc = idesc_mx(2 * kBM, kBN);
      const uint64_t desc0 = sdesc_k_sw128(smem_u32(ops));
      const uint64_t sfdesc0 = sdesc_scales(smem_u32(sf));
      uint32_t s = 0, ph = 0, it = 0, g = 0, n = 0;     // operand stage, its phase; tile; scale word, slot
      bool ok = true;
      for (int tile = tile0; tile < ntiles && ok; tile += tstep, ++it) {
        const uint32_t a = it & 1u, use = it >> 1;
        if (use >= 1 && !mbar_warp_wait_cl(&tl->acc_empty[a], (use - 1) & 1, abort)) { ok = false; break; }
        if (it >= 1 && !mbar_warp_wait_cl(&tl->overlap, (it - 1) & 1, abort)) { ok = false; break; }
        tc_fence_after();
        const uint32_t acc = tmem + a * kAcc1;
        for (int ks0 = 0; ks0 < KS && ok; ks0 += kGroup, ++g) {
          const uint32_t slot = n % kSfSlots, q = (ks0 / kGroup) % kGroups;
          if (q == 0 && !mbar_warp_wait_cl(&tl->sf_full[slot], (n / kSfSlots) & 1, abort)) { ok = false; break; }
          // the MMAs that read this buffer's last contents (word g - 2) have completed
          if (g >= 2 && !mbar_warp_wait(&tl->sf_used[g & 1u], (g / 2 - 1) & 1, abort)) { ok = false; break; }
          tc_fence_after();
          const uint32_t sfa = tmem + kSfCol + (g & 1u) * kSfCols;
          const uint64_t sd = sfdesc0 + ((slot * kSfSlot + q * kSfWord) >> 4);
          if (elect_one()) {
            cp_scales<true>(sfa, sd);
            cp_scales<true>(sfa + 4, sd + (kSfBlock >> 4));
            cp_scales<true>(sfa + 8, sd + (2 * kSfBlock >> 4));
          }
#pragma unroll
          for (int j = 0; j < kGroup; ++j) {
            if (!ok || ks0 + j >= KS) break;
            if (!mbar_warp_wait(&tl->full[s], ph, abort)) { ok = false; break; }
            tc_fence_after();
            const uint64_t ad = desc0 + ((s * static_cast<uint32_t>(kStage)) >> 4);
            const uint64_t bd = ad + (kATile >> 4);
            const uint32_t id = kIdesc | idesc_byte(j), add = j != 0 || ks0 != 0;
            if (elect_one()) {
              umma_mx<true>(acc, ad, bd, id, sfa, sfa + 4, add);
              umma_mx<true>(acc, ad + 2, bd + 2, id, sfa, sfa + 4, 1u);     // +32 bytes = 32 values of K
              umma_mx<true>(acc, ad + 4, bd + 4, id, sfa, sfa + 4, 1u);
              umma_mx<true>(acc, ad + 6, bd + 6, id, sfa, sfa + 4, 1u);
              umma_commit_pair(&tl->empty[s], 3);
            }
            if (++s == kStages) { s = 0; ph ^= 1u; }
          }
          if (!ok) break;
          const bool last = q == kGroups - 1 || ks0 + kGroup >= KS;
          if (elect_one()) {
            umma_commit_pair(&tl->sf_used[g & 1u], 1);
            if (last) umma_commit_pair(&tl->sf_empty[slot], 3);
          }
          if (last) ++n;
        }
        if (ok && elect_one()) umma_commit_pair(&tl->acc_full[a], 3);
      }
      if (!ok && lane == 0) atomicOr(p.err, 2u);
      issuer = elect_one();
    }
  } else if (warp == kTmaWarp) {
    // ---------------- TMA producer: each CTA its own rows, both CTAs' bytes on the even CTA's barrier ----------------
    if (elect_one()) {
      tma_prefetch_desc(&tmA);
      tma_prefetch_desc(&tmB);
      uint32_t s = 0, ph = 0;
      bool first = true, ok = true;
      for (int tile = tile0; tile < ntiles && ok; tile += tstep) {
        int mt, nt;
        tiles::tile_coords(tile, ntiles_m, ntiles_n, p.order, mt, nt);
        const int m0 = mt * 2 * kBM + static_cast<int>(rank) * kBM;
        const int n0 = nt * kBN + static_cast<int>(rank) * (kBN / 2);
        for (int ks = 0; ks < KS; ++ks) {
          if (!first && !mbar_wait_or_abort(&tl->empty[s], ph ^ 1u, abort)) { ok = false; break; }
          uint8_t* st = ops + s * kStage;
          if (rank == 0) mbar_arrive_expect_tx(&tl->full[s], 2 * kStage);
          const uint32_t bar = mapa_shared(&tl->full[s], 0);
          tma_load_2d_pair(st, &tmA, ks * kBK, m0, bar);
          tma_load_2d_pair(st + kATile, &tmB, ks * kBK, n0, bar);
          if (++s == kStages) { s = 0; ph ^= 1u; first = false; }
        }
      }
      if (!ok) atomicOr(p.err, 16u);
    }
  } else if (warp >= kScaleWarp) {
    // ---------------- scale loaders: this CTA's 128 rows of A, all 256 of B ----------------
    const bool ok = p.sf_align == 16  ? load_pair_scales<16>(p, *tl, sf, rank, tile0, tstep)
                    : p.sf_align == 4 ? load_pair_scales<4>(p, *tl, sf, rank, tile0, tstep)
                                      : load_pair_scales<1>(p, *tl, sf, rank, tile0, tstep);
    if (!ok && lane == 0) atomicOr(p.err, 32u);
  } else {
    // ---------------- epilogue ----------------
    uint8_t* piece = sf + kSfSlots * kSfSlot + warp * kPiece;
    uint32_t it = 0;
    for (int tile = tile0; tile < ntiles; tile += tstep, ++it) {
      const uint32_t a = it & 1u, use = it >> 1;
      int mt, nt;                             // before the wait: the next tile's MMAs wait for what follows it
      tiles::tile_coords(tile, ntiles_m, ntiles_n, p.order, mt, nt);
      if (!mbar_warp_wait(&tl->acc_full[a], use & 1, abort)) {   // warp-uniform: tmem loads follow
        if (lane == 0) atomicOr(p.err, 4u);
        break;
      }
      tc_fence_after();
      const int m0 = mt * 2 * kBM + static_cast<int>(rank) * kBM + 32 * warp;     // this warp's rows
      const uint32_t tq = tmem + (static_cast<uint32_t>(32 * warp) << 16) + a * kAcc1;
#pragma unroll 1
      for (int c = 0; c < kBN / 64; ++c) {
        const int cc = a == 0 ? kBN / 64 - 1 - c : c;   // the columns both accumulators share come first
        uint32_t o[32];
        {
          uint32_t u[32], v[32];
          tmem_ld32(tq + 64 * cc, u);
          tmem_ld32(tq + 64 * cc + 32, v);
          tmem_wait_ld();
          if (c == 0) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_relaxed(mapa_shared(&tl->overlap, 0));
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            o[j] = bf16x2(u[2 * j], u[2 * j + 1]);
            o[16 + j] = bf16x2(v[2 * j], v[2 * j + 1]);
          }
        }
        const int nb = nt * kBN + 64 * cc;
        if (m0 >= p.M || nb >= p.N) continue;           // the same in the whole warp
        if (p.y_tma) {
          if (lane == 0) bulk_wait_read<0>();              // the last piece has left
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(piece + sw128_offset(lane, j)) =
                make_uint4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) tma_store_2d(&tmY, nb, m0, piece);
        } else {
          put_rows(reinterpret_cast<uint32_t*>(piece), lane, o, p, m0, nb);
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
  if (tl->abort) {                 // the same value in every thread after the barrier
    drain_after_abort(issuer, &tl->drain, true);
    __syncthreads();
  }
  // Neither CTA of a pair leaves while the other may still signal its
  // barriers or the MMAs may still read its shared memory.
  cluster_sync();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ---- few tokens ----------------------------------------------------------------
// Tile: 128 output columns (weight rows) x NT tokens; the S CTAs of a cluster
// take consecutive parts of the K slices.
template <int NT>
struct Few {
  static constexpr int kWTile = kBM * kBK;                       // 16 KB of weights
  static constexpr int kTTile = NT * kBK;
  static constexpr int kStage = kWTile + kTTile;
  static constexpr int kStages = (NT <= 64 ? 8 : NT == 128 ? 6 : 4);
  static constexpr int kSfWord = kSfBlock * (NT > 128 ? 3 : 2);
  static constexpr int kSfSlot = kGroups * kSfWord;
  static constexpr uint32_t kSfCol = NT, kSfCols = NT > 128 ? 12 : 8;     // columns of a scale buffer
  static constexpr uint32_t kTmemCols = NT <= 16 ? 32 : NT <= 32 ? 64 : NT == 64 ? 128 : NT == 128 ? 256 : 512;
  static constexpr int kRing = kStages * kStage;
  static constexpr size_t kSmem = 1024 + kRing + kSfSlots * kSfSlot + 512;
  static_assert(kSfCol + 2 * kSfCols <= kTmemCols, "accumulator and scales fit");
  static_assert(NT * kBM * 4 <= kRing, "the partial sums fit where the operands were");
};

struct __align__(8) FewTail {
  uint64_t full[8];
  uint64_t empty[8];
  uint64_t sf_full[kSfSlots];
  uint64_t sf_empty[kSfSlots];
  uint64_t sf_used[2];           // a tensor-memory buffer of scales
  uint64_t acc_full;
  uint64_t drain;
  uint32_t tmem_slot;
  volatile uint32_t abort;
};
static_assert(sizeof(FewTail) <= 512, "the tail fits");

// The scale loaders of a CTA: its 128 weight rows, its NT tokens, K slices kb0 to kb1.
template <int NT, int ALIGN>
__device__ __forceinline__ bool load_few_scales(const Params& p, FewTail& tl, uint8_t* sf, int nt, int m0, int kb0,
                                                int kb1) {
  constexpr int kRows = NT > 128 ? 3 : 2;
  const int r = threadIdx.x - 32 * kScaleWarp, lane = threadIdx.x & 31;
  ScaleRow<ALIGN> rows[kRows];
  int kb = kb0;
  const auto next = [&](ScaleRow<ALIGN> (&row)[kRows]) {
    if (kb >= kb1) return false;
    if (kb == kb0) {
      row[0].start(p.sw + static_cast<long long>(nt) * p.kbs + kb0, p.kbs - kb0, p.sw,
                   static_cast<long long>(blocks(p.N)) * p.kbs);
#pragma unroll
      for (int j = 1; j < kRows; ++j) {
        const int t = r + 128 * (j - 1);
        if (t < NT && m0 + t < p.M)
          row[j].start(p.sa + static_cast<long long>(m0 + t) * p.kbs + kb0, p.kbs - kb0, p.sa,
                       static_cast<long long>(p.M) * p.kbs);
        else
          row[j].none();
      }
    } else {
#pragma unroll
      for (int j = 0; j < kRows; ++j) row[j].step();
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) row[j].load();
    kb += kSlotSlices;
    return true;
  };
  return feed_scales(
      rows, next, sf, r,
      [&](uint32_t slot, uint32_t use) {
        return use < 1 || mbar_warp_wait(&tl.sf_empty[slot], (use - 1) & 1, &tl.abort);
      },
      [&](uint32_t slot) {
        if (lane == 0) mbar_arrive(&tl.sf_full[slot]);
      });
}

// Tokens rank, rank + S, ... of the tile: a warp per token, a lane's four
// columns from each of the cluster's S partial sums (`red`: [token][128] fp32
// at the same place in every CTA), added in their order and written.
template <int S>
__device__ __forceinline__ void finish_tokens(const Params& p, uint32_t red, uint32_t rank, int m0, int n0,
                                              int tokens) {
  const int lane = threadIdx.x & 31, n = n0 + 4 * lane;
  uint32_t base[S];
#pragma unroll
  for (int c = 0; c < S; ++c)
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(base[c]) : "r"(red + 16u * lane), "r"(c));
#pragma unroll(S > 2 ? 1 : 4 / S)
  for (int t = static_cast<int>(rank) + S * (threadIdx.x >> 5); t < tokens; t += S * (kThreads / 32)) {
    float4 v[S];
#pragma unroll
    for (int c = 0; c < S; ++c)
      asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                   : "=f"(v[c].x), "=f"(v[c].y), "=f"(v[c].z), "=f"(v[c].w)
                   : "r"(base[c] + 4u * kBM * t)
                   : "memory");
#pragma unroll
    for (int c = 1; c < S; ++c) {
      v[0].x += v[c].x;
      v[0].y += v[c].y;
      v[0].z += v[c].z;
      v[0].w += v[c].w;
    }
    const __nv_bfloat162 a = __floats2bfloat162_rn(v[0].x, v[0].y), b = __floats2bfloat162_rn(v[0].z, v[0].w);
    const uint32_t w0 = *reinterpret_cast<const uint32_t*>(&a), w1 = *reinterpret_cast<const uint32_t*>(&b);
    uint16_t* dst = p.Y + static_cast<long long>(m0 + t) * p.N + n;
    if (n + 4 <= p.N && p.y_four) {
      *reinterpret_cast<uint2*>(dst) = make_uint2(w0, w1);
    } else {
      if (n < p.N) dst[0] = static_cast<uint16_t>(w0);
      if (n + 1 < p.N) dst[1] = static_cast<uint16_t>(w0 >> 16);
      if (n + 2 < p.N) dst[2] = static_cast<uint16_t>(w1);
      if (n + 3 < p.N) dst[3] = static_cast<uint16_t>(w1 >> 16);
    }
  }
}

template <int NT>
__global__ void __launch_bounds__(kThreads, 1)
    fp8_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmT, const Params p) {
  using F = Few<NT>;
  constexpr int kS = F::kStages;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  uint8_t* ops = smem_raw + (((raw + 1023u) & ~1023u) - raw);
  uint8_t* sf = ops + F::kRing;
  FewTail* tl = reinterpret_cast<FewTail*>(sf + kSfSlots * F::kSfSlot);
  const int tid = threadIdx.x, warp = warp_number(), lane = tid & 31;
  uint32_t rank, S;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(S));
  const int ntiles_n = blocks(p.N);
  const int tile = static_cast<int>(cluster_id_x());
  const int nt = tile % ntiles_n, mt = tile / ntiles_n;
  const int n0 = nt * kBM, m0 = mt * NT;
  const int kb0 = static_cast<int>(static_cast<long long>(p.kbs) * rank / S);
  const int kb1 = static_cast<int>(static_cast<long long>(p.kbs) * (rank + 1) / S);   // S <= kbs: never empty
  volatile uint32_t* abort = &tl->abort;
  bool issuer = false;                     // the thread that issues the MMAs

  if (tid == 0) {
    for (int s = 0; s < kS; ++s) {
      mbar_init(&tl->full[s], 1);
      mbar_init(&tl->empty[s], 1);
    }
    for (int s = 0; s < kSfSlots; ++s) {
      mbar_init(&tl->sf_full[s], 4);
      mbar_init(&tl->sf_empty[s], 1);
    }
    mbar_init(&tl->sf_used[0], 1);
    mbar_init(&tl->sf_used[1], 1);
    mbar_init(&tl->acc_full, 1);
    mbar_init(&tl->drain, 1);
    tl->abort = 0u;
    mbar_fence_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&tl->tmem_slot, F::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tl->tmem_slot;
  griddep_wait();
  griddep_launch_dependents();

  if (warp == kMmaWarp) {
    if (elect_one()) {
      issuer = true;
      constexpr uint32_t kIdesc = idesc_mx(kBM, NT);
      const uint64_t desc0 = sdesc_k_sw128(smem_u32(ops));
      const uint64_t sfdesc0 = sdesc_scales(smem_u32(sf));
      uint32_t s = 0, ph = 0, g = 0;
      bool ok = true;
      for (int kg = kb0; kg < kb1 && ok; kg += kGroup, ++g) {
        const uint32_t q = g % kGroups, n = g / kGroups, slot = n % kSfSlots;
        if (q == 0 && !mbar_wait_or_abort(&tl->sf_full[slot], (n / kSfSlots) & 1, abort)) { ok = false; break; }
        if (g >= 2 && !mbar_wait_or_abort(&tl->sf_used[g & 1u], (g / 2 - 1) & 1, abort)) { ok = false; break; }
        tc_fence_after();
        const uint32_t sfa = tmem + F::kSfCol + (g & 1u) * F::kSfCols;
        const uint64_t sd = sfdesc0 + ((slot * F::kSfSlot + q * F::kSfWord) >> 4);
        cp_scales<false>(sfa, sd);
        cp_scales<false>(sfa + 4, sd + (kSfBlock >> 4));
        if constexpr (NT > 128) cp_scales<false>(sfa + 8, sd + (2 * kSfBlock >> 4));
#pragma unroll
        for (int j = 0; j < kGroup; ++j) {
          if (!ok || kg + j >= kb1) break;
          if (!mbar_wait_or_abort(&tl->full[s], ph, abort)) { ok = false; break; }
          tc_fence_after();
          const uint64_t ad = desc0 + ((s * static_cast<uint32_t>(F::kStage)) >> 4);
          const uint64_t bd = ad + (F::kWTile >> 4);
          const uint32_t id = kIdesc | idesc_byte(j);
          umma_mx<false>(tmem, ad, bd, id, sfa, sfa + 4, j != 0 || kg != kb0);
          umma_mx<false>(tmem, ad + 2, bd + 2, id, sfa, sfa + 4, 1u);
          umma_mx<false>(tmem, ad + 4, bd + 4, id, sfa, sfa + 4, 1u);
          umma_mx<false>(tmem, ad + 6, bd + 6, id, sfa, sfa + 4, 1u);
          umma_commit(&tl->empty[s]);
          if (++s == kS) { s = 0; ph ^= 1u; }
        }
        if (!ok) break;
        umma_commit(&tl->sf_used[g & 1u]);
        if (q == kGroups - 1) umma_commit(&tl->sf_empty[slot]);
      }
      if (ok)
        umma_commit(&tl->acc_full);
      else
        atomicOr(p.err, 2u);
    }
  } else if (warp == kTmaWarp) {
    if (elect_one()) {
      tma_prefetch_desc(&tmW);
      tma_prefetch_desc(&tmT);
      uint32_t s = 0, ph = 0;
      bool first = true, ok = true;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!first && !mbar_wait_or_abort(&tl->empty[s], ph ^ 1u, abort)) { ok = false; break; }
        uint8_t* st = ops + s * F::kStage;
        mbar_arrive_expect_tx(&tl->full[s], F::kStage);
        tma_load_2d(st, &tmW, kb * kBK, n0, &tl->full[s]);
        tma_load_2d(st + F::kWTile, &tmT, kb * kBK, m0, &tl->full[s]);
        if (++s == kS) { s = 0; ph ^= 1u; first = false; }
      }
      if (!ok) atomicOr(p.err, 16u);
    }
  } else if (warp >= kScaleWarp) {
    const bool ok = p.sf_align == 16  ? load_few_scales<NT, 16>(p, *tl, sf, nt, m0, kb0, kb1)
                    : p.sf_align == 4 ? load_few_scales<NT, 4>(p, *tl, sf, nt, m0, kb0, kb1)
                                      : load_few_scales<NT, 1>(p, *tl, sf, nt, m0, kb0, kb1);
    if (!ok && lane == 0) atomicOr(p.err, 32u);
  } else {
    // partial sums -> red[token][128 columns] where the operands were: every
    // slice has been loaded and multiplied once acc_full completes
    float* red = reinterpret_cast<float*>(ops);
    if (mbar_warp_wait(&tl->acc_full, 0, abort)) {
      tc_fence_after();
      constexpr int kStep = NT < 32 ? 16 : 32;
#pragma unroll 1
      for (int c = 0; c < NT && m0 + c < p.M; c += kStep) {
        uint32_t v[32];
        if constexpr (kStep == 32)
          tmem_ld32(tmem + (static_cast<uint32_t>(32 * warp) << 16) + c, v);
        else
          tmem_ld16(tmem + (static_cast<uint32_t>(32 * warp) << 16) + c, v);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < kStep; ++j) red[(c + j) * kBM + 32 * warp + lane] = __uint_as_float(v[j]);
      }
    } else if (lane == 0) {
      atomicOr(p.err, 4u);
    }
  }
  tc_fence_before();
  __syncthreads();
  const bool failed = tl->abort != 0u;
  if (failed) {
    drain_after_abort(issuer, &tl->drain);
    __syncthreads();
  }
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, F::kTmemCols);
  }
  // the cluster's partial sums, added in the order of their K slices; CTA
  // `rank` finishes tokens rank, rank + S, ...
  if (S > 1) cluster_sync();
  const int tokens = min(NT, p.M - m0);
  const uint32_t red = smem_u32(ops);
  if (S == 1)
    finish_tokens<1>(p, red, 0, m0, n0, tokens);
  else if (S == 2)
    finish_tokens<2>(p, red, rank, m0, n0, tokens);
  else if (S == 4)
    finish_tokens<4>(p, red, rank, m0, n0, tokens);
  else
    finish_tokens<8>(p, red, rank, m0, n0, tokens);
  __syncwarp();
  if (S > 1) cluster_sync();       // no CTA leaves while another reads its sums
}

// BF16 [M, N], boxes of 32 rows x 64 columns, 128B swizzle.
int encode_out_map(CUtensorMap* map, uint16_t* base, int M, int N) {
  auto fn = qfast::encode_fn();
  if (!fn) return RBQ_ECUDA;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(M)};
  const cuuint64_t strides[1] = {2 * static_cast<cuuint64_t>(N)};
  const cuuint32_t box[2] = {64, 32};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? RBQ_OK : RBQ_ECUDA;
}

// ---- single tokens ---------------------------------------------------------------
// Up to four tokens on the CUDA cores: a CTA of 128 threads takes four weight
// rows, a thread 16 codes of each (and the 16 that lie 2048 on), all rows'
// loads in flight together.  Products of codes are exact in fp32 and are summed
// by 16, two to an instruction; then come the two scales, and the sum over the
// CTA in a fixed order.  No tensor maps, no tensor memory, no cluster: besides
// the weights' way a token pays for a launch and one reduction.  1 x 4096 x
// 4096 takes 4.3 us (5.8 from HBM) and fp8_few_kernel 5.0 (6.1); 1 x 1536 x
// 1536 1.9 and 3.4; with more tokens or weights the tensor cores win (4 x
// 4096 x 4096: 8.6 and 5.0).  Eight rows or several groups of threads to a
// CTA, or 4096 codes at once, were slower: 4.6 to 6.9 us.
constexpr int kDotThreads = 128, kDotRows = 4, kDotTokens = 4;
constexpr int kDotSpan = 16 * kDotThreads;        // codes of a row that a CTA takes at a time

using f2 = unsigned long long;                    // two fp32 in one 64-bit register
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
// Sixteen codes -> pairs of fp32.
__device__ __forceinline__ void decode16(const uint4& c, f2 (&v)[8]) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 t = decode2(w[i / 2] >> (16 * (i & 1)));
    asm("mov.b64 %0, {%1, %2};" : "=l"(v[i]) : "f"(t.x), "f"(t.y));
  }
}
// A scale 2^e, e = b - 127, as two factors 2^ceil(e/2) and 2^floor(e/2); NaN for b = 255.
struct Halves {
  float up, down;
};
__device__ __forceinline__ Halves halves(uint32_t b) {
  return {b == 255u ? __uint_as_float(0x7FFFFFFFu) : __uint_as_float(((b + 128u) >> 1) << 23),
          __uint_as_float(((b + 127u) >> 1) << 23)};
}

// (With the 1 of the launch bounds the compiler takes 80 registers for one token,
// 64 without it: 1 x 1536 x 8960 4.10 us and 4.71.)
template <int MT>
__global__ void __launch_bounds__(kDotThreads, 1) fp8_dot_kernel(const uint8_t* a, const uint8_t* w, const Params p) {
  __shared__ float sums[kDotThreads / 32][kDotRows * MT];
  griddep_wait();
  griddep_launch_dependents();
  const int n0 = blockIdx.x * kDotRows, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // rows behind the last one repeat it and are not written
  const uint8_t *rows[kDotRows], *scales[kDotRows];
#pragma unroll
  for (int r = 0; r < kDotRows; ++r) {
    const int n = min(n0 + r, p.N - 1);
    rows[r] = w + static_cast<long long>(n) * p.K;
    scales[r] = p.sw + static_cast<long long>(n / kBlock) * p.kbs;
  }
  float acc[kDotRows][MT] = {};
  for (int k = 16 * threadIdx.x; k < p.K; k += kDotSpan) {
    uint4 c[kDotRows], xc[MT];
    uint32_t wb[kDotRows], xb[MT];
#pragma unroll
    for (int r = 0; r < kDotRows; ++r) {
      c[r] = *reinterpret_cast<const uint4*>(rows[r] + k);
      wb[r] = scales[r][k / kBlock];
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      const int row = min(m, p.M - 1);
      xc[m] = *reinterpret_cast<const uint4*>(a + static_cast<long long>(row) * p.K + k);
      xb[m] = p.sa[static_cast<long long>(row) * p.kbs + k / kBlock];
    }
    // Both scales of a pair are applied in two steps, the larger half of one with
    // the smaller half of the other, so that neither step overflows, or costs
    // digits, on the way to a result that does neither (one scale after the other
    // does: 2^-117 * 2^117 and a sum of 2^11): a sum is 0 or within 2^-18 and
    // 2^22, and each step's factor the root of the whole within a factor of 2.
    Halves wh[kDotRows], xh[MT];
#pragma unroll
    for (int r = 0; r < kDotRows; ++r) wh[r] = halves(wb[r]);
#pragma unroll
    for (int m = 0; m < MT; ++m) xh[m] = halves(xb[m]);
    f2 x[MT][8];
#pragma unroll
    for (int m = 0; m < MT; ++m) decode16(xc[m], x[m]);
#pragma unroll
    for (int r = 0; r < kDotRows; ++r) {
      f2 v[8];
      decode16(c[r], v);
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        f2 s = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) s = fma2(v[i], x[m][i], s);
        float even, odd;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(even), "=f"(odd) : "l"(s));
        acc[r][m] = fmaf((even + odd) * (xh[m].up * wh[r].down), xh[m].down * wh[r].up, acc[r][m]);
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kDotRows; ++r)
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) acc[r][m] += __shfl_xor_sync(0xffffffffu, acc[r][m], o);
      if (lane == 0) sums[warp][r * MT + m] = acc[r][m];
    }
  __syncthreads();
  if (threadIdx.x < kDotRows * MT) {
    const int r = threadIdx.x / MT, m = threadIdx.x % MT;
    float s = sums[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < kDotThreads / 32; ++i) s += sums[i][threadIdx.x];
    if (m < p.M && n0 + r < p.N)
      p.Y[static_cast<long long>(m) * p.N + n0 + r] = __bfloat16_as_ushort(__float2bfloat16_rn(s));
  }
}

// uint8 [rows, K] K-major, boxes of box_rows x 128 bytes, 128B swizzle.
int encode_map(CUtensorMap* map, const uint8_t* base, int rows, int K, int box_rows) {
  auto fn = qfast::encode_fn();
  if (!fn) return RBQ_ECUDA;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(K), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(K)};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(kBK), static_cast<cuuint32_t>(box_rows)};
  const cuuint32_t estr[2] = {1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? RBQ_OK : RBQ_ECUDA;
}

cudaLaunchAttribute cluster_attr(int size) {
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeClusterDimension;
  a.val.clusterDim.x = size;
  a.val.clusterDim.y = 1;
  a.val.clusterDim.z = 1;
  return a;
}
cudaLaunchAttribute pdl_attr() {
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  return a;
}

// Pairs of the pair kernel that can be resident on device `dev`, asked once per device (0: none).
int pair_clusters(int dev) {
  static int cached[kMaxDevices] = {};        // 0 = not yet asked; else pairs + 1
  if (cached[dev]) return cached[dev] - 1;
  if (cudaFuncSetAttribute(fp8_pair_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kSmem)) !=
      cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cudaLaunchAttribute attr[1] = {cluster_attr(2)};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, fp8_pair_kernel, &cfg) != cudaSuccess) {
    cudaGetLastError();
    n = 0;
  }
  cached[dev] = n + 1;
  return n;
}

int launch_pair(const uint8_t* a, const uint8_t* w, Params p, int dev, cudaStream_t st) {
  int clusters = pair_clusters(dev);
  if (clusters < 1) return RBQ_ECUDA;
  p.order = tiles::tile_order(dev, 1LL * p.M * p.K, 1LL * p.N * p.K);
  CUtensorMap mA, mB, mY{};
  int rc = p.y_tma ? encode_out_map(&mY, p.Y, p.M, p.N) : RBQ_OK;
  if (rc != RBQ_OK) return rc;
  rc = encode_map(&mA, a, p.M, p.K, kBM);
  if (rc != RBQ_OK) return rc;
  if ((rc = encode_map(&mB, w, p.N, p.K, kBN / 2)) != RBQ_OK) return rc;
  const long long ntiles = ((p.M + 2LL * kBM - 1) / (2 * kBM)) * ((p.N + kBN - 1) / kBN);
  if (ntiles > 0x7FFFFFFFll) return RBQ_EINVAL;
  if (clusters > ntiles) clusters = static_cast<int>(ntiles);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(2 * clusters, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2] = {pdl_attr(), cluster_attr(2)};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, fp8_pair_kernel, mA, mB, mY, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? RBQ_OK : cuda_fail(e);
}

template <int NT>
int launch_few(const uint8_t* a, const uint8_t* w, const Params& p, int S, int dev, cudaStream_t st) {
  using F = Few<NT>;
  static bool ready[kMaxDevices] = {};
  if (!ready[dev]) {
    const cudaError_t e = cudaFuncSetAttribute(fp8_few_kernel<NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               static_cast<int>(F::kSmem));
    if (e != cudaSuccess) return cuda_fail(e);
    ready[dev] = true;
  }
  const long long ntiles = static_cast<long long>(blocks(p.N)) * ((p.M + NT - 1) / NT);
  if (ntiles * S > 0x7FFFFFFFll) return RBQ_EINVAL;
  CUtensorMap mW, mT;
  int rc = encode_map(&mW, w, p.N, p.K, kBM);
  if (rc != RBQ_OK) return rc;
  if ((rc = encode_map(&mT, a, p.M, p.K, NT)) != RBQ_OK) return rc;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(ntiles * S), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = F::kSmem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2] = {pdl_attr(), cluster_attr(S)};
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  cudaError_t e = cudaLaunchKernelEx(&cfg, fp8_few_kernel<NT>, mW, mT, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? RBQ_OK : cuda_fail(e);
}

// Which kernel, with how many tokens to a tile and how many CTAs to a tile's
// K: what takes least by a linear model, in ns: a launch `start`, each K slice of
// a wave of CTAs `slice` or what 17 TB/s take from L2 for all of them, each
// further wave 5000 (2400 by pairs), a cluster's joint sum 600 + 200 S + 8 NT.
// One to four tokens: fp8_dot_kernel where 1200 + 0.15 N + (250 + 260 M) for
// each 2048 codes of a row + (45 + 80 M) for a million weights is less.
// Few tokens to a tile fill the GPU and share little; the pair kernel shares
// most and pays from about 60 tiles of 256 x 256.  For instance 512 x 4096 x
// 4096: 14.4 us by pairs, 9.7 with NT = 128 (S = 1), 12.1 with NT = 256 and
// S = 2; 1 x 4096 x 4096 without the dot kernel: 5.0 us with S = 4, 6.2 with S =
// 1; 4096 x 4096 x 4096: 56 us by pairs, 67 with NT = 256; 333 x 1001 x 1552:
// 5.8 us with NT = 32, 10.6 by pairs.
// Measured on 70 layers of 1 to 4096 tokens and seven weights of 64 x 256 to
// 16384 x 4096, every choice in each: its choice is the best or within 7 % of
// it in 65 of them with the weights in L2, and in 65 with the weights from HBM,
// whose bytes it does not count.  It loses most where clusters leave SMs idle,
// which it does not count either: of S = 4, 33 run at once and 36 do not (333 x
// 1408 x 8960 10.4 us, 333 x 1536 x 8960 17.9; the latter 11.1 with NT = 64 and
// S = 2), and, at a few microseconds, by leaving K whole (8 x 1001 x 1552: 4.9,
// 3.9 with S = 4).
constexpr int kDotPlan = -1;
struct Plan {
  int NT, S;                // tokens to a tile (0: the pair kernel, kDotPlan), CTAs to a cluster
};
Plan make_plan(int M, int N, int K, int sms) {
  const int kbs = blocks(K);
  const auto up = [](double a, double b) { return std::ceil(a / b); };
  const double pair_waves = up(up(M, 256) * up(N, 256), sms / 2);
  Plan best{0, 1};
  double least = 6500 + 2400 * (pair_waves - 1) + 328 * pair_waves * kbs;
  constexpr struct {
    int NT, start, slice;
  } kinds[] = {{16, 2350, 145}, {32, 2850, 145}, {64, 2950, 180}, {128, 3250, 218}, {256, 6200, 289}};
  for (const auto& k : kinds) {
    const double tiles = up(N, 128) * up(M, k.NT);
    const double l2 = tiles * kbs * ((kBM + k.NT) * kBK) / 17000;
    for (int S = 1; S <= 8 && S <= kbs; S *= 2) {
      const double waves = up(tiles * S, sms);
      const double t = k.start + 5000 * (waves - 1) + std::max(waves * up(kbs, S) * k.slice, l2) +
                       (S > 1 ? 600 + 200 * S + 8 * k.NT : 0);
      if (t < least) {
        least = t;
        best = {k.NT, S};
      }
    }
    if (k.NT >= M) break;
  }
  if (M <= kDotTokens && 1200 + 0.15 * N + (250 + 260 * M) * up(K, kDotSpan) + (45 + 80 * M) * 1e-6 * N * K < least)
    best = {kDotPlan, 1};
  return best;
}

template <int MT>
int launch_dot(const uint8_t* a, const uint8_t* w, const Params& p, cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((p.N + kDotRows - 1) / kDotRows), 1, 1);
  cfg.blockDim = dim3(kDotThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1] = {pdl_attr()};
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, fp8_dot_kernel<MT>, a, w, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  return e == cudaSuccess ? RBQ_OK : cuda_fail(e);
}

}  // namespace
}  // namespace fp8
}  // namespace rbq

using namespace rbq;

extern "C" int qlinear_fp8(const uint8_t* a_codes, const uint8_t* a_scales, const uint8_t* w_codes,
                           const uint8_t* w_scales, int M, int N, int K, uint16_t* Y, void* stream) {
  if (M < 0 || M > fp8::kMaxSize || N < 0 || N > fp8::kMaxSize || K <= 0 || K > fp8::kMaxSize || K % 16)
    return RBQ_EINVAL;
  if (M == 0 || N == 0) return RBQ_OK;
  if (!a_codes || !a_scales || !w_codes || !w_scales || !Y) return RBQ_EINVAL;
  if (!aligned(a_codes, 16) || !aligned(w_codes, 16) || !aligned(Y, 2)) return RBQ_EALIGN;
  fp8::Params p{};
  p.M = M;
  p.N = N;
  p.K = K;
  p.kbs = fp8::blocks(K);
  p.sa = a_scales;
  p.sw = w_scales;
  p.Y = Y;
  p.sf_align = p.kbs % 16 == 0 && aligned(a_scales, 16) && aligned(w_scales, 16) ? 16
               : p.kbs % 4 == 0 && aligned(a_scales, 4) && aligned(w_scales, 4)  ? 4
                                                                                  : 1;
  p.y_four = N % 4 == 0 && aligned(Y, 8);
  p.y_tma = N % 8 == 0 && aligned(Y, 16);
  int rc = device_error_word_ptr(&p.err);
  if (rc != RBQ_OK) return rc;
  int dev = 0, sms = 148;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e);
  if (dev < 0 || dev >= kMaxDevices) return RBQ_EINVAL;
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const fp8::Plan plan = fp8::make_plan(M, N, K, sms);
  const int S = plan.S;
  for (int r = 1; r < S; ++r)
    while (static_cast<long long>(p.kbs) * r / S % p.sf_align) p.sf_align = p.sf_align == 16 ? 4 : 1;
  switch (plan.NT) {
    case fp8::kDotPlan:
      return M == 1   ? fp8::launch_dot<1>(a_codes, w_codes, p, st)
             : M == 2 ? fp8::launch_dot<2>(a_codes, w_codes, p, st)
                      : fp8::launch_dot<4>(a_codes, w_codes, p, st);
    case 16: return fp8::launch_few<16>(a_codes, w_codes, p, S, dev, st);
    case 32: return fp8::launch_few<32>(a_codes, w_codes, p, S, dev, st);
    case 64: return fp8::launch_few<64>(a_codes, w_codes, p, S, dev, st);
    case 128: return fp8::launch_few<128>(a_codes, w_codes, p, S, dev, st);
    case 256: return fp8::launch_few<256>(a_codes, w_codes, p, S, dev, st);
  }
  return fp8::launch_pair(a_codes, w_codes, p, dev, st);
}
