// Products of rows sorted by expert with the experts' weights, their weight
// gradients, and the same product of MX FP4 operands.
//
//   product       y[r, n] = sum_k x[r, k] W[e][k, n] + b[e][n],  r in expert e's rows
//   weight grad   dW[e][k, n] = sum over r in expert e's rows of x[r, k] dy[r, n]
//   MX FP4        the product with x = a code times 2^(a scale - 127), W likewise, a scale
//                 per 32 elements of K
//
// All are one kernel: a CTA pair (tcgen05 cta_group::2) takes 256 columns n of the weight as
// the MMA's rows (TMEM lanes) and up to TM rows of y, or rows k of dW, as its columns.  With
// the ragged side in the MMA's N, a tile takes as many columns as it has rows, rounded up to
// 32: experts of 1, 40 or 300 rows cost what they have, and one kernel serves a decode step's
// few rows (bound by the weights' bytes) and a long prefill (bound by the tensor cores).
//
// Measured on a GB300; in brackets the operands' and outputs' bytes at a copy's 6.79 TB/s (reads
// alone reach 7.0), or the operations at cuBLAS's 1912 TFLOP/s (FP4 four times that), 1711 in
// calls back to back, where the clock is down to 1.4 GHz:
//   product 8192 rows of 8 experts, 4096 x 28672        1272-1300 us (1006; 1125 sustained)
//   product 32 rows of 8 experts, 14336 x 4096          133-136 us (137: HBM)
//   weight grad 8192 rows of 8, 14336 x 4096 to fp32    750-756 us (503; 562 sustained: the
//     output's stores)
//   weight grad 131064 rows of 128, 2048 x 1536, bf16   655-666 us (431; 482 sustained: tiles of
//     unequal cost go to the pairs in turn)
//   FP4 8192 x 7168 x 4096                              83 us (63: the round trip of the
//     five stages that shared memory holds)
//   FP4 64 rows of 32 experts, 7168 x 4096              72-76 us with the rows' quantisation (64)
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "dense.cuh"
#include "ptx.cuh"
#include "raw_scales.cuh"

namespace gbmoe {
namespace {

// W [E, K, N], [E, N, K]; FP4: [E, N, K], rows of scales of whole 16 bytes, and of any size
enum Mode { kProduct, kProductT, kWeightGrad, kFp4, kFp4Rows };

constexpr int kGrThreads = 128 + 256;  // TMA, MMA, two helper warps; 8 output warps
constexpr int kGrMaxExperts = 1024;
constexpr int kGrGroup = 8;            // row tiles of a raster group
constexpr int kScaleChunks = 3;        // FP4: chunks of 1024 elements whose scales are on their way
constexpr int kScaleChunkBytes = 384 * 32;
// Rows of scales that are not whole 16 bytes: the 48 bytes, aligned, that hold a row's 32; or
// for K up to 1024 the rows as they lie in memory, the weight's and then the tile's.
constexpr int kRawChunks = 2, kRawChunkBytes = 384 * 48;
constexpr int kRawTile = 128 * 32 + 256;
static_assert(kRawChunks * kRawChunkBytes <= kScaleChunks * kScaleChunkBytes &&
                  kRawTile + 256 * 32 + 32 <= kRawChunkBytes,
              "in the same ring");
constexpr int kGrRelay = 16;           // bytes by which the odd CTA signals the even one
// Registers: as in the dense FP8 pairs, the first warpgroup gives up what the output
// warps, with up to 128 sums each, need.
constexpr int kGrRegsLaunch = 168, kGrRegsFew = 88, kGrRegsMany = 208;
static_assert(128 * kGrRegsFew + 256 * kGrRegsMany <= kGrThreads * kGrRegsLaunch,
              "register split within the launch's registers");

// SPLIT, over the pairs of a cluster: products of up to 32 rows in all, K in parts; weight
// gradients of few tiles, an expert's rows in parts.
constexpr int kGrSplitRows = 32, kGrMaxParts = 4, kGrPartStages = 12;
template <int MODE, bool SPLIT = false>
struct GrGeo {
  static constexpr bool FP4 = MODE == kFp4 || MODE == kFp4Rows, WG = MODE == kWeightGrad;
  static constexpr bool A_MN = MODE == kProduct || WG;  // MN-major first operand
  static constexpr int BK = FP4 ? 256 : 64;    // reduced elements of a stage (128 bytes of a row)
  // columns of a tile; FP4: two accumulators and the scales share the 512 TMEM columns
  static constexpr bool FEW = SPLIT && !WG;    // rows
  static constexpr int TM = FEW ? kGrSplitRows : FP4 ? 224 : 256;
  static constexpr int ACC = FP4 ? 224 : 256;  // TMEM columns from one accumulator to the other
  static constexpr int SCALES = FP4 ? (128 + 256) * 8 : 0;  // of a stage: 128 + 256 rows by 8 bytes
  static constexpr int SCALES_AT = FEW ? 18432 : 32768;  // A, then TM / 2 rows or columns of B
  static constexpr int STAGE = SCALES_AT + SCALES;
  static constexpr int STAGES = FEW ? (FP4 ? 6 : 8) : FP4 ? 5 : 6;
  // the other parts' sums, [part][4 columns][128 lanes] of 16 bytes (weight grad: the stages')
  static constexpr int PARTS = FEW ? (kGrMaxParts - 1) * kGrSplitRows * 128 * 4 : 0;
  static constexpr int SCALE_RING = FP4 ? kScaleChunks * kScaleChunkBytes : 0;
  static constexpr size_t SMEM = 1024 + STAGES * STAGE + SCALE_RING + PARTS;
};
constexpr uint32_t kScaleCol = 448;  // TMEM columns of FP4's scales, 24 for each of two stages

// Where a row's half of a chunk is among 32 rows: the halves change places with every fourth
// row, so that 8 rows' halves, read together, are in all banks.
__device__ __forceinline__ int scale_place(int row, int half) {
  return row * 32 + ((half ^ (row >> 2 & 1)) << 4);
}

template <int MODE, bool SPLIT>
struct GrCtl {
  static constexpr int S = GrGeo<MODE, SPLIT>::STAGES;
  uint64_t full[S], empty[S];
  uint64_t tail[S];               // weight grad: the expert's last rows; FP4: the odd CTA's scales
  uint64_t tmem_full[2], tmem_empty[2];
  uint64_t scales_full[kScaleChunks], scales_empty[kScaleChunks];  // FP4
  uint32_t tmem_base;
  int32_t abort;
  // the odd CTA signals by a copy of 16 bytes into relay[stage] of the even one, which
  // completes on that CTA's full barrier the way its loads do (an arrival with release at
  // cluster scope waits for the thread's memory operations in flight, ~1000 cycles)
  alignas(16) uint8_t relay[S][kGrRelay];
  alignas(16) uint8_t relay_src[kGrRelay];
  int64_t blocks;                 // stages that this CTA's loads went through
  int32_t total;                  // tiles
  int32_t start[kGrMaxExperts];   // first row and rows of each expert
  int32_t count[kGrMaxExperts];
  int32_t tile0[kGrMaxExperts];   // its first tile (products)
};
static_assert(kGrSplitRows / 2 == 16, "the boxes of 16 rows are a CTA's half of these tiles");
static_assert(GrGeo<kFp4>::SMEM + sizeof(GrCtl<kFp4, false>) <= 232448 &&
                  GrGeo<kFp4, true>::SMEM + sizeof(GrCtl<kFp4, true>) <= 232448 &&
                  GrGeo<kProduct>::SMEM + sizeof(GrCtl<kProduct, false>) <= 232448 &&
                  GrGeo<kProduct, true>::SMEM + sizeof(GrCtl<kProduct, true>) <= 232448 &&
                  GrGeo<kWeightGrad>::SMEM + sizeof(GrCtl<kWeightGrad, false>) <= 232448 &&
                  GrGeo<kWeightGrad, true>::SMEM + sizeof(GrCtl<kWeightGrad, true>) <= 232448,
              "shared memory budget");

// dense_wait, which also ends at once where a wait of this CTA has run out: the loops of the
// loading and issuing warps go on to the tile's end then.
__device__ __forceinline__ bool gr_wait(uint64_t* bar, uint32_t parity, int32_t* abort,
                                        int32_t* err) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  if (*reinterpret_cast<volatile int32_t*>(abort)) return false;
  return dense_wait(bar, parity, abort, err);
}

// n / d for 0 <= n < 2^31: with d in (2^(l-1), 2^l] and m = ceil(2^(31+l) / d), n m is
// 2^(31+l) n / d + n e, 0 <= e < d, and n e < 2^(31+l) carries it to no next whole number.
struct GrDiv {
  uint32_t m = 0, shift = 0;
  GrDiv() = default;
  explicit GrDiv(int64_t d) {
    while ((int64_t(1) << shift) < d) ++shift;
    shift += 31;
    m = static_cast<uint32_t>(((uint64_t(1) << shift) + d - 1) / d);
  }
  __device__ __forceinline__ int operator()(int n) const {
    return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(n)) * m >> shift);
  }
};

struct GrParams {
  const int32_t* offsets;  // [E + 1], or null: all R rows are expert 0's
  int64_t R;
  int E, K, N;             // weight grad: K rows of dW
  const bf16* bias;        // [E, N] or null
  const uint8_t* x_scale;  // FP4: [R, K / 32], [E, N, K / 32]
  const uint8_t* w_scale;
  void* out;
  int out_f32, accumulate;
  int parts;               // SPLIT: of K
  int chunk;               // stages summed in the tensor core before they go to registers
  GrDiv raster;            // by the tiles of a raster group (products)
  int32_t* error_word;
};

// Tensor maps: the weight (or dy), the rows in boxes of half a tile's columns (only calls of
// more rows than tiles with one less 32 take have such tiles; the others go without the map,
// whose making is part of a small call's time) and of 16, and FP4's scales of both.
struct GrMaps {
  CUtensorMap a, b, b16, sa, sb;
};

struct GrTile {
  int e, n0;        // expert, first column of the weight
  int64_t c0;       // first row of y, or of dW[e]
  int cols, T;      // how many, and rounded up to what the MMA takes
  int r0, rows;     // the expert's rows (weight grad in parts: the part's)
};

// By whole warps: their lanes look for the expert together.  (Products, without divisions in
// most calls: 650 cycles of each tile before, a seventh of a short sum's tile.  The weight
// gradient's short sums were 3 % slower so.)
template <int MODE, bool SPLIT>
__device__ __forceinline__ GrTile gr_tile(const GrCtl<MODE, SPLIT>& ctl, const GrParams& P, int t) {
  using G = GrGeo<MODE, SPLIT>;
  const int nt = ceil_div(P.N, 256);
  GrTile tl;
  int r, ct;  // tile within the expert, column tiles (of y's rows or dW's)
  if constexpr (G::WG) {
    ct = ceil_div(P.K, G::TM);
    tl.e = t / (ct * nt);
    r = t - tl.e * (ct * nt);
  } else {
    // the last expert whose first tile is not behind t: of each 32nd, then of 32
    const int lane = threadIdx.x & 31;
    int e = 0;
#pragma unroll
    for (int step = 32; step > 0; step -= 31) {
      if (step == 32 && P.E <= 32) continue;
      const int i = e + lane * step;
      e += (__popc(__ballot_sync(0xffffffffu, i < P.E && ctl.tile0[min(i, P.E - 1)] <= t)) - 1) * step;
    }
    tl.e = e;
    r = t - ctl.tile0[e];
    ct = ceil_div(ctl.count[e], G::TM);
  }
  tl.r0 = ctl.start[tl.e];
  tl.rows = ctl.count[tl.e];
  if constexpr (G::WG && SPLIT) {  // this part's of them, whole stages but for the last
    const int part = static_cast<int>(ptx::cluster_ctarank()) / 2, blocks = ceil_div(tl.rows, G::BK);
    const int first = static_cast<int>(int64_t(blocks) * part / P.parts) * G::BK;
    const int end = static_cast<int>(int64_t(blocks) * (part + 1) / P.parts) * G::BK;
    tl.rows = min(tl.rows, end) - first;
    tl.r0 += first;
  }
  // raster groups of kGrGroup column tiles by all weight tiles, columns innermost: tiles in
  // flight together share the weight's columns and the rows in L2
  const int per = kGrGroup * nt;
  const int g = G::WG ? r / per : P.raster(r), q = r - g * per;
  const int in_group = min(kGrGroup, ct - g * kGrGroup);
  const int nq = !G::WG && in_group == kGrGroup ? q / kGrGroup : q / in_group;
  const int c = (g * kGrGroup + q - nq * in_group) * G::TM;
  tl.n0 = nq * 256;
  tl.cols = min(G::TM, (G::WG ? P.K : tl.rows) - c);
  tl.c0 = G::WG ? c : static_cast<int64_t>(tl.r0) + c;
  // (MN-major columns come in swizzled chunks of 64 per CTA)
  tl.T = G::WG ? (tl.cols > 128 ? 256 : 128) : (tl.cols + 31) & ~31;
  return tl;
}

// The tile as one value of the warp, for loops whose values have to be known as uniform:
// a reduction's result is, a shared-memory load's is not (with loop bounds loaded from there
// an MMA of the weight gradient took 80 cycles to issue, 26 with these).
__device__ __forceinline__ int warp_value(int v) {
  return static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<unsigned>(v)));
}
__device__ __forceinline__ GrTile warp_value(const GrTile& t) {  // (all fields are >= 0)
  return GrTile{warp_value(t.e),    warp_value(t.n0), warp_value(static_cast<int>(t.c0)),
                warp_value(t.cols), warp_value(t.T),  warp_value(t.r0),
                warp_value(t.rows)};
}

// Stages of a tile, of the part of K that is this pair's: from the first one on.
struct GrRange {
  int first, count;
};
template <int MODE, bool SPLIT>
__device__ __forceinline__ GrRange gr_blocks(const GrParams& P, const GrTile& tl, int part,
                                             int parts) {
  using G = GrGeo<MODE, SPLIT>;
  const int KB = ceil_div(G::WG ? tl.rows : P.K, G::BK);
  if constexpr (!G::FEW) return GrRange{0, KB};
  constexpr int UNIT = G::FP4 ? 4 : 1;  // (FP4: whole chunks of scales)
  const int units = ceil_div(KB, UNIT);
  const int first = units * part / parts * UNIT, last = min(units * (part + 1) / parts * UNIT, KB);
  return GrRange{first, last - first};
}

// ---- MX FP4 instructions ----
// Scales from shared memory to TMEM: 128 rows by 4 bytes, row r at (r % 32) * 16 + r / 32 * 4,
// become 4 columns, repeated for the four warps' lanes, in both CTAs of the pair.
__device__ __forceinline__ void copy_scales_pair_if(uint32_t go, uint32_t tmem, uint32_t saddr) {
  // no swizzle, 8-row groups 128 bytes apart
  asm volatile(
      "{\n\t.reg .pred q;\n\t.reg .b64 d;\n\tmov.b64 d, {%1, %2};\n\tsetp.ne.b32 q, %3, 0;\n\t"
      "@q tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], d;\n\t}" ::"r"(tmem),
      "r"(saddr >> 4), "r"(8u | 1u << 14), "r"(go)
      : "memory");
}
__device__ __forceinline__ void mma_mxfp4_pair_if(uint32_t go, uint32_t d_tmem, uint32_t a_lo,
                                                  uint32_t b_lo, uint32_t hi, uint32_t idesc,
                                                  uint32_t sa, uint32_t sb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %3};\n\tmov.b64 b, {%2, %3};\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.ne.b32 q, %8, 0;\n\t"
      "@q tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], a, b, %4, [%6], [%7], p;\n\t}"
      ::"r"(d_tmem), "r"(a_lo), "r"(b_lo), "r"(hi), "r"(idesc), "r"(accumulate), "r"(sa), "r"(sb),
      "r"(go)
      : "memory");
}
// Instruction descriptor for kind::mxf4: bits 4-5 the byte pair of B's scales, 7-9 and
// 10-12 the types (1 = E2M1), 17-22 N >> 3, bit 23 UE8M0 scales, 24-28 M >> 4, 29-30 the
// byte pair of A's scales.
__device__ __forceinline__ uint32_t idesc_mxfp4(int M, int N, uint32_t scale_id) {
  return scale_id << 4 | 1u << 7 | 1u << 10 | static_cast<uint32_t>(N >> 3) << 17 | 1u << 23 |
         static_cast<uint32_t>(M >> 4) << 24 | scale_id << 29;
}

template <int MODE, bool SPLIT>
__global__ void __launch_bounds__(kGrThreads, 1)
    grouped_kernel(const __grid_constant__ GrMaps maps, const GrParams P) {
  using G = GrGeo<MODE, SPLIT>;
  pdl_begin();
  extern __shared__ uint8_t smem_raw[];
  __shared__ GrCtl<MODE, SPLIT> ctl;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // the pair's rank in the cluster, this CTA's in the pair
  const int cta = SPLIT ? warp_value(static_cast<int>(ptx::cluster_ctarank()))
                        : static_cast<int>(ptx::cluster_ctarank());
  const int even = SPLIT ? cta & ~1 : 0;  // the even CTA of the pair
  const int rank = cta - even;
  const int part = even / 2, parts = SPLIT ? P.parts : 1;
  const uint16_t both = static_cast<uint16_t>(3u << even);
  uint8_t* tiles = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  // The odd CTA's word that stage's part of it is in place: its scales, or its cleared tail.
  // Their writers fence them to the async proxy before they arrive on the tail barrier that
  // the sender of this copy waits for (or sent it themselves), and the copy is of that proxy
  // and behind them.  That its completion on the even CTA's barrier makes them visible to the
  // pair's MMA rests on this: they are read by the tensor core of the SM that wrote them, as what
  // TMA loads there is, whose completion reaches the even CTA the same way.  The PTX memory
  // model itself promises a completed copy's own bytes only.
  auto relay = [&](int stage) {
    ptx::bulk_copy_to_cluster(ptx::mapa_shared(ptx::smem_u32(ctl.relay[stage]), even), ctl.relay_src,
                              kGrRelay, ptx::mapa_shared(ptx::smem_u32(&ctl.full[stage]), even));
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < G::STAGES; ++i) {
      // full: the loads of both CTAs (one arrival); weight grad: one more, for the even CTA's
      // tail; FP4: one more, for its scales
      ptx::mbar_init(&ctl.full[i], G::WG || G::FP4 ? 2 : 1);
      ptx::mbar_init(&ctl.empty[i], 1);
      ptx::mbar_init(&ctl.tail[i], 1);
    }
    for (int i = 0; i < kScaleChunks; ++i) {
      ptx::mbar_init(&ctl.scales_full[i], MODE == kFp4Rows && P.K > 1024 ? 32 : 1);
      ptx::mbar_init(&ctl.scales_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&ctl.tmem_full[i], 1);
      ptx::mbar_init(&ctl.tmem_empty[i], 2 * 8);  // the output warps of both CTAs
    }
    ctl.abort = 0;
    ctl.blocks = 0;
    ptx::fence_barrier_init();
    ptx::prefetch_tmap(&maps.a);
    ptx::prefetch_tmap(&maps.b);
    ptx::prefetch_tmap(&maps.b16);
    if (G::FP4) {
      ptx::prefetch_tmap(&maps.sa);
      ptx::prefetch_tmap(&maps.sb);
    }
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(&ctl.tmem_base, 512);
    ptx::tmem_relinquish_pair();
  }
  const int nt = ceil_div(P.N, 256);
  if (warp == 2) {
    // the experts' rows and their tiles.  Offsets are clipped to the R rows there are, and to
    // the ends of the experts before: whatever they hold, no two experts share a row.
    int total = 0;
    const int R = static_cast<int>(P.R);
    int end = 0;  // of the experts before
    for (int e0 = 0; e0 < P.E; e0 += 32) {
      const int e = e0 + lane;
      int n = 0, b0 = 0, c0 = R;
      if (P.offsets != nullptr && e < P.E) {
        b0 = __ldg(P.offsets + e);
        c0 = __ldg(P.offsets + e + 1);
      }
      int ends = e < P.E ? min(max(c0, 0), R) : 0;  // the largest of this lane's and those before
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, ends, o);
        if (lane >= o) ends = max(ends, v);
      }
      int before = __shfl_up_sync(0xffffffffu, ends, 1);
      before = max(end, lane > 0 ? before : 0);
      end = max(end, __shfl_sync(0xffffffffu, ends, 31));
      if (e < P.E) {
        const int b = max(min(max(b0, 0), R), before);
        const int c = max(min(max(c0, 0), R), b);
        if (b != b0 || c != c0) record_error(P.error_word, MOE_ERR_INVALID_ARG);
        ctl.start[e] = b;
        ctl.count[e] = c - b;
        n = ceil_div(c - b, G::TM) * nt;
      }
      if constexpr (!G::WG) {
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += v;
        }
        if (e < P.E) ctl.tile0[e] = total + sum - n;
        total += __shfl_sync(0xffffffffu, sum, 31);
      }
    }
    if (lane == 0) ctl.total = G::WG ? P.E * ceil_div(P.K, G::TM) * nt : total;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = warp_value(ctl.tmem_base);
  const int total = warp_value(ctl.total);
  // (SPLIT: as many clusters as tiles at least)
  const int unit = static_cast<int>(blockIdx.x) / (2 * parts);
  const int units = static_cast<int>(gridDim.x) / (2 * parts);

  if (warp < 4) {
    if constexpr (!G::FEW) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kGrRegsFew));
    // (The loading and the issuing warp run their loops as one, an elected lane issuing: in a
    // branch of one lane an MMA took 70 cycles to issue, the loop 730 for the 512 that a stage
    // of 256 columns computes.  8 x 1024 rows, K 4096, N 28672: 1193 us so, 1077 as here;
    // the weight gradient of 128 x 1024 rows, 2048 x 1536: 726 and 597.  A wait that ran out
    // does not end a loop before its tile's end: all others end at once then.)
    auto aborted = [&]() { return warp_value(*reinterpret_cast<volatile int32_t*>(&ctl.abort)) != 0; };
    if (warp == 0) {
      // ---- loads ----
      const uint32_t go = ptx::elect_one();
      const uint32_t tiles0 = ptx::smem_u32(tiles);
      int stage = 0;
      uint32_t phase = 0;
      int64_t blocks = 0;
      const uint32_t full0 = ptx::mapa_shared(ptx::smem_u32(&ctl.full[0]), even);
      const uint32_t tail0 = ptx::mapa_shared(ptx::smem_u32(&ctl.tail[0]), cta);
      for (int t = unit; t < total && !aborted(); t += units) {
        const GrTile tl = warp_value(gr_tile(ctl, P, t));
        const GrRange range = gr_blocks<MODE, SPLIT>(P, tl, part, parts);
        const int KB = range.count;
        const int half = tl.T / 2;
        const int n = tl.n0 + rank * 128, c = static_cast<int>(tl.c0) + rank * half;
        const uint32_t bytes = 16384u + static_cast<uint32_t>(half) * 128u;
        for (int kb = 0; kb < KB; ++kb) {
          gr_wait(&ctl.empty[stage], phase ^ 1u, &ctl.abort, P.error_word);
          const uint32_t sa = tiles0 + stage * G::STAGE, sb = sa + 16384;
          // both CTAs' copies complete on the even CTA's barrier
          uint32_t bar = full0 + stage * 8;
          if (G::WG && kb == KB - 1 && tl.rows % 16 != 0) {
            // the last rows of the expert: to this CTA's tail barrier, and on from there
            bar = tail0 + stage * 8;
            ptx::mbar_arrive_expect_tx_if(go, &ctl.tail[stage], bytes);
            if (rank == 0) ptx::mbar_arrive_expect_tx_if(go, &ctl.full[stage], kGrRelay);
          } else if (rank == 0) {
            ptx::mbar_arrive_expect_tx_if(go, &ctl.full[stage],
                                          2 * bytes + (G::FP4 ? kGrRelay : 0));
            if (G::WG) ptx::mbar_arrive_if(go, &ctl.full[stage]);
          }
          if constexpr (G::WG) {
            const int r = tl.r0 + kb * 64;
#pragma unroll
            for (int i = 0; i < 2; ++i)
              ptx::tma_load_2d_pair_if(go, sa + i * 8192, &maps.a, bar, n + i * 64, r);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (i < half / 64)
                ptx::tma_load_2d_pair_if(go, sb + i * 8192, &maps.b, bar, c + i * 64, r);
          } else {
            const int k = (range.first + kb) * (G::FP4 ? 128 : 64);  // bytes, or elements
            if constexpr (MODE == kProduct) {
#pragma unroll
              for (int i = 0; i < 2; ++i)
                ptx::tma_load_3d_pair_if(go, sa + i * 8192, &maps.a, bar, n + i * 64, k, tl.e);
            } else {
              ptx::tma_load_3d_pair_if(go, sa, &maps.a, bar, k, n, tl.e);
            }
            if (SPLIT || tl.T == G::TM) {
              ptx::tma_load_2d_pair_if(go, sb, &maps.b, bar, k, c);
            } else {
              for (int i = 0; i < half; i += 16)
                ptx::tma_load_2d_pair_if(go, sb + i * 128, &maps.b16, bar, k, c + i);
            }
          }
          ++blocks;
          if (++stage == G::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
      if (lane == 0) ctl.blocks = blocks;
    } else if (warp == 1 && rank == 0) {
      // ---- MMAs ----
      const uint32_t go = ptx::elect_one();
      // (descriptors hold 18 bits of an address; above them is the CTA's place in the cluster)
      const uint32_t tiles0 = ptx::smem_u32(tiles) & 0x3ffffu;
      constexpr uint32_t HI = 64u | 1u << 14 | 2u << 29;  // (8-row groups 1024 bytes apart)
      // K-major: 32 bytes of a row per step; MN-major: 16 rows, chunks of 64 columns 8192 apart
      constexpr uint32_t A_STEP = G::A_MN ? 128 : 2, B_STEP = G::WG ? 128 : 2;
      constexpr uint32_t A_LO = (G::A_MN ? 512u : 1u) << 16, B_LO = (G::WG ? 512u : 1u) << 16;
      int stage = 0;
      uint32_t phase = 0, acc = 0, turn = 0, block = 0;
      for (int t = unit; t < total && !aborted(); t += units) {
        const GrTile tl = warp_value(gr_tile(ctl, P, t));
        const int KB = gr_blocks<MODE, SPLIT>(P, tl, part, parts).count;
        const uint32_t idesc = ptx::idesc_bf16_f32(256, tl.T, G::A_MN, G::WG);
        int in_chunk = 0;
        // one stage's MMAs, of `rows` of K; end: the tile's last
        auto stage_mmas = [&](auto rows, bool end) {
          [[maybe_unused]] const int steps = rows;
          if (in_chunk == 0)
            gr_wait(&ctl.tmem_empty[acc], turn ^ 1u, &ctl.abort, P.error_word);
          gr_wait(&ctl.full[stage], phase, &ctl.abort, P.error_word);
          ptx::tc_fence_after();
          const uint32_t sa = tiles0 + stage * G::STAGE;
          const uint32_t a = (sa >> 4) + A_LO, b = ((sa + 16384) >> 4) + B_LO;
          const uint32_t d = tmem + acc * static_cast<uint32_t>(G::ACC);
          if constexpr (G::FP4) {
            const uint32_t sc = tmem + kScaleCol + (block & 1u) * 24u, ss = sa + G::SCALES_AT;
#pragma unroll
            for (int ka = 0; ka < 2; ++ka) {
              copy_scales_pair_if(go, sc + ka * 4, ss + ka * 512);
              copy_scales_pair_if(go, sc + 8 + ka * 8, ss + 1024 + ka * 1024);
              copy_scales_pair_if(go, sc + 12 + ka * 8, ss + 1536 + ka * 1024);
            }
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              mma_mxfp4_pair_if(go, d, a + ks * A_STEP, b + ks * B_STEP, HI,
                                idesc_mxfp4(256, tl.T, (ks & 1) * 2), sc + (ks >> 1) * 4,
                                sc + 8 + (ks >> 1) * 8, (in_chunk | ks) != 0);
          } else {
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              ptx::mma_bf16_pair_if(ks * 16 < steps ? go : 0, d, a + ks * A_STEP, b + ks * B_STEP,
                                    HI, idesc, (in_chunk | ks) != 0);
          }
          const bool last = ++in_chunk == P.chunk || end;
          if (last) ptx::mma_commit_pair_if(go, &ctl.tmem_full[acc], both);
          ptx::mma_commit_pair_if(go, &ctl.empty[stage], both);
          if (last) {
            in_chunk = 0;
            acc ^= 1u;
            turn ^= acc == 0 ? 1u : 0u;
          }
          if (++stage == G::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
          ++block;
        };
        // (the weight gradient's last stage by itself: with MMAs that depend on its rows
        // in the loop, a stage took 740 cycles, 579 so)
        for (int kb = 0; kb < KB - G::WG; ++kb)
          stage_mmas(std::integral_constant<int, 64>{}, !G::WG && kb == KB - 1);
        if (G::WG && KB > 0) stage_mmas(tl.rows - (KB - 1) * 64, true);
      }
    } else if (G::FP4 && warp == 1 && lane == 0) {
      // ---- odd CTA: a stage's scales are in place ----
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      const int KB = gr_blocks<MODE, SPLIT>(P, GrTile{}, part, parts).count;
      for (int t = unit; t < total && ok; t += units) {
        for (int kb = 0; kb < KB; ++kb) {
          if (!gr_wait(&ctl.tail[stage], phase, &ctl.abort, P.error_word)) {
            ok = false;
            break;
          }
          relay(stage);
          if (++stage == G::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    } else if (G::WG && warp == 2) {
      // ---- tails: rows of the last 16 that are not the expert's become zeros ----
      // (they are the next expert's, or nobody's, and may hold anything)
      int64_t block = 0;
      uint32_t parity = 0;  // of each stage's tail barrier
      bool ok = true;
      for (int t = unit; t < total && ok; t += units) {
        const GrTile tl = gr_tile(ctl, P, t);
        const int KB = gr_blocks<MODE, SPLIT>(P, tl, part, parts).count;
        block += KB;
        if (tl.rows % 16 == 0) continue;
        const int stage = static_cast<int>((block - 1) % G::STAGES);
        const bool got =
            gr_wait(&ctl.tail[stage], parity >> stage & 1u, &ctl.abort, P.error_word);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        parity ^= 1u << stage;
        const int last = tl.rows - (KB - 1) * 64;        // rows of the block
        const int clear = ((last + 15) & ~15) - last;    // 1 to 15
        uint8_t* base = tiles + stage * G::STAGE + last * 128;
        // units of 16 bytes: 8 of a row, in each operand's chunks of 64 columns
        for (int i = lane; i < clear * 8 * 4; i += 32) {
          const int chunk = i / (clear * 8), u = i - chunk * (clear * 8);
          *reinterpret_cast<uint4*>(base + chunk * 8192 + u * 16) = make_uint4(0, 0, 0, 0);
        }
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          if (rank == 0)
            ptx::mbar_arrive(&ctl.full[stage]);
          else
            relay(stage);
        }
      }
    } else if (G::FP4 && warp == 2) {
      // ---- scales into shared memory, of the weight's 128 rows and the tile's 256, 32 bytes
      // of a row (a chunk: 1024 elements, four stages) at a time, into a ring ----
      // By TMA where rows of scales are whole 16 bytes (K a multiple of 512); else for K up to
      // 1024 as the rows lie in memory, in bulk copies; else by the warp's lanes, a row
      // each, in asynchronous copies.  Those are as many requests as lanes, and slower
      // than the MMAs (8192 x 7168 x 4096: 155 us from registers, 93-100 by asynchronous
      // copies, 83 by TMA, 78 without any; 8192 x 7200 x 4096: 209; a bulk copy for each
      // row 849; 32768 rows of 64 experts, K 768, N 2048: 88 by the lanes, 74 in bulk).
      // The warp that takes the scales from the ring is another one: its fence for the
      // tensor core's reads would wait for copies in flight.
      const int KG = P.K / 32;
      uint8_t* ring = tiles + G::STAGES * G::STAGE;
      const uint32_t go = ptx::elect_one();
      int slot = 0;
      uint32_t phase = 0;
      for (int t = unit; t < total && !aborted(); t += units) {
        const GrTile tl = warp_value(gr_tile(ctl, P, t));
        const int n = tl.n0 + rank * 128;
        const GrRange range = gr_blocks<MODE, SPLIT>(P, tl, part, parts);
        const int last = min((range.first + range.count) * 8, KG);
        for (int g = range.first * 8; g < last; g += 32) {
          gr_wait(&ctl.scales_empty[slot], phase ^ 1u, &ctl.abort, P.error_word);
          uint64_t* bar = &ctl.scales_full[slot];
          if constexpr (MODE == kFp4) {
            // (rows and scales that are not there are read as zeros, 2^-127; past K the codes
            // are zeros too)
            uint8_t* dst = ring + slot * kScaleChunkBytes;
            ptx::mbar_arrive_expect_tx_if(go, bar, tl.T > 128 ? 12288 : 8192);
            ptx::tma_load_3d_if(go, dst, &maps.sa, bar, g, n, tl.e);
            ptx::tma_load_2d_if(go, dst + 4096, &maps.sb, bar, g, static_cast<int>(tl.c0));
            if (tl.T > 128)
              ptx::tma_load_2d_if(go, dst + 8192, &maps.sb, bar, g, static_cast<int>(tl.c0) + 128);
          } else if (KG <= 32) {
            // the rows that are there, in one piece each of the two tensors
            if (go) {
              uint8_t* dst = ring + slot * kRawChunkBytes;
              const RawSpan span[2] = {weight_scale_span(P.E, P.N, KG, tl.e, n),
                                       row_scale_span(P.R, KG, tl.c0, tl.T)};
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint8_t* src = i == 0 ? P.w_scale : P.x_scale;
                // (a tensor's last bytes)
                for (int64_t q = span[i].begin + span[i].bulk; q < span[i].end; ++q)
                  dst[i * kRawTile + static_cast<int>(q - span[i].begin)] = __ldg(src + q);
              }
              ptx::mbar_arrive_expect_tx(bar, span[0].bulk + span[1].bulk);
#pragma unroll
              for (int i = 0; i < 2; ++i)
                if (span[i].bulk > 0)
                  ptx::bulk_load(dst + i * kRawTile,
                                 (i == 0 ? P.w_scale : P.x_scale) + span[i].begin, span[i].bulk, bar);
            }
            __syncwarp();
          } else {
            // row lane + 32 i: zeros where it is not there, and nothing read past the tensor
            uint8_t* dst = ring + slot * kRawChunkBytes + lane * 16;
            const int64_t wrow = static_cast<int64_t>(tl.e) * P.N + n;
            const int64_t wend = static_cast<int64_t>(P.E) * P.N * KG, xend = P.R * KG;
#pragma unroll 4
            for (int i = 0; i < 12; ++i) {
              const int r = lane + 32 * (i < 4 ? i : i - 4);
              const bool in = i < 4 ? n + r < P.N : r < tl.T && tl.c0 + r < P.R;
              const uint8_t* base = i < 4 ? P.w_scale : P.x_scale;
              const int64_t at = ((i < 4 ? wrow : tl.c0) + r) * KG + g, from = at & ~int64_t(15);
              const int64_t need = at + min(32, KG - g), end = i < 4 ? wend : xend;
#pragma unroll
              for (int j = 0; j < 3; ++j) {
                const int64_t f = from + 16 * j;
                const bool there = in && f < need;
                ptx::cp_async_16(dst + (i * 3 + j) * 512, there ? base + f : base,
                                 there ? static_cast<uint32_t>(min(end - f, int64_t(16))) : 0u);
              }
            }
            ptx::cp_async_arrive(bar);
          }
          if (++slot == (MODE == kFp4 ? kScaleChunks : kRawChunks)) {
            slot = 0;
            phase ^= 1u;
          }
        }
      }
      ptx::cp_async_wait_all();
    } else if (G::FP4 && warp == 3) {
      // ---- and on to where the tensor core's copy takes them: there, 16 bytes are 128
      // elements' scales of a lane's four rows ----
      const uint8_t* ring = tiles + G::STAGES * G::STAGE;
      int stage = 0, slot = 0;
      uint32_t phase = 0, slot_phase = 0;
      bool ok = true;
      const GrRange range = gr_blocks<MODE, SPLIT>(P, GrTile{}, part, parts);
      const int KB = range.count;
      auto chunk_in = [&]() {
        const bool got = gr_wait(&ctl.scales_full[slot], slot_phase, &ctl.abort, P.error_word);
        return __all_sync(0xffffffffu, got);
      };
      auto chunk_out = [&]() {
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(&ctl.scales_empty[slot]);
        if (++slot == (MODE == kFp4 ? kScaleChunks : kRawChunks)) {
          slot = 0;
          slot_phase ^= 1u;
        }
      };
      // a stage's scales: of row lane + 32 i of the weight (i < 4) and of the tile, two words
      auto put_stage = [&](auto word) {
        const bool got = gr_wait(&ctl.empty[stage], phase ^ 1u, &ctl.abort, P.error_word);
        if (!__all_sync(0xffffffffu, got)) return false;
        uint8_t* sc = tiles + stage * G::STAGE + G::SCALES_AT + lane * 16;
#pragma unroll
        for (int a = 0; a < 3; ++a)  // the weight's rows, the tile's first 128, its others
#pragma unroll
          for (int ka = 0; ka < 2; ++ka)
            *reinterpret_cast<uint4*>(sc + (a == 0 ? ka * 512 : 1024 + ka * 1024 + (a - 1) * 512)) =
                make_uint4(word(4 * a, ka), word(4 * a + 1, ka), word(4 * a + 2, ka),
                           word(4 * a + 3, ka));
        ptx::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive(rank == 0 ? &ctl.full[stage] : &ctl.tail[stage]);
        if (++stage == G::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
        return true;
      };
      if constexpr (MODE == kFp4) {
        for (int t = unit; t < total && ok; t += units) {
          for (int kb = 0; kb < KB && ok; kb += 4) {
            if (!chunk_in()) {
              ok = false;
              break;
            }
#pragma unroll
            for (int b = 0; b < 4; b += 2) {  // two stages: 16 bytes of a row
              if (kb + b >= KB || !ok) break;
              uint32_t v[12][4];
#pragma unroll
              for (int i = 0; i < 12; ++i) {
                const uint4 u = *reinterpret_cast<const uint4*>(
                    ring + slot * kScaleChunkBytes + i * 1024 + scale_place(lane, b >> 1));
                v[i][0] = u.x;
                v[i][1] = u.y;
                v[i][2] = u.z;
                v[i][3] = u.w;
              }
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                if (kb + b + h >= KB || !ok) break;
                ok = put_stage([&](int i, int ka) { return v[i][2 * h + ka]; });
              }
            }
            chunk_out();
          }
        }
      } else {
        // from rows at any place: the 8 bytes of a stage, from two aligned 8s, by bytes, or
        // by words where all rows begin at whole ones
        const int KG = P.K / 32;
        auto run = [&](auto unit_bytes) {
          constexpr uint32_t UNIT = decltype(unit_bytes)::value;
          for (int t = unit; t < total && ok; t += units) {
            const GrTile tl = gr_tile(ctl, P, t);
            const int n = tl.n0 + rank * 128;
            // where the first row of the weight and of the tile begins, mod 16
            const uint32_t w0 = (static_cast<uint32_t>(tl.e) * P.N + n) * static_cast<uint32_t>(KG);
            const uint32_t x0 = static_cast<uint32_t>(tl.c0) * static_cast<uint32_t>(KG);
            for (int kb = 0; kb < KB && ok; ++kb) {
              const int h = kb & 3, g = (range.first + kb - h) * 8;  // stage of the chunk, its start
              if (h == 0 && !chunk_in()) {
                ok = false;
                break;
              }
              uint32_t v[12][2];
#pragma unroll
              for (int i = 0; i < 12; ++i) {
                const int r = lane + 32 * (i < 4 ? i : i - 4);
                const uint8_t* raw = ring + slot * kRawChunkBytes;
                uint32_t at;  // of the stage's bytes, from raw on
                bool in = true;
                if (KG <= 32) {
                  at = ((i < 4 ? w0 : x0) & 15u) + r * KG + 8 * h;
                  raw += i < 4 ? 0 : kRawTile;
                  in = i < 4 ? n + r < P.N : r < tl.T && tl.c0 + r < P.R;
                } else {
                  at = (((i < 4 ? w0 : x0) + r * KG + g) & 15u) + 8 * h;
                  raw += i * 1536 + lane * 16;
                }
                auto eight = [&](uint32_t o) {  // at a multiple of 8
                  const uint8_t* from = raw + (KG <= 32 ? o : (o >> 4) * 512 + (o & 8u));
                  return in ? *reinterpret_cast<const uint2*>(from) : make_uint2(0, 0);
                };
                const uint2 lo = eight(at & ~7u);
                if constexpr (UNIT == 8) {
                  v[i][0] = lo.x;
                  v[i][1] = lo.y;
                } else {
                  const uint2 hi = eight((at & ~7u) + 8);
                  const uint32_t a = at & 4u ? lo.y : lo.x, b = at & 4u ? hi.x : lo.y;
                  const uint32_t c = at & 4u ? hi.y : hi.x;
                  v[i][0] = UNIT == 4 ? a : __funnelshift_r(a, b, 8 * (at & 3u));
                  v[i][1] = UNIT == 4 ? b : __funnelshift_r(b, c, 8 * (at & 3u));
                }
              }
              const int left = KG - g - 8 * h;  // scales of the row from here on (past them: 0)
              if (left < 8) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  const int bytes = min(max(left - 4 * k, 0), 4);
                  const uint32_t mask = bytes == 4 ? ~0u : (1u << (8 * bytes)) - 1u;
#pragma unroll
                  for (int i = 0; i < 12; ++i) v[i][k] &= mask;
                }
              }
              ok = put_stage([&](int i, int ka) { return v[i][ka]; });
              if (h == 3 || kb == KB - 1) chunk_out();
            }
          }
        };
        if (KG % 8 == 0)
          run(std::integral_constant<uint32_t, 8>{});
        else if (KG % 4 == 0)
          run(std::integral_constant<uint32_t, 4>{});
        else
          run(std::integral_constant<uint32_t, 1>{});
      }
    }
  } else {
    // ---- output: 32 columns n of the weight (lanes) by half of the tile's columns a warp ----
    if constexpr (!G::FEW) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kGrRegsMany));
    const int q = warp & 3, half = (warp - 4) >> 2;
    [[maybe_unused]] uint8_t* sums = tiles + G::STAGES * G::STAGE + G::SCALE_RING;
    const uint32_t empty0 = ptx::mapa_shared(ptx::smem_u32(&ctl.tmem_empty[0]), even);
    uint32_t acc = 0, turn = 0;
    bool ok = true;
    if (SPLIT && unit >= total) {  // (for the others of the CTA: theirs below)
      ptx::cluster_sync();
      if (G::WG) ptx::cluster_sync();
    }
    for (int t = unit; t < total && ok; t += units) {
      const GrTile tl = gr_tile(ctl, P, t);
      const int KB = gr_blocks<MODE, SPLIT>(P, tl, part, parts).count;
      const int n = tl.n0 + rank * 128 + q * 32 + lane;
      const int groups = tl.T / 32;  // of 16 columns
      const float b = P.bias != nullptr && n < P.N
                          ? __bfloat162float(P.bias[static_cast<int64_t>(tl.e) * P.N + n])
                          : 0.f;
      uint64_t sum[G::TM / 4];
#pragma unroll
      for (int j = 0; j < G::TM / 4; ++j) sum[j] = part == 0 ? pair_of(b, b) : 0;
      for (int kb = 0; kb < KB; kb += P.chunk) {
        const bool got = gr_wait(&ctl.tmem_full[acc], turn, &ctl.abort, P.error_word);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t ta = tmem + (static_cast<uint32_t>(q * 32) << 16) +
                            acc * static_cast<uint32_t>(G::ACC) + half * groups * 16;
        uint32_t v[2][16];
        ptx::tmem_ld_16cols(ta, v[0]);
#pragma unroll
        for (int i = 0; i < G::TM / 32; ++i) {
          if (i >= groups) break;
          tmem_wait(v[i & 1]);
          if (i + 1 < groups) {
            ptx::tmem_ld_16cols(ta + 16 * (i + 1), v[(i + 1) & 1]);
          } else {  // the accumulator is in registers
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_relaxed(empty0 + acc * 8);
          }
#pragma unroll
          for (int j = 0; j < 16; j += 2)
            sum[8 * i + j / 2] = add2(sum[8 * i + j / 2], pair_of(__uint_as_float(v[i & 1][j]),
                                                                  __uint_as_float(v[i & 1][j + 1])));
        }
        acc ^= 1u;
        turn ^= acc == 0 ? 1u : 0u;
      }
      // in parts: the groups of 16 columns go round the parts, each of which takes the others'
      // sums of its groups, where the stages were, adds them in order and writes them
      auto mine = [&](int i) { return !(G::WG && SPLIT) || (i & (parts - 1)) == part; };
      if constexpr (G::WG && SPLIT) {
        constexpr int GROUPS = G::TM / 32;
        const int each = GROUPS / parts;
        auto place = [&](int i, int from) {  // group i of part `from`, 16 bytes of a lane's 64
          const int owner = i & (parts - 1), slot = from - (from > owner ? 1 : 0);
          return ((((slot * each + i / parts) * 2 + half) * 4 + q) * 128 + lane) * 16;
        };
        static_assert((kGrMaxParts - 1) * (GROUPS / kGrMaxParts) * 8 * 2048 <= G::STAGES * G::STAGE &&
                          GROUPS / 2 * 8 * 2048 <= G::STAGES * G::STAGE, "room for the sums");
        __syncwarp();
        ptx::cluster_sync();  // every part's MMAs are through, its stages free
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) {
          if (i < groups && !mine(i)) {
            const uint32_t to = ptx::mapa_shared(ptx::smem_u32(tiles + place(i, part)),
                                                 2 * (i & (parts - 1)) + rank);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 x = unpair(sum[8 * i + 2 * j]), y = unpair(sum[8 * i + 2 * j + 1]);
              st_cluster_f32x4(to + j * 512, x.x, x.y, y.x, y.y);
            }
          }
        }
        __syncwarp();
        ptx::cluster_sync();
#pragma unroll
        for (int i = 0; i < GROUPS; ++i) {
          if (i < groups && mine(i)) {
            for (int p = 0; p < parts; ++p) {
              if (p == part) continue;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float4 v = *reinterpret_cast<const float4*>(tiles + place(i, p) + j * 512);
                sum[8 * i + 2 * j] = add2(sum[8 * i + 2 * j], pair_of(v.x, v.y));
                sum[8 * i + 2 * j + 1] = add2(sum[8 * i + 2 * j + 1], pair_of(v.z, v.w));
              }
            }
          }
        }
      }
      if constexpr (G::FEW) {
        // the other parts' sums to the first part's CTA of this rank, which adds them in order
        if (part > 0) {
          const uint32_t to = ptx::mapa_shared(
              ptx::smem_u32(sums + ((part - 1) * 8 + half * 4) * 2048 + (q * 32 + lane) * 16), rank);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 x = unpair(sum[2 * j]), y = unpair(sum[2 * j + 1]);
            st_cluster_f32x4(to + j * 2048, x.x, x.y, y.x, y.y);
          }
        }
        __syncwarp();
        ptx::cluster_sync();
        if (part > 0) break;
        for (int p = 1; p < parts; ++p) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 v = *reinterpret_cast<const float4*>(
                sums + ((p - 1) * 8 + half * 4 + j) * 2048 + (q * 32 + lane) * 16);
            sum[2 * j] = add2(sum[2 * j], pair_of(v.x, v.y));
            sum[2 * j + 1] = add2(sum[2 * j + 1], pair_of(v.z, v.w));
          }
        }
      }
      if (!ok) break;
      const int first = half * groups * 16;
      const int64_t row0 = (G::WG ? static_cast<int64_t>(tl.e) * P.K : 0) + tl.c0 + first;
      const int left = min(tl.cols - first, groups * 16);
      // Products: the sums change lanes among fours, so that a store is four rows of 32
      // neighbouring columns n, four columns a lane (FP4 64287 x 320 x 960 to bf16 83.6 -> 70.8
      // us, 14765 x 288 x 3456 64.2 -> 58.4; long sums the same to 3 % less.  Eight rows,
      // 16 bytes of bf16 a lane: 79.7 and 66.8).  Weight gradients: a store is 32 columns of one
      // row (short sums to bf16 10 % slower than by fours, longer ones to fp32 1.5 % faster,
      // accumulating ones 6 %; through shared memory and out in 16-byte stores: the same).
      auto put4 = [&](auto* out) {
        using O = std::remove_pointer_t<decltype(out)>;
        const int col = n & ~3;
        const int64_t step = 4 * static_cast<int64_t>(P.N);
        const bool b0 = lane & 1, b1 = lane & 2;
        O* p = out + (row0 + (lane & 3)) * P.N + col;
#pragma unroll
        for (int i = 0; i < G::TM / 32; ++i) {
          if (16 * i >= left) break;
          auto in = [&](int j) { return 16 * i + 4 * j + (lane & 3) < left && col < P.N; };
          if constexpr (sizeof(O) == 2) {  // two columns' values of a row a word first
            uint32_t h[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float2 o = unpair(sum[8 * i + j]);
              const uint32_t own = pack2(o.x, o.y);
              h[j] = __byte_perm(own, __shfl_xor_sync(0xffffffffu, own, 1), b0 ? 0x3276 : 0x5410);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t got = __shfl_xor_sync(0xffffffffu, b1 ? h[2 * j] : h[2 * j + 1], 2);
              if (in(j))
                *reinterpret_cast<uint2*>(p) =
                    b1 ? make_uint2(got, h[2 * j + 1]) : make_uint2(h[2 * j], got);
              p += step;
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 x = unpair(sum[8 * i + 2 * j]), y = unpair(sum[8 * i + 2 * j + 1]);
              const float gx = __shfl_xor_sync(0xffffffffu, b0 ? x.x : x.y, 1);
              const float gy = __shfl_xor_sync(0xffffffffu, b0 ? y.x : y.y, 1);
              const float2 u = b0 ? make_float2(gx, x.y) : make_float2(x.x, gx);
              const float2 v = b0 ? make_float2(gy, y.y) : make_float2(y.x, gy);
              const float g0 = __shfl_xor_sync(0xffffffffu, b1 ? u.x : v.x, 2);
              const float g1 = __shfl_xor_sync(0xffffffffu, b1 ? u.y : v.y, 2);
              if (in(j))
                *reinterpret_cast<float4*>(p) =
                    b1 ? make_float4(g0, g1, v.x, v.y) : make_float4(u.x, u.y, g0, g1);
              p += step;
            }
          }
        }
      };
      auto put = [&](auto* out, auto add) {
        using O = std::remove_pointer_t<decltype(out)>;
        O* p = out + row0 * P.N + n;
        auto row = [&](int c) { return p + static_cast<int64_t>(c) * P.N; };
        auto store = [&](int i, auto whole) {
          constexpr bool WHOLE = decltype(whole)::value;
          [[maybe_unused]] float old[16];
          if constexpr (decltype(add)::value) {
#pragma unroll
            for (int j = 0; j < 16; ++j)
              old[j] = WHOLE || 16 * i + j < left ? static_cast<float>(*row(16 * i + j)) : 0.f;
          }
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            float2 o = unpair(sum[8 * i + j / 2]);
            if constexpr (decltype(add)::value) {
              o.x += old[j];
              o.y += old[j + 1];
            }
            if (WHOLE || 16 * i + j < left) *row(16 * i + j) = static_cast<O>(o.x);
            if (WHOLE || 16 * i + j + 1 < left) *row(16 * i + j + 1) = static_cast<O>(o.y);
          }
        };
#pragma unroll
        for (int i = 0; i < G::TM / 32; ++i) {
          if (16 * i >= left) break;
          if (!mine(i)) continue;
          if (16 * i + 16 <= left)
            store(i, std::true_type{});
          else
            store(i, std::false_type{});
        }
      };
      auto put_as = [&](auto* out) {
        if (P.accumulate)
          put(out, std::true_type{});
        else
          put(out, std::false_type{});
      };
      if constexpr (!G::WG) {
        if (P.out_f32)
          put4(static_cast<float*>(P.out));
        else
          put4(static_cast<bf16*>(P.out));
      } else if (n < P.N) {
        if (P.out_f32)
          put_as(static_cast<float*>(P.out));
        else
          put_as(static_cast<bf16*>(P.out));
      }
      __syncwarp();
    }
  }
  __syncwarp();
  if (SPLIT && warp < 4) {  // the exchange of the parts' sums
    ptx::cluster_sync();
    if (G::WG) ptx::cluster_sync();
  }
  ptx::cluster_sync();
  // the commits of the last use of every stage have to arrive before the barriers' memory
  // goes: each of them (see the dense FP8 pairs)
  if (threadIdx.x < G::STAGES && ctl.blocks > static_cast<int64_t>(threadIdx.x)) {
    const int64_t g = ctl.blocks - 1 - threadIdx.x;
    dense_wait(&ctl.empty[g % G::STAGES], static_cast<uint32_t>(g / G::STAGES) & 1u, &ctl.abort,
               P.error_word);
  }
  if (*reinterpret_cast<volatile int32_t*>(&ctl.abort)) {
    // copies and MMAs in flight get time to land before their memory goes
    const uint64_t t0 = ptx::globaltimer_ns();
    while (ptx::globaltimer_ns() - t0 < 2000000ull) __nanosleep(1000);
  }
  __syncwarp();
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, 512);
  }
}

// Stages per accumulation.  The tensor core's accumulator drops what lies below its last bit
// at every addition instead of rounding (measured: a product of K = 14336 comes out 1.4e-5
// too small, in proportion to K), so that sums go to registers, where they are rounded to
// nearest, every 512 rows or columns where they leave in fp32 (FP4: 2048; an MMA is four
// times as deep), and every 1024 (4096) where they leave in bf16: 64 MMAs drop 1.5e-5 at
// most, whatever the sum's length, beside the output's own rounding of 4e-3 (2^22 positive
// products in the tensor core alone come out 2.4 % too small).  Against the whole sum there:
// 8192 rows of 8, 4096 x 28672, 1326 -> 1332 us; 131064 rows of 128, 1536 x 2048, 582 -> 575,
// their weight gradient 681 -> 684; 1 x 7168 x 4096 11.6 -> 11.7 (every 512: 1336, 578, 692
// and 11.8).
int gr_chunk(const GroupedProductArgs& a) { return a.out_f32 ? 8 : 16; }

// A launch with clusters of `ctas` (cfg.attrs: room for two).
void grouped_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* at, int ctas, unsigned grid,
                    size_t smem) {
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kGrThreads);
  cfg.dynamicSmemBytes = smem;
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = static_cast<unsigned>(ctas);
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
}

template <int MODE, bool SPLIT>
cudaError_t grouped_prepare(int* regs) {  // once per device
  static PerDevice attr;
  return attr.get(
      [](int* v) {
        cudaFuncAttributes fa;
        const cudaError_t e = cudaFuncGetAttributes(&fa, grouped_kernel<MODE, SPLIT>);
        if (e != cudaSuccess) return e;
        *v = fa.numRegs;
        return cudaFuncSetAttribute(grouped_kernel<MODE, SPLIT>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    static_cast<int>(GrGeo<MODE, SPLIT>::SMEM));
      },
      regs);
}

// How many clusters of `parts` pairs fit on the GPU at a time.
template <int MODE>
int clusters_that_fit(int parts) {
  int dev = 0, regs = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || grouped_prepare<MODE, true>(&regs) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  thread_local int room_dev = -1, room[kGrMaxParts + 1];
  if (dev != room_dev) {  // how many clusters fit: asked once per host thread and device
    for (int c = 2; c <= kGrMaxParts; ++c) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute at[2];
      grouped_config(cfg, at, 2 * c, 2 * c, GrGeo<MODE, true>::SMEM);
      if (cudaOccupancyMaxActiveClusters(&room[c], grouped_kernel<MODE, true>, &cfg) !=
          cudaSuccess) {
        cudaGetLastError();
        room[c] = 0;
      }
    }
    room_dev = dev;
  }
  return room[parts];
}

// Parts of K for a product of up to 32 rows, of `tiles` tiles at most and `units` that a part
// can be made of: as many as leave all clusters resident, where one part of K leaves
// SMs idle.  1 x 7168 x 4096: bf16 25.4 us in one part, 11.8 so; FP4 12.6 and 10.0; 2 x
// 14336 x 4096, an expert each: 49.1 and 37.4.  (The tiles are those of the experts that R rows
// can reach: counted by E, calls of fewer rows than experts would have fewer parts.)
template <int MODE>
int grouped_parts(const GroupedProductArgs& a, int64_t tiles, int units) {
  if (a.R > kGrSplitRows || tiles * 4 > a.num_sms) return 1;
  int parts = 1;
  for (int c = 2; c <= kGrMaxParts && c <= units && tiles <= clusters_that_fit<MODE>(c); ++c) parts = c;
  return parts;
}

template <int MODE, bool SPLIT>
moe_status_t launch_grouped(const char* name, const GroupedProductArgs& a, const GrMaps& maps,
                            int64_t tiles, int parts, cudaStream_t s) {
  int regs = 0;
  if (grouped_prepare<MODE, SPLIT>(&regs) != cudaSuccess)
    return set_error(MOE_ERR_CUDA, "attributes of %s: %s", name,
                     cudaGetErrorString(cudaGetLastError()));
  // fewer registers at launch would leave the output warps waiting for more
  if (!GrGeo<MODE, SPLIT>::FEW && regs < kGrRegsLaunch)
    return set_error(MOE_ERR_CUDA, "%s was compiled to %d registers, %d needed", name, regs,
                     kGrRegsLaunch);
  GrParams P{};
  P.offsets = a.offsets;
  P.R = a.R;
  P.E = a.E;
  P.K = a.K;
  P.N = a.N;
  P.bias = a.bias;
  P.x_scale = a.x_scale;
  P.w_scale = a.w_scale;
  P.out = a.out;
  P.out_f32 = a.out_f32;
  P.accumulate = a.accumulate;
  P.parts = parts;
  P.chunk = gr_chunk(a);
  P.raster = GrDiv(int64_t(kGrGroup) * ceil_div(a.N, 256));
  P.error_word = a.error_word;
  const int64_t clusters = SPLIT ? tiles : std::min<int64_t>(tiles, a.num_sms / 2);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  grouped_config(cfg, at, 2 * parts, static_cast<unsigned>(2 * parts * clusters),
                 GrGeo<MODE, SPLIT>::SMEM);
  cfg.stream = s;
  prof_before(name, s);
  cudaLaunchKernelEx(&cfg, grouped_kernel<MODE, SPLIT>, maps, P);
  prof_after(name, s);
  return check_launch(name);
}

// At most how many tiles a product has: an expert with rows has one more than whole ones.
int64_t product_tiles(const GroupedProductArgs& a, int TM) {
  return ceil_div(a.N, 256) * (a.R / TM + std::min<int64_t>(a.E, a.R));
}

moe_status_t map_2d(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t pitch,
                    uint32_t box_cols, uint32_t box_rows, CUtensorMapDataType type,
                    CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  const uint64_t d[2] = {cols, rows}, st[1] = {pitch};
  const uint32_t box[2] = {box_cols, box_rows};
  return encode_tensor_map(m, base, 2, d, st, box, type, swizzle);
}
moe_status_t map_3d(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t mats,
                    uint64_t pitch, uint32_t box_cols, uint32_t box_rows,
                    CUtensorMapDataType type,
                    CUtensorMapSwizzle swizzle = CU_TENSOR_MAP_SWIZZLE_128B) {
  const uint64_t d[3] = {cols, rows, mats}, st[2] = {pitch, pitch * rows};
  const uint32_t box[3] = {box_cols, box_rows, 1};
  return encode_tensor_map(m, base, 3, d, st, box, type, swizzle);
}

constexpr auto kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
constexpr auto kBytes = CU_TENSOR_MAP_DATA_TYPE_UINT8;

}  // namespace

moe_status_t launch_grouped_matmul(const GroupedProductArgs& a, cudaStream_t s) {
  const uint64_t K = a.K, N = a.N, E = a.E, R = static_cast<uint64_t>(a.R);
  const int64_t tiles = product_tiles(a, 256);
  const int units = ceil_div(a.K, 64) / 4;
  const int parts = a.transposed ? grouped_parts<kProductT>(a, tiles, units)
                                 : grouped_parts<kProduct>(a, tiles, units);
  GrMaps m;
  if (moe_status_t st = a.transposed ? map_3d(&m.a, a.w, K, N, E, 2 * K, 64, 128, kBf16)
                                     : map_3d(&m.a, a.w, N, K, E, 2 * N, 64, 64, kBf16))
    return st;
  if (moe_status_t st = map_2d(&m.b16, a.x, K, R, 2 * K, 64, 16, kBf16)) return st;
  m.b = m.b16;
  if (parts > 1)
    return a.transposed
               ? launch_grouped<kProductT, true>("grouped_matmul_t_split", a, m, tiles, parts, s)
               : launch_grouped<kProduct, true>("grouped_matmul_split", a, m, tiles, parts, s);
  if (a.R > 256 - 32)
    if (moe_status_t st = map_2d(&m.b, a.x, K, R, 2 * K, 64, 128, kBf16)) return st;
  return a.transposed ? launch_grouped<kProductT, false>("grouped_matmul_t", a, m, tiles, 1, s)
                      : launch_grouped<kProduct, false>("grouped_matmul", a, m, tiles, 1, s);
}

moe_status_t launch_grouped_weight_grad(const GroupedProductArgs& a, cudaStream_t s) {
  const uint64_t K = a.K, N = a.N, R = static_cast<uint64_t>(a.R);
  GrMaps m;
  if (moe_status_t st = map_2d(&m.a, a.w, N, R, 2 * N, 64, 64, kBf16)) return st;
  if (moe_status_t st = map_2d(&m.b, a.x, K, R, 2 * K, 64, 64, kBf16)) return st;
  m.b16 = m.b;
  const int64_t tiles = int64_t(a.E) * ceil_div(a.K, 256) * ceil_div(a.N, 256);
  // Rows in parts where the tiles leave half of the pairs idle, and an expert's rows are
  // kGrPartStages stages of each part at least (by the mean: their offsets are on the
  // device).  49722 x 3856 x 72 to fp32 242 -> 129 us, 8192 x 512 x 1024 41.3 -> 21.2, 4096 x
  // 1024 x 1024 24.7 -> 19.0; the exchange takes 2 us: in parts of 4 stages 1024 x 1024 x 1024
  // would take 12.6 instead of 12.1, 512 x 1024 x 2048 12.3 instead of 10.2.
  int parts = 1;
  for (int c = 2; c <= kGrMaxParts; c *= 2)
    if (tiles * 2 * c <= a.num_sms && a.R >= int64_t(a.E) * c * 64 * kGrPartStages &&
        tiles <= clusters_that_fit<kWeightGrad>(c))
      parts = c;
  if (parts > 1)
    return launch_grouped<kWeightGrad, true>("grouped_weight_grad_split", a, m, tiles, parts, s);
  return launch_grouped<kWeightGrad, false>("grouped_weight_grad", a, m, tiles, 1, s);
}

moe_status_t launch_matmul_fp4(const GroupedProductArgs& a, cudaStream_t s) {
  const uint64_t KB = a.K / 2, N = a.N, E = a.E, R = static_cast<uint64_t>(a.R);
  const int64_t tiles = product_tiles(a, 224);
  const bool rows16 = a.K % 512 == 0;  // rows of scales of whole 16 bytes
  const int units = ceil_div(a.K, 1024);
  const int parts = rows16 ? grouped_parts<kFp4>(a, tiles, units)
                           : grouped_parts<kFp4Rows>(a, tiles, units);
  GrMaps m;
  if (moe_status_t st = map_3d(&m.a, a.w, KB, N, E, KB, 128, 128, kBytes)) return st;
  if (moe_status_t st = map_2d(&m.b16, a.x, KB, R, KB, 128, 16, kBytes)) return st;
  m.b = m.b16;
  if (parts == 1 && a.R > 224 - 32)
    if (moe_status_t st = map_2d(&m.b, a.x, KB, R, KB, 128, 112, kBytes)) return st;
  if (rows16) {
    const uint64_t KG = a.K / 32;
    const auto s32 = CU_TENSOR_MAP_SWIZZLE_32B;
    if (moe_status_t st = map_3d(&m.sa, a.w_scale, KG, N, E, KG, 32, 128, kBytes, s32)) return st;
    if (moe_status_t st = map_2d(&m.sb, a.x_scale, KG, R, KG, 32, 128, kBytes, s32)) return st;
  } else {
    m.sa = m.sb = m.b;
  }
  if (parts > 1)
    return rows16 ? launch_grouped<kFp4, true>("matmul_fp4_split", a, m, tiles, parts, s)
                  : launch_grouped<kFp4Rows, true>("matmul_fp4_split", a, m, tiles, parts, s);
  return rows16 ? launch_grouped<kFp4, false>("matmul_fp4", a, m, tiles, 1, s)
                : launch_grouped<kFp4Rows, false>("matmul_fp4", a, m, tiles, 1, s);
}

}  // namespace gbmoe
