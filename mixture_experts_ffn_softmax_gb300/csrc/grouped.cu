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
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "dense.cuh"
#include "ptx.cuh"

namespace gbmoe {
namespace {

enum Mode { kProduct, kProductT, kWeightGrad, kFp4 };  // W [E, K, N], [E, N, K]; FP4: [E, N, K]

constexpr int kGrThreads = 128 + 256;  // TMA, MMA, two helper warps; 8 output warps
constexpr int kGrMaxExperts = 1024;
constexpr int kGrGroup = 8;            // row tiles of a raster group
constexpr int kGrStaging = 2048;       // an output warp's: 16 rows by 32 columns of fp32
constexpr int kScaleChunks = 3;        // FP4: chunks of 512 elements whose scales are on their way
constexpr int kGrRelay = 16;           // bytes by which the odd CTA signals the even one
// Registers: as in the dense FP8 pairs, the first warpgroup gives up what the output
// warps, with up to 128 sums each, need.
constexpr int kGrRegsLaunch = 168, kGrRegsFew = 88, kGrRegsMany = 208;
static_assert(128 * kGrRegsFew + 256 * kGrRegsMany <= kGrThreads * kGrRegsLaunch,
              "register split within the launch's registers");

template <int MODE>
struct GrGeo {
  static constexpr bool FP4 = MODE == kFp4, WG = MODE == kWeightGrad;
  static constexpr bool A_MN = MODE == kProduct || WG;  // MN-major first operand
  static constexpr int BK = FP4 ? 256 : 64;    // reduced elements of a stage (128 bytes of a row)
  // columns of a tile; FP4: two accumulators and the scales share the 512 TMEM columns
  static constexpr int TM = FP4 ? 224 : 256;
  static constexpr int SCALES = FP4 ? 3072 : 0;  // of a stage: 128 + 256 rows by 8 bytes
  static constexpr int STAGE = 32768 + SCALES;
  static constexpr int STAGES = FP4 ? 5 : 6;
  static constexpr size_t SMEM =
      1024 + STAGES * STAGE + 8 * kGrStaging + (FP4 ? kScaleChunks * 6144 : 0);
};
constexpr uint32_t kScaleCol = 448;  // TMEM columns of FP4's scales, 24 for each of two stages

template <int MODE>
struct GrCtl {
  static constexpr int S = GrGeo<MODE>::STAGES;
  uint64_t full[S], empty[S];
  uint64_t tail[S];               // weight grad: the expert's last rows; FP4: the odd CTA's scales
  uint64_t tmem_full[2], tmem_empty[2];
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
static_assert(GrGeo<kFp4>::SMEM + sizeof(GrCtl<kFp4>) <= 232448, "shared memory budget");

struct GrParams {
  const int32_t* offsets;  // [E + 1], or null: all R rows are expert 0's
  int64_t R;
  int E, K, N;             // weight grad: K rows of dW
  const bf16* bias;        // [E, N] or null
  const uint8_t* x_scale;  // FP4: [R, K / 32], [E, N, K / 32]
  const uint8_t* w_scale;
  void* out;
  int out_f32, accumulate;
  int chunk;               // stages summed in the tensor core before they go to registers
  int32_t* error_word;
};

struct GrTile {
  int e, n0;        // expert, first column of the weight
  int64_t c0;       // first row of y, or of dW[e]
  int cols, T;      // how many, and rounded up to what the MMA takes
  int r0, rows;     // the expert's rows
};

template <int MODE>
__device__ __forceinline__ GrTile gr_tile(const GrCtl<MODE>& ctl, const GrParams& P, int t) {
  using G = GrGeo<MODE>;
  const int nt = ceil_div(P.N, 256);
  GrTile tl;
  int r, ct;  // tile within the expert, column tiles (of y's rows or dW's)
  if constexpr (G::WG) {
    ct = ceil_div(P.K, G::TM);
    tl.e = t / (ct * nt);
    r = t - tl.e * (ct * nt);
  } else {
    int lo = 0, hi = P.E;  // the last expert whose first tile is not behind t
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (ctl.tile0[mid] <= t) lo = mid;
      else hi = mid;
    }
    tl.e = lo;
    r = t - ctl.tile0[lo];
    ct = ceil_div(ctl.count[lo], G::TM);
  }
  tl.r0 = ctl.start[tl.e];
  tl.rows = ctl.count[tl.e];
  // raster groups of kGrGroup column tiles by all weight tiles, columns innermost: tiles in
  // flight together share the weight's columns and the rows in L2
  const int per = kGrGroup * nt;
  const int g = r / per, q = r - g * per;
  const int in_group = min(kGrGroup, ct - g * kGrGroup);
  const int c = (g * kGrGroup + q % in_group) * G::TM;
  tl.n0 = q / in_group * 256;
  tl.cols = min(G::TM, (G::WG ? P.K : tl.rows) - c);
  tl.c0 = G::WG ? c : static_cast<int64_t>(tl.r0) + c;
  // (MN-major columns come in swizzled chunks of 64 per CTA)
  tl.T = G::WG ? (tl.cols > 128 ? 256 : 128) : (tl.cols + 31) & ~31;
  return tl;
}

template <int MODE>
__device__ __forceinline__ int gr_blocks(const GrParams& P, const GrTile& tl) {
  return ceil_div(GrGeo<MODE>::WG ? tl.rows : P.K, GrGeo<MODE>::BK);
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

template <int MODE>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGrThreads, 1)
    grouped_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmB16, const GrParams P) {
  using G = GrGeo<MODE>;
  pdl_begin();
  extern __shared__ uint8_t smem_raw[];
  __shared__ GrCtl<MODE> ctl;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(ptx::cluster_ctarank());
  uint8_t* tiles = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  // the odd CTA's word that stage's part of it is in place
  auto relay = [&](int stage) {
    ptx::bulk_copy_to_cluster(ptx::mapa_shared(ptx::smem_u32(ctl.relay[stage]), 0), ctl.relay_src,
                              kGrRelay, ptx::mapa_shared(ptx::smem_u32(&ctl.full[stage]), 0));
  };
  if (threadIdx.x == 0) {
    for (int i = 0; i < G::STAGES; ++i) {
      // full: the loads of both CTAs (one arrival); weight grad: one more, for the even CTA's
      // tail; FP4: two more, for its scale warps
      ptx::mbar_init(&ctl.full[i], G::WG ? 2 : G::FP4 ? 3 : 1);
      ptx::mbar_init(&ctl.empty[i], 1);
      ptx::mbar_init(&ctl.tail[i], G::FP4 ? 2 : 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&ctl.tmem_full[i], 1);
      ptx::mbar_init(&ctl.tmem_empty[i], 2 * 8);  // the output warps of both CTAs
    }
    ctl.abort = 0;
    ctl.blocks = 0;
    ptx::fence_barrier_init();
    ptx::prefetch_tmap(&tmA);
    ptx::prefetch_tmap(&tmB);
    ptx::prefetch_tmap(&tmB16);
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(&ctl.tmem_base, 512);
    ptx::tmem_relinquish_pair();
  }
  const int nt = ceil_div(P.N, 256);
  if (warp == 2) {
    // the experts' rows, clipped to the R there are, and their tiles
    int total = 0;
    for (int e0 = 0; e0 < P.E; e0 += 32) {
      const int e = e0 + lane;
      int n = 0;
      if (e < P.E) {
        int64_t b = 0, c = P.R;
        if (P.offsets != nullptr) {
          const int64_t b0 = __ldg(P.offsets + e), c0 = __ldg(P.offsets + e + 1);
          b = min(max(b0, int64_t(0)), P.R);
          c = min(max(c0, b), P.R);
          if (b != b0 || c != c0) record_error(P.error_word, MOE_ERR_INVALID_ARG);
        }
        ctl.start[e] = static_cast<int32_t>(b);
        ctl.count[e] = static_cast<int32_t>(c - b);
        n = ceil_div(static_cast<int>(c - b), G::TM) * nt;
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
  const uint32_t tmem = ctl.tmem_base;
  const int total = ctl.total;
  const int unit = static_cast<int>(blockIdx.x >> 1), units = static_cast<int>(gridDim.x >> 1);

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kGrRegsFew));
    // (The loading and the issuing warp run their loops as one, an elected lane issuing: in a
    // branch of one lane an MMA took 70 cycles to issue, the loop 730 for the 512 that a stage
    // of 256 columns computes.  8 x 1024 rows, K 4096, N 28672: 1193 us so, 1077 as here;
    // the weight gradient of 128 x 1024 rows, 2048 x 1536: 726 and 597.  A wait that ran out
    // does not end a loop: once it has, all others end at once, and the loop runs out.)
    if (warp == 0) {
      // ---- loads ----
      const uint32_t go = ptx::elect_one();
      const uint32_t tiles0 = ptx::smem_u32(tiles);
      int stage = 0;
      uint32_t phase = 0;
      int64_t blocks = 0;
      for (int t = unit; t < total; t += units) {
        const GrTile tl = gr_tile(ctl, P, t);
        const int KB = gr_blocks<MODE>(P, tl);
        const int half = tl.T / 2;
        const int n = tl.n0 + rank * 128, c = static_cast<int>(tl.c0) + rank * half;
        const uint32_t bytes = 16384u + static_cast<uint32_t>(half) * 128u;
        for (int kb = 0; kb < KB; ++kb) {
          dense_wait(&ctl.empty[stage], phase ^ 1u, &ctl.abort, P.error_word);
          const uint32_t sa = tiles0 + stage * G::STAGE, sb = sa + 16384;
          // both CTAs' copies complete on the even CTA's barrier
          uint32_t bar = ptx::mapa_shared(ptx::smem_u32(&ctl.full[stage]), 0);
          if (G::WG && kb == KB - 1 && tl.rows % 16 != 0) {
            // the last rows of the expert: to this CTA's tail barrier, and on from there
            bar = ptx::mapa_shared(ptx::smem_u32(&ctl.tail[stage]), rank);
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
              ptx::tma_load_2d_pair_if(go, sa + i * 8192, &tmA, bar, n + i * 64, r);
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (i < half / 64)
                ptx::tma_load_2d_pair_if(go, sb + i * 8192, &tmB, bar, c + i * 64, r);
          } else {
            const int k = kb * (G::FP4 ? 128 : 64);  // bytes, or elements
            if constexpr (MODE == kProduct) {
#pragma unroll
              for (int i = 0; i < 2; ++i)
                ptx::tma_load_3d_pair_if(go, sa + i * 8192, &tmA, bar, n + i * 64, k, tl.e);
            } else {
              ptx::tma_load_3d_pair_if(go, sa, &tmA, bar, k, n, tl.e);
            }
            if (tl.T == G::TM) {
              ptx::tma_load_2d_pair_if(go, sb, &tmB, bar, k, c);
            } else {
              for (int i = 0; i < half; i += 16)
                ptx::tma_load_2d_pair_if(go, sb + i * 128, &tmB16, bar, k, c + i);
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
      const uint32_t tiles0 = ptx::smem_u32(tiles);
      constexpr uint32_t HI = 64u | 1u << 14 | 2u << 29;  // (8-row groups 1024 bytes apart)
      // K-major: 32 bytes of a row per step; MN-major: 16 rows, chunks of 64 columns 8192 apart
      constexpr uint32_t A_STEP = G::A_MN ? 128 : 2, B_STEP = G::WG ? 128 : 2;
      constexpr uint32_t A_LO = (G::A_MN ? 512u : 1u) << 16, B_LO = (G::WG ? 512u : 1u) << 16;
      int stage = 0;
      uint32_t phase = 0, acc = 0, turn = 0, block = 0;
      for (int t = unit; t < total; t += units) {
        const GrTile tl = gr_tile(ctl, P, t);
        const int KB = gr_blocks<MODE>(P, tl);
        const uint32_t idesc = ptx::idesc_bf16_f32(256, tl.T, G::A_MN, G::WG);
        int in_chunk = 0;
        for (int kb = 0; kb < KB; ++kb, ++block) {
          if (in_chunk == 0)
            dense_wait(&ctl.tmem_empty[acc], turn ^ 1u, &ctl.abort, P.error_word);
          dense_wait(&ctl.full[stage], phase, &ctl.abort, P.error_word);
          ptx::tc_fence_after();
          const uint32_t sa = tiles0 + stage * G::STAGE;
          const uint32_t a = (sa >> 4) + A_LO, b = ((sa + 16384) >> 4) + B_LO;
          const uint32_t d = tmem + acc * static_cast<uint32_t>(G::TM);
          if constexpr (G::FP4) {
            const uint32_t sc = tmem + kScaleCol + (block & 1u) * 24u, ss = sa + 32768;
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
            // weight grad: the last block's MMAs end with the expert's rows
            const int steps = G::WG && kb == KB - 1 ? ceil_div(tl.rows - kb * 64, 16) : 4;
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
              if (ks < steps)
                ptx::mma_bf16_pair_if(go, d, a + ks * A_STEP, b + ks * B_STEP, HI, idesc,
                                      (in_chunk | ks) != 0);
          }
          const bool last = ++in_chunk == P.chunk || kb == KB - 1;
          if (last) ptx::mma_commit_pair_if(go, &ctl.tmem_full[acc], 0x3);
          ptx::mma_commit_pair_if(go, &ctl.empty[stage], 0x3);
          if (last) {
            in_chunk = 0;
            acc ^= 1u;
            turn ^= acc == 0 ? 1u : 0u;
          }
          if (++stage == G::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    } else if (G::FP4 && warp == 1 && lane == 0) {
      // ---- odd CTA: a stage's scales are in place ----
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = unit; t < total && ok; t += units) {
        const int KB = gr_blocks<MODE>(P, gr_tile(ctl, P, t));
        for (int kb = 0; kb < KB; ++kb) {
          if (!dense_wait(&ctl.tail[stage], phase, &ctl.abort, P.error_word)) {
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
        const int KB = gr_blocks<MODE>(P, tl);
        block += KB;
        if (tl.rows % 16 == 0) continue;
        const int stage = static_cast<int>((block - 1) % G::STAGES);
        const bool got =
            dense_wait(&ctl.tail[stage], parity >> stage & 1u, &ctl.abort, P.error_word);
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
    } else if (G::FP4 && warp >= 2) {
      // ---- scales: each lane two of the weight's 128 rows and four of the tile's 256, 16
      // bytes (512 elements, two stages) of each at a time ----
      // They come by asynchronous copies into a ring of the lane's own, kScaleChunks ahead and
      // across tiles (held in registers one chunk ahead, their latency was in every
      // chunk: 8192 x 7168 x 4096 155 us, 119 with the ring), and go from there to where
      // the tensor core's copy takes them.
      const int w = warp - 2;
      const int KG = P.K / 32;
      uint8_t* ring = tiles + G::STAGES * G::STAGE + 8 * kGrStaging + (w * 32 + lane) * 16;
      constexpr int ROW = 64 * 16, CHUNK = 6 * ROW;  // a row of both warps' lanes, six of them
      int ft = unit, fg = 0, fslot = 0;  // what is fetched next: tile, scale of K, slot
      const uint8_t* src[6];             // its rows; null: no such row
      auto rows = [&]() {
        const GrTile tl = gr_tile(ctl, P, ft);
#pragma unroll
        for (int i = 0; i < 6; ++i) {
          if (i < 2) {
            const int n = tl.n0 + rank * 128 + (w * 2 + i) * 32 + lane;
            src[i] = n < P.N ? P.w_scale + (static_cast<int64_t>(tl.e) * P.N + n) * KG : nullptr;
          } else {
            const int c = (w * 4 + i - 2) * 32 + lane;
            src[i] = c < tl.T && tl.c0 + c < P.R ? P.x_scale + (tl.c0 + c) * KG : nullptr;
          }
        }
      };
      // (zeros for rows that are not there and past K, where the codes are zeros: 2^-127)
      auto fetch = [&]() {
        if (ft < total) {
          uint8_t* dst = ring + fslot * CHUNK;
#pragma unroll
          for (int i = 0; i < 6; ++i) {
            const uint8_t* from = src[i] != nullptr ? src[i] + fg : P.w_scale;
            if (KG % 16 == 0) {
              ptx::cp_async_16(dst + i * ROW, from, src[i] != nullptr ? 16 : 0);
            } else if (KG % 4 == 0) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const bool in = src[i] != nullptr && fg + 4 * j < KG;
                ptx::cp_async_4(dst + i * ROW + 4 * j, in ? from + 4 * j : P.w_scale, in ? 4 : 0);
              }
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t v = 0;
                for (int q = 0; q < 4; ++q)
                  if (src[i] != nullptr && fg + 4 * j + q < KG)
                    v |= static_cast<uint32_t>(__ldg(from + 4 * j + q)) << (8 * q);
                *reinterpret_cast<uint32_t*>(dst + i * ROW + 4 * j) = v;
              }
            }
          }
          fslot = fslot + 1 == kScaleChunks ? 0 : fslot + 1;
          fg += 16;
          if (fg >= KG) {
            fg = 0;
            ft += units;
            if (ft < total) rows();
          }
        }
        ptx::cp_async_commit();  // (of nothing, at the end: the count of groups stays)
      };
      if (ft < total) rows();
#pragma unroll
      for (int i = 0; i < kScaleChunks; ++i) fetch();
      int stage = 0, slot = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = unit; t < total && ok; t += units) {
        const int KB = ceil_div(P.K, G::BK);
        for (int kb = 0; kb < KB && ok; kb += 2) {
          uint4 v[6];
          ptx::cp_async_wait<kScaleChunks - 1>();
#pragma unroll
          for (int i = 0; i < 6; ++i)
            v[i] = *reinterpret_cast<const uint4*>(ring + slot * CHUNK + i * ROW);
          slot = slot + 1 == kScaleChunks ? 0 : slot + 1;
          fetch();
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (kb + h >= KB) break;
            const bool got = dense_wait(&ctl.empty[stage], phase ^ 1u, &ctl.abort, P.error_word);
            if (!__all_sync(0xffffffffu, got)) {
              ok = false;
              break;
            }
            uint8_t* sc = tiles + stage * G::STAGE + 32768 + lane * 16;
#pragma unroll
            for (int i = 0; i < 6; ++i) {
              uint8_t* at = i < 2 ? sc + (w * 2 + i) * 4 : sc + 1024 + w * 512 + (i - 2) * 4;
              const int next = i < 2 ? 512 : 1024;  // the second 128 elements of the stage
              *reinterpret_cast<uint32_t*>(at) = h == 0 ? v[i].x : v[i].z;
              *reinterpret_cast<uint32_t*>(at + next) = h == 0 ? v[i].y : v[i].w;
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(rank == 0 ? &ctl.full[stage] : &ctl.tail[stage]);
            if (++stage == G::STAGES) {
              stage = 0;
              phase ^= 1u;
            }
          }
        }
      }
      ptx::cp_async_wait<0>();
    }
  } else {
    // ---- output: 32 columns n of the weight (lanes) by half of the tile's columns a warp ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kGrRegsMany));
    const int q = warp & 3, part = (warp - 4) >> 2;
    const uint32_t empty0 = ptx::mapa_shared(ptx::smem_u32(&ctl.tmem_empty[0]), 0);
    uint8_t* staging = tiles + G::STAGES * G::STAGE + (warp - 4) * kGrStaging;
    uint32_t acc = 0, turn = 0;
    bool ok = true;
    for (int t = unit; t < total && ok; t += units) {
      const GrTile tl = gr_tile(ctl, P, t);
      const int KB = gr_blocks<MODE>(P, tl);
      const int n = tl.n0 + rank * 128 + q * 32 + lane;
      const int groups = tl.T / 32;  // of 16 columns
      const float b = P.bias != nullptr && n < P.N
                          ? __bfloat162float(P.bias[static_cast<int64_t>(tl.e) * P.N + n])
                          : 0.f;
      uint64_t sum[64];
#pragma unroll
      for (int j = 0; j < 64; ++j) sum[j] = pair_of(b, b);
      for (int kb = 0; kb < KB; kb += P.chunk) {
        const bool got = dense_wait(&ctl.tmem_full[acc], turn, &ctl.abort, P.error_word);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t ta = tmem + (static_cast<uint32_t>(q * 32) << 16) +
                            acc * static_cast<uint32_t>(G::TM) + part * groups * 16;
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
      if (!ok) break;
      // 16 rows by the warp's 32 columns at a time through its staging block and out in
      // 16-byte stores (each lane storing its own column's elements, one warp's store 64 or
      // 128 bytes, took 60 of 1210 us at 8 x 1024 rows, K 4096, N 28672, and 170 of 880 us
      // in the weight gradient of 8 x 1024 rows, 14336 x 4096)
      const int first = part * groups * 16;
      const int64_t row0 = (G::WG ? static_cast<int64_t>(tl.e) * P.K : 0) + tl.c0 + first;
      const int left = min(tl.cols - first, groups * 16);
      const int nw = tl.n0 + rank * 128 + q * 32;  // the warp's first column
      auto put = [&](auto* out) {
        using O = std::remove_pointer_t<decltype(out)>;
        constexpr bool F32 = sizeof(O) == 4;
        constexpr int PER = 16 / sizeof(O);        // elements of a store
        constexpr int LANES = 32 / PER;            // lanes of a row
        constexpr int STEP = 32 / LANES;           // rows of a store
        const int ln = lane % LANES * PER, lr = lane / LANES;
        O* dst = out + (row0 + lr) * P.N + nw + ln;
        const uint32_t sel = lane & 1 ? 0x3276u : 0x5410u;
#pragma unroll
        for (int i = 0; i < G::TM / 32; ++i) {
          if (16 * i >= left) break;
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            float2 o = unpair(sum[8 * i + j / 2]);
            if (!F32 && G::WG && P.accumulate && nw + lane < P.N) {  // (added before it is rounded)
              const O* old = out + (row0 + 16 * i + j) * P.N + nw + lane;
              if (16 * i + j < left) o.x += static_cast<float>(old[0]);
              if (16 * i + j + 1 < left) o.y += static_cast<float>(old[P.N]);
            }
            if constexpr (F32) {
              *reinterpret_cast<float*>(staging + j * 128 + lane * 4) = o.x;
              *reinterpret_cast<float*>(staging + j * 128 + 128 + lane * 4) = o.y;
            } else {
              // row j of two columns in even lanes, row j + 1 of them in odd ones
              const uint32_t mine = pack2(o.x, o.y), other = __shfl_xor_sync(0xffffffffu, mine, 1);
              *reinterpret_cast<uint32_t*>(staging + (j + (lane & 1)) * 64 + (lane & ~1) * 2) =
                  __byte_perm(mine, other, sel);
            }
          }
          __syncwarp();
          if (nw + ln < P.N) {  // (N is a multiple of 8)
#pragma unroll
            for (int r = 0; r < 16; r += STEP) {
              if (16 * i + r + lr < left) {
                uint4 v = *reinterpret_cast<const uint4*>(staging + r * 32 * sizeof(O) + lane * 16);
                uint4* at = reinterpret_cast<uint4*>(dst + static_cast<int64_t>(16 * i + r) * P.N);
                if (F32 && G::WG && P.accumulate) {
                  const uint4 old = *at;
                  v.x = __float_as_uint(__uint_as_float(v.x) + __uint_as_float(old.x));
                  v.y = __float_as_uint(__uint_as_float(v.y) + __uint_as_float(old.y));
                  v.z = __float_as_uint(__uint_as_float(v.z) + __uint_as_float(old.z));
                  v.w = __float_as_uint(__uint_as_float(v.w) + __uint_as_float(old.w));
                }
                *at = v;
              }
            }
          }
        }
      };
      if (P.out_f32)
        put(static_cast<float*>(P.out));
      else
        put(static_cast<bf16*>(P.out));
    }
  }
  __syncwarp();
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
// too small, in proportion to K), so that sums that leave in fp32 go to registers, where they
// are rounded to nearest, every 512 rows or columns (FP4: 2048; an MMA is four times as
// deep).  Sums that leave in bf16 lose 4e-3 in their own rounding, and go there once.
int gr_chunk(const GroupedProductArgs& a) { return a.out_f32 ? 8 : 1 << 30; }

template <int MODE>
moe_status_t launch_grouped(const char* name, const GroupedProductArgs& a, const CUtensorMap& tmA,
                            const CUtensorMap& tmB, const CUtensorMap& tmB16, int64_t tiles,
                            cudaStream_t s) {
  using G = GrGeo<MODE>;
  static PerDevice attr;
  int regs = 0;
  if (attr.get(
          [](int* v) {
            cudaFuncAttributes fa;
            const cudaError_t e = cudaFuncGetAttributes(&fa, grouped_kernel<MODE>);
            if (e != cudaSuccess) return e;
            *v = fa.numRegs;
            return cudaFuncSetAttribute(grouped_kernel<MODE>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(G::SMEM));
          },
          &regs) != cudaSuccess)
    return set_error(MOE_ERR_CUDA, "attributes of %s: %s", name,
                     cudaGetErrorString(cudaGetLastError()));
  // fewer registers at launch would leave the output warps waiting for more
  if (regs < kGrRegsLaunch)
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
  P.chunk = gr_chunk(a);
  P.error_word = a.error_word;
  const unsigned grid = 2u * static_cast<unsigned>(std::min<int64_t>(tiles, a.num_sms / 2));
  prof_before(name, s);
  launch_kernel(grouped_kernel<MODE>, grid, kGrThreads, G::SMEM, s, tmA, tmB, tmB16, P);
  prof_after(name, s);
  return check_launch(name);
}

// At most how many tiles a product has: an expert with rows has one more than whole ones.
int64_t product_tiles(const GroupedProductArgs& a, int TM) {
  return ceil_div(a.N, 256) * (a.R / TM + std::min<int64_t>(a.E, a.R));
}

moe_status_t map_2d(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t pitch,
                    uint32_t box_cols, uint32_t box_rows, CUtensorMapDataType type) {
  const uint64_t d[2] = {cols, rows}, st[1] = {pitch};
  const uint32_t box[2] = {box_cols, box_rows};
  return encode_tensor_map(m, base, 2, d, st, box, type, CU_TENSOR_MAP_SWIZZLE_128B);
}
moe_status_t map_3d(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint64_t mats,
                    uint64_t pitch, uint32_t box_cols, uint32_t box_rows,
                    CUtensorMapDataType type) {
  const uint64_t d[3] = {cols, rows, mats}, st[2] = {pitch, pitch * rows};
  const uint32_t box[3] = {box_cols, box_rows, 1};
  return encode_tensor_map(m, base, 3, d, st, box, type, CU_TENSOR_MAP_SWIZZLE_128B);
}

constexpr auto kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
constexpr auto kBytes = CU_TENSOR_MAP_DATA_TYPE_UINT8;

}  // namespace

moe_status_t launch_grouped_matmul(const GroupedProductArgs& a, cudaStream_t s) {
  const uint64_t K = a.K, N = a.N, E = a.E, R = static_cast<uint64_t>(a.R);
  CUtensorMap tmA, tmB, tmB16;
  if (moe_status_t st = a.transposed ? map_3d(&tmA, a.w, K, N, E, 2 * K, 64, 128, kBf16)
                                     : map_3d(&tmA, a.w, N, K, E, 2 * N, 64, 64, kBf16))
    return st;
  if (moe_status_t st = map_2d(&tmB, a.x, K, R, 2 * K, 64, 128, kBf16)) return st;
  if (moe_status_t st = map_2d(&tmB16, a.x, K, R, 2 * K, 64, 16, kBf16)) return st;
  const int64_t tiles = product_tiles(a, 256);
  return a.transposed
             ? launch_grouped<kProductT>("grouped_matmul_t", a, tmA, tmB, tmB16, tiles, s)
             : launch_grouped<kProduct>("grouped_matmul", a, tmA, tmB, tmB16, tiles, s);
}

moe_status_t launch_grouped_weight_grad(const GroupedProductArgs& a, cudaStream_t s) {
  const uint64_t K = a.K, N = a.N, R = static_cast<uint64_t>(a.R);
  CUtensorMap tmA, tmB;
  if (moe_status_t st = map_2d(&tmA, a.w, N, R, 2 * N, 64, 64, kBf16)) return st;
  if (moe_status_t st = map_2d(&tmB, a.x, K, R, 2 * K, 64, 64, kBf16)) return st;
  const int64_t tiles = int64_t(a.E) * ceil_div(a.K, 256) * ceil_div(a.N, 256);
  return launch_grouped<kWeightGrad>("grouped_weight_grad", a, tmA, tmB, tmB, tiles, s);
}

moe_status_t launch_matmul_fp4(const GroupedProductArgs& a, cudaStream_t s) {
  const uint64_t KB = a.K / 2, N = a.N, E = a.E, R = static_cast<uint64_t>(a.R);
  CUtensorMap tmA, tmB, tmB16;
  if (moe_status_t st = map_3d(&tmA, a.w, KB, N, E, KB, 128, 128, kBytes)) return st;
  if (moe_status_t st = map_2d(&tmB, a.x, KB, R, KB, 128, 112, kBytes)) return st;
  if (moe_status_t st = map_2d(&tmB16, a.x, KB, R, KB, 128, 16, kBytes)) return st;
  return launch_grouped<kFp4>("matmul_fp4", a, tmA, tmB, tmB16, product_tiles(a, 224), s);
}

}  // namespace gbmoe
