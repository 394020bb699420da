// Dense FP8 products with block scales, and the activations' quantisation
// for them.
//
// "fused_moe.py 分析" (FP8 W8A8, block-wise): within each 128-wide K block
// the FP8 dot product is multiplied by the activation's scale (per row and
// block) and the weight's (per 128 x 128 block), and the blocks are summed:
//   y[m, n] = sum_b sa[m, b] sw[b, n / 128] sum_{k in b} a[m, k] w[k, n]
// The experts' GEMMs of that scheme are in gemm.cu; here the product is one
// matrix's, for the linear layers beside the experts.
#include <algorithm>

#include "common.cuh"
#include "fp8q.cuh"
#include "ptx.cuh"

namespace gbmoe {
namespace {

constexpr int kQgWarps = 8;

// z of 8 columns as fp32: x itself, or SiLU(gate) * up.
__device__ __forceinline__ void qg_unpack(const uint4 u, float (&f)[8]) {
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = __bfloat1622float2(h[i]);
    f[2 * i] = v.x;
    f[2 * i + 1] = v.y;
  }
}

// One half-warp per (row, group of 128 columns), 8 columns per lane.
template <bool SWIGLU>
__global__ void __launch_bounds__(kQgWarps * 32)
    quant_groups_kernel(const bf16* __restrict__ x, int64_t M, int K, uint8_t* __restrict__ q8,
                        float* __restrict__ scale) {
  pdl_begin();
  const int64_t G = (K + 127) / 128;
  const int lane = threadIdx.x & 31;
  const int64_t half0 =
      (static_cast<int64_t>(blockIdx.x) * kQgWarps + (threadIdx.x >> 5)) * 2 + (lane >> 4);
  const int64_t halves = static_cast<int64_t>(gridDim.x) * kQgWarps * 2;
  const int64_t total = M * G;
  for (int64_t base = half0 - (lane >> 4); base < total; base += halves) {
    const int64_t i = base + (lane >> 4);  // (row, group); the warp stays together
    const int64_t row = i / G;
    const int col = static_cast<int>(i - row * G) * 128 + (lane & 15) * 8;
    const bool in = i < total && col < K;
    float f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) f[j] = 0.f;
    if (in) {
      const bf16* src = x + row * K * (SWIGLU ? 2 : 1) + col;
      qg_unpack(*reinterpret_cast<const uint4*>(src), f);
      if constexpr (SWIGLU) {
        float u[8];
        qg_unpack(*reinterpret_cast<const uint4*>(src + K), u);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = f[j] / (1.0f + expf(-f[j])) * u[j];
      }
    }
    // max |z| as an unsigned maximum of the bits: NaN is above every number
    uint32_t mb = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) mb = max(mb, __float_as_uint(f[j]) & 0x7fffffffu);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, o));
    const float s = mb == 0u ? 1.0f : __fdiv_rn(__uint_as_float(mb), 448.0f);
    if (!in) continue;
    uint32_t c[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      c[j >> 2] |= static_cast<uint32_t>(
                       __nv_cvt_float_to_fp8(__fdiv_rn(f[j], s), __NV_SATFINITE, __NV_E4M3))
                   << (8 * (j & 3));
    *reinterpret_cast<uint2*>(q8 + row * K + col) = make_uint2(c[0], c[1]);
    if ((lane & 15) == 0) scale[i] = s;
  }
}

__device__ __forceinline__ float e4m3_f32(uint8_t c) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

struct DenseParams {
  const uint8_t* a;
  const float* a_scale;
  const uint8_t* w;
  const float* w_scale;
  const bf16* bias;
  void* out;
  int64_t M;
  int K, N, transposed, out_f32;
  int32_t* error_word;
};

// 64 x 64 tile, 256 threads, 4 x 4 outputs each.
__global__ void __launch_bounds__(256) dense_fp8_simt_kernel(DenseParams P) {
  pdl_begin();
  __shared__ float sa[16][65], sw[16][65];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t m0 = static_cast<int64_t>(blockIdx.x) * 64;
  const int n0 = static_cast<int>(blockIdx.y) * 64;
  const int KB = ceil_div(P.K, 128), NB = ceil_div(P.N, 128);
  float acc[4][4] = {}, part[4][4] = {};
  for (int k0 = 0; k0 < P.K; k0 += 16) {
    for (int i = threadIdx.x; i < 1024; i += 256) {
      const int r = i >> 4, kk = i & 15;
      const int64_t m = m0 + r;
      sa[kk][r] = m < P.M ? e4m3_f32(P.a[m * P.K + k0 + kk]) : 0.f;
      const int n = P.transposed ? r : i & 63, k = P.transposed ? kk : i >> 6;
      float v = 0.f;
      if (n0 + n < P.N)
        v = e4m3_f32(P.transposed ? P.w[static_cast<int64_t>(n0 + n) * P.K + k0 + k]
                                  : P.w[static_cast<int64_t>(k0 + k) * P.N + n0 + n]);
      sw[k][n] = v;
    }
    __syncthreads();
#pragma unroll
    for (int kk = 0; kk < 16; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          part[i][j] = fmaf(sa[kk][ty * 4 + i], sw[kk][tx * 4 + j], part[i][j]);
    __syncthreads();
    if ((k0 & 127) == 112 || k0 + 16 == P.K) {
      const int b = k0 >> 7, nb = n0 >> 7;
      const float ws = P.transposed ? P.w_scale[nb * KB + b] : P.w_scale[b * NB + nb];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t m = m0 + ty * 4 + i;
        const float as = m < P.M ? P.a_scale[m * KB + b] : 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          acc[i][j] = fmaf(part[i][j], as * ws, acc[i][j]);
          part[i][j] = 0.f;
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t m = m0 + ty * 4 + i;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + tx * 4 + j;
      if (m >= P.M || n >= P.N) continue;
      const float v = acc[i][j] + (P.bias ? __bfloat162float(P.bias[n]) : 0.f);
      if (P.out_f32)
        static_cast<float*>(P.out)[m * P.N + n] = v;
      else
        static_cast<bf16*>(P.out)[m * P.N + n] = __float2bfloat16(v);
    }
  }
}

// ---- large products: CTA pairs, tcgen05 cta_group::2 ----
// Tile 256 x 256 of the output per pair, each CTA holding 128 rows; a stage
// is 128 of K (one scale block): 128 rows of A and half of B's columns per
// CTA.  Each K block is an accumulation of its own in one of two TMEM
// accumulators (256 columns each), scaled and added into registers by eight
// warps (32 rows x 128 columns each) while the other accumulator is filled.
constexpr int kDpThreads = 128 + 256;     // TMA warp, MMA warp (and two idle), 8 promotion warps
// Registers: the launch holds 168 per thread; the first warpgroup returns
// what it does not need and the promotion warps, with 128 sums each, take it
// (128 x 40 + 256 x 224 <= 384 x 168).
constexpr int kDpRegsLaunch = 168, kDpRegsFew = 40, kDpRegsMany = 224;
static_assert(128 * kDpRegsFew + 256 * kDpRegsMany <= kDpThreads * kDpRegsLaunch,
              "register split within the launch's registers");
constexpr int kDpStages = 6;
constexpr int kDpStage = 2 * 16384;       // A 128 x 128 bytes, B 128 x 128 bytes
constexpr size_t kDpSmem = 1024 + kDpStages * kDpStage;
constexpr int kDpGroupM = 8;              // row tiles of a raster group

struct DpCtl {
  uint64_t full[kDpStages], empty[kDpStages];
  uint64_t tmem_full[2], tmem_empty[2];
  uint32_t tmem_base;
  int32_t abort;
};

// Waits for phase `parity` of `bar`; gives up after kWaitLimitNs (error word,
// abort flag) or when another role of the CTA has given up.
__device__ __forceinline__ bool dense_wait(uint64_t* bar, uint32_t parity, int32_t* abort,
                                           int32_t* err) {
  if (ptx::mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = ptx::globaltimer_ns();
  while (true) {
    if (ptx::mbar_try_wait_suspend(bar, parity, 1000000u)) return true;
    if (*reinterpret_cast<volatile int32_t*>(abort)) return false;
    if (ptx::globaltimer_ns() - t0 > kWaitLimitNs) {
      *reinterpret_cast<volatile int32_t*>(abort) = 1;
      record_error(err, MOE_ERR_TIMEOUT);
      return false;
    }
  }
}

// Waits for the warp's TMEM loads, the registers tied to the wait so that
// nothing reads them before it.
__device__ __forceinline__ void tmem_wait32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

// Arrives on an mbarrier of a CTA of the cluster without ordering this
// thread's other memory operations: what the accumulator's next writer has
// to follow are TMEM loads, which the tcgen05 fences order.  The releasing
// form waits for the thread's outstanding memory operations first, ~1000
// cycles in every K block (8192 x 7168 x 4096: 453 us with it, 247 without).
__device__ __forceinline__ void arrive_relaxed(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr)
               : "memory");
}

struct TileMN {
  int m, n;
};
// Tile t in raster groups of kDpGroupM row tiles by all column tiles, rows
// innermost: tiles in flight together share rows of A and columns of B in L2.
__device__ __forceinline__ TileMN dense_tile(int t, int mt, int nt) {
  const int per = kDpGroupM * nt;
  const int g = t / per, r = t - g * per;
  const int rows = min(kDpGroupM, mt - g * kDpGroupM);
  return TileMN{g * kDpGroupM + r % rows, r / rows};
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}

// 16 columns of one output row: bias, rounding, 16-byte stores.
__device__ __forceinline__ void store16(const DenseParams& P, int64_t m, int n, const float* v) {
  float o[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) o[j] = v[j];
  if (P.bias != nullptr) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float b[8];
      qg_unpack(__ldg(reinterpret_cast<const uint4*>(P.bias + n) + h), b);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[8 * h + j] += b[j];
    }
  }
  if (P.out_f32) {
    float4* d = reinterpret_cast<float4*>(static_cast<float*>(P.out) + m * P.N + n);
#pragma unroll
    for (int j = 0; j < 4; ++j) d[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
  } else {
    uint4* d = reinterpret_cast<uint4*>(static_cast<bf16*>(P.out) + m * P.N + n);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      d[j] = make_uint4(pack2(o[8 * j], o[8 * j + 1]), pack2(o[8 * j + 2], o[8 * j + 3]),
                        pack2(o[8 * j + 4], o[8 * j + 5]), pack2(o[8 * j + 6], o[8 * j + 7]));
  }
}

template <bool TR>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kDpThreads, 1)
    dense_fp8_pair_kernel(const __grid_constant__ CUtensorMap tmA,
                          const __grid_constant__ CUtensorMap tmB, const DenseParams P) {
  pdl_begin();
  extern __shared__ uint8_t smem_raw[];
  __shared__ DpCtl ctl;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  uint8_t* tiles = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kDpStages; ++i) {
      ptx::mbar_init(&ctl.full[i], 1);
      ptx::mbar_init(&ctl.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&ctl.tmem_full[i], 1);
      ptx::mbar_init(&ctl.tmem_empty[i], 2 * 8);  // the promotion warps of both CTAs
    }
    ctl.abort = 0;
    ptx::fence_barrier_init();
    ptx::prefetch_tmap(&tmA);
    ptx::prefetch_tmap(&tmB);
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(&ctl.tmem_base, 512);
    ptx::tmem_relinquish_pair();
  }
  ptx::tc_fence_before();
  ptx::cluster_sync();
  ptx::tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;

  const int KB = ceil_div(P.K, 128), NB = ceil_div(P.N, 128);
  const int mt = static_cast<int>(ceil_div<int64_t>(P.M, 256)), nt = ceil_div(P.N, 256);
  const int total = mt * nt;
  const int unit = static_cast<int>(blockIdx.x >> 1), units = static_cast<int>(gridDim.x >> 1);

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kDpRegsFew));
    if (warp == 0 && lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = unit; t < total && ok; t += units) {
        const TileMN tl = dense_tile(t, mt, nt);
        const int row = tl.m * 256 + static_cast<int>(rank) * 128;
        const int col = tl.n * 256 + static_cast<int>(rank) * 128;
        for (int kb = 0; kb < KB; ++kb) {
          if (!dense_wait(&ctl.empty[stage], phase ^ 1u, &ctl.abort, P.error_word)) {
            ok = false;
            break;
          }
          // both CTAs' copies complete on the even CTA's barrier
          const uint32_t full0 = ptx::mapa_shared(ptx::smem_u32(&ctl.full[stage]), 0);
          if (rank == 0) ptx::mbar_arrive_expect_tx(&ctl.full[stage], 2 * kDpStage);
          uint8_t* sa = tiles + stage * kDpStage;
          ptx::tma_load_2d_pair(sa, &tmA, full0, kb * 128, row);
          if constexpr (TR)
            ptx::tma_load_2d_pair(sa + 16384, &tmB, full0, kb * 128, col);
          else
            ptx::tma_load_2d_pair(sa + 16384, &tmB, full0, col, kb * 128);
          if (++stage == kDpStages) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    } else if (warp == 1 && lane == 0 && rank == 0) {
      constexpr uint32_t idesc = ptx::idesc_e4m3_f32(256, 256, false, !TR);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int t = unit; t < total && ok; t += units) {
        for (int kb = 0; kb < KB; ++kb) {
          if (!dense_wait(&ctl.tmem_empty[acc], acc_phase ^ 1u, &ctl.abort, P.error_word) ||
              !dense_wait(&ctl.full[stage], phase, &ctl.abort, P.error_word)) {
            ok = false;
            break;
          }
          ptx::tc_fence_after();
          const uint32_t sa = ptx::smem_u32(tiles + stage * kDpStage), sb = sa + 16384;
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint64_t ad = ptx::smem_desc_sw128(sa + ks * 32, 16, 1024);
            const uint64_t bd = TR ? ptx::smem_desc_sw128(sb + ks * 32, 16, 1024)
                                   : ptx::smem_desc_sw128(sb + ks * 4096, 16384, 1024);
            ptx::mma_e4m3_pair(tmem + acc * 256, ad, bd, idesc, ks != 0);
          }
          ptx::mma_commit_pair(&ctl.empty[stage], 0x3);
          ptx::mma_commit_pair(&ctl.tmem_full[acc], 0x3);
          if (++stage == kDpStages) {
            stage = 0;
            phase ^= 1u;
          }
          if (++acc == 2) {
            acc = 0;
            acc_phase ^= 1u;
          }
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kDpRegsMany));
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(q * 32) << 16) + half * 128;
    const uint32_t empty0 = ptx::mapa_shared(ptx::smem_u32(&ctl.tmem_empty[0]), 0);
    // scales of four K blocks at a time, loaded four blocks ahead (across
    // tiles too): a load in the block that uses it would put an L2 round trip
    // into every block
    auto load4 = [&](int t, int kb0, float (&sa)[4], float (&sw)[4]) {
      const TileMN tl = dense_tile(t, mt, nt);
      const int64_t m = static_cast<int64_t>(tl.m) * 256 + rank * 128 + q * 32 + lane;
      const int nb = min(tl.n * 2 + half, NB - 1);
      const float* pa = P.a_scale + (m < P.M ? m : P.M - 1) * KB;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int kb = min(kb0 + j, KB - 1);
        sa[j] = __ldg(pa + kb);
        sw[j] = __ldg(P.w_scale + (TR ? static_cast<int64_t>(nb) * KB + kb
                                      : static_cast<int64_t>(kb) * NB + nb));
      }
    };
    float na[4], nw[4];
    if (unit < total) load4(unit, 0, na, nw);
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int t = unit; t < total && ok; t += units) {
      float sum[128];
#pragma unroll
      for (int j = 0; j < 128; ++j) sum[j] = 0.f;
      float c[4];
      for (int kb = 0; kb < KB; ++kb) {
        if ((kb & 3) == 0) {
#pragma unroll
          for (int j = 0; j < 4; ++j) c[j] = na[j] * nw[j];
          if (kb + 4 < KB)
            load4(t, kb + 4, na, nw);
          else if (t + units < total)
            load4(t + units, 0, na, nw);
        }
        const float sc = c[0];
        c[0] = c[1];
        c[1] = c[2];
        c[2] = c[3];
        const bool got = dense_wait(&ctl.tmem_full[acc], acc_phase, &ctl.abort, P.error_word);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t ta = lane_addr + acc * 256;
        uint32_t v[2][32];
        ptx::tmem_ld_32cols(ta, v[0]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          tmem_wait32(v[i & 1]);
          if (i < 3) {
            ptx::tmem_ld_32cols(ta + 32 * (i + 1), v[(i + 1) & 1]);
          } else {  // the accumulator is in registers
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_relaxed(empty0 + acc * 8);
          }
#pragma unroll
          for (int j = 0; j < 32; j += 2)
            ptx::fma2(sum[32 * i + j], sum[32 * i + j + 1], __uint_as_float(v[i & 1][j]),
                      __uint_as_float(v[i & 1][j + 1]), sc);
        }
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1u;
        }
      }
      if (!ok) break;
      const TileMN tl = dense_tile(t, mt, nt);
      const int64_t m = static_cast<int64_t>(tl.m) * 256 + rank * 128 + q * 32 + lane;
      const int n0 = tl.n * 256 + half * 128;
      if (m < P.M) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (n0 + 16 * i < P.N) store16(P, m, n0 + 16 * i, sum + 16 * i);
      }
    }
  }
  __syncwarp();
  ptx::cluster_sync();
  if (*reinterpret_cast<volatile int32_t*>(&ctl.abort)) {
    // copies and MMAs in flight get time to land before their memory goes
    const uint64_t t0 = ptx::globaltimer_ns();
    while (ptx::globaltimer_ns() - t0 < 2000000ull) __nanosleep(1000);
  }
  ptx::cluster_sync();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem, 512);
  }
}

// Tensor maps of A [M, K] and of the weight, boxes of 128 x 128 bytes.
moe_status_t dense_maps(const MatmulFp8Args& a, uint32_t a_rows, CUtensorMap* tmA,
                        CUtensorMap* tmB) {
  const uint64_t K = a.K, N = a.N;
  const uint64_t da[2] = {K, static_cast<uint64_t>(a.M)}, sa[1] = {K};
  const uint32_t ba[2] = {128, a_rows}, bb[2] = {128, 128};
  if (moe_status_t st = encode_tensor_map(tmA, a.a, 2, da, sa, ba, CU_TENSOR_MAP_DATA_TYPE_UINT8,
                                          CU_TENSOR_MAP_SWIZZLE_128B))
    return st;
  const uint64_t db[2] = {a.transposed ? K : N, a.transposed ? N : K}, sb[1] = {db[0]};
  return encode_tensor_map(tmB, a.w, 2, db, sb, bb, CU_TENSOR_MAP_DATA_TYPE_UINT8,
                           CU_TENSOR_MAP_SWIZZLE_128B);
}

template <bool TR>
moe_status_t launch_pair(const MatmulFp8Args& a, const DenseParams& P, cudaStream_t s) {
  static PerDevice attr;
  int regs = 0;
  if (attr.get(
          [](int* v) {
            cudaFuncAttributes fa;
            const cudaError_t e = cudaFuncGetAttributes(&fa, dense_fp8_pair_kernel<TR>);
            if (e != cudaSuccess) return e;
            *v = fa.numRegs;
            return cudaFuncSetAttribute(dense_fp8_pair_kernel<TR>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(kDpSmem));
          },
          &regs) != cudaSuccess)
    return set_error(MOE_ERR_CUDA, "attributes of matmul_fp8: %s",
                     cudaGetErrorString(cudaGetLastError()));
  // fewer registers at launch would leave the promotion warps waiting for more
  if (regs < kDpRegsLaunch)
    return set_error(MOE_ERR_CUDA, "matmul_fp8 was compiled to %d registers, %d needed", regs,
                     kDpRegsLaunch);
  CUtensorMap tmA, tmB;
  if (moe_status_t st = dense_maps(a, 128, &tmA, &tmB)) return st;
  const int64_t tiles = ceil_div<int64_t>(a.M, 256) * ceil_div(a.N, 256);
  const unsigned grid = 2u * static_cast<unsigned>(std::min<int64_t>(tiles, a.num_sms / 2));
  prof_before("matmul_fp8", s);
  launch_kernel(dense_fp8_pair_kernel<TR>, grid, kDpThreads, kDpSmem, s, tmA, tmB, P);
  prof_after("matmul_fp8", s);
  return check_launch("matmul_fp8");
}

}  // namespace

moe_status_t launch_quant_groups_fp8(const QuantGroupsArgs& a, cudaStream_t s) {
  const int64_t warps = ceil_div<int64_t>(a.M * ceil_div(a.K, 128), 2);
  const unsigned grid =
      static_cast<unsigned>(std::min<int64_t>(ceil_div<int64_t>(warps, kQgWarps), 152 * 64));
  prof_before("quant_groups_fp8", s);
  launch_kernel(a.swiglu ? quant_groups_kernel<true> : quant_groups_kernel<false>, grid,
                kQgWarps * 32, 0, s, a.x, a.M, a.K, a.q8, a.scale);
  prof_after("quant_groups_fp8", s);
  return check_launch("quant_groups_fp8");
}

moe_status_t launch_matmul_fp8(const MatmulFp8Args& a, cudaStream_t s) {
  const DenseParams P{a.a, a.a_scale, a.w, a.w_scale, a.bias, a.out, a.M, a.K, a.N, a.transposed,
                      a.out_f32, a.error_word};
  if (a.M > 128) return a.transposed ? launch_pair<true>(a, P, s) : launch_pair<false>(a, P, s);
  const dim3 grid(static_cast<unsigned>(ceil_div<int64_t>(a.M, 64)),
                  static_cast<unsigned>(ceil_div(a.N, 64)));
  prof_before("matmul_fp8", s);
  launch_kernel(dense_fp8_simt_kernel, grid, 256, 0, s, P);
  prof_after("matmul_fp8", s);
  return check_launch("matmul_fp8");
}

}  // namespace gbmoe
