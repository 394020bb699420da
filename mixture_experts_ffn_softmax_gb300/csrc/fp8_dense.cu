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
#include <type_traits>

#include "common.cuh"
#include "fp8q.cuh"
#include "ptx.cuh"

namespace gbmoe {
namespace {

// ---- quantisation ----
constexpr int kQgWarps = 8, kQgBlocks = 3;  // warps of a block, blocks of an SM

// Pairs of fp32 in one register pair, and operations on both at once (each
// rounded as the plain one): half the issue slots, which bound these kernels.
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
// div_fixed (fp8q.cuh) of a pair: x / s from r = 1 / s, ns = -s.
__device__ __forceinline__ uint64_t div_fixed2(uint64_t x, uint64_t ns, uint64_t r) {
  const uint64_t q = mul2(x, r);
  return fma2(fma2(q, ns, x), r, q);
}
// max(a, |b|), NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(fabsf(b)));
  return r;
}

__device__ __forceinline__ void unpack8(const uint4 u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// SiLU(g) * u of eight columns.  With h = fp32(g log2 e) and the small
// t = g - h ln 2 (ln 2 in two parts, so that t is what h's rounding left of g),
//   e^-g = 2^-h (1 - t),
// all but 2^-h on packed pairs (expf for each: 19.0 us at 8191 x 2048, this 17.2).
// The quotient g / (1 + e^-g) by the reciprocal (within an ulp) and one correction
// (div_fixed: the remainder is exact, one rounding); for gates outside the range in
// which that holds, by the division.
// This gives up a little precision for that time.  In 2^-24: 2^-h 2.45 (the largest
// of every fp32 argument below 116; ex2.approx states 4), 1 - t, the sum and the
// quotient 1 each, 5.5 in all; over every bf16 gate below 80 SiLU is off by at most
// 3.18 and 0.173 in the mean, where expf and the division are by 2.63 and 0.167.
constexpr float kLog2E = 1.44269504f, kLn2Hi = 0.693147182f, kLn2Lo = -1.90465430e-9f;
__device__ __forceinline__ void swiglu8(float (&g)[8], const float (&u)[8]) {
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(g[j]));
  if (top < 80.f) {
    const uint64_t minus1 = pair_of(-1.0f, -1.0f);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const uint64_t x = pair_of(g[j], g[j + 1]);
      const uint64_t h = mul2(x, pair_of(kLog2E, kLog2E));
      const uint64_t t = fma2(h, pair_of(-kLn2Lo, -kLn2Lo), fma2(h, pair_of(-kLn2Hi, -kLn2Hi), x));
      const float2 h1 = unpair(h);
      float p[2], r[2];
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p[0]) : "f"(-h1.x));
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p[1]) : "f"(-h1.y));
      const uint64_t nden = fma2(pair_of(p[0], p[1]), add2(t, minus1), minus1);  // -(1 + e^-g)
      const float2 d = unpair(nden);
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r[0]) : "f"(-d.x));
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r[1]) : "f"(-d.y));
      const float2 z =
          unpair(mul2(div_fixed2(x, nden, pair_of(r[0], r[1])), pair_of(u[j], u[j + 1])));
      g[j] = z.x;
      g[j + 1] = z.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = g[j] / (1.0f + expf(-g[j])) * u[j];
  }
}

// E4M3 codes of eight values, each fp32(z / s) rounded to nearest even; r = 1 / s
// where fast (no remainder of the correction underflows).
__device__ __forceinline__ uint2 e4m3_codes8(const float (&z)[8], float s, float r, bool fast) {
  uint32_t c[4];
  if (fast) {
    const uint64_t ns = pair_of(-s, -s), r2 = pair_of(r, r);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c[j] = __nv_cvt_float2_to_fp8x2(unpair(div_fixed2(pair_of(z[2 * j], z[2 * j + 1]), ns, r2)),
                                      __NV_SATFINITE, __NV_E4M3);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c[j] = __nv_cvt_float2_to_fp8x2(
          make_float2(__fdiv_rn(z[2 * j], s), __fdiv_rn(z[2 * j + 1], s)), __NV_SATFINITE,
          __NV_E4M3);
  }
  return make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
}

// A half-warp per (row, group of 128 columns), 8 columns per lane.  A warp
// takes U passes of 256 columns of a row at a time, the next ones' loads in
// flight while it works on them (resident blocks only, three per SM: 8192 x 7168 in
// 30.0 us, 31.0 without the loads ahead, 32.8 in blocks of one row segment after
// another).  Bound: HBM (3 bytes per element of x, 5.9 TB/s of 6.8 measured), and
// for SiLU(gate) * up, 5 per element of z, issue slots (8191 x 2048: 17.2 us).
template <bool SWIGLU>
__global__ void __launch_bounds__(kQgWarps * 32, kQgBlocks)
    quant_groups_kernel(const bf16* __restrict__ x, int64_t M, int K, uint8_t* __restrict__ q8,
                        float* __restrict__ scale) {
  pdl_begin();
  constexpr int U = SWIGLU ? 2 : 4;
  const int lane = threadIdx.x & 31;
  const int64_t G = ceil_div(K, 128);
  const int segs = ceil_div(K, 256 * U);
  const int64_t warps = static_cast<int64_t>(gridDim.x) * kQgWarps;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kQgWarps + (threadIdx.x >> 5);
  // (row, segment) stepped without a division in the loop
  int64_t row = first / segs;
  int seg = static_cast<int>(first - row * segs);
  const int64_t step_row = warps / segs;
  const int step_seg = static_cast<int>(warps - step_row * segs);
  uint4 a[U], b[SWIGLU ? U : 1];
  auto load = [&]() {  // of (row, seg); zeros past K and M
    const int col0 = seg * (256 * U) + lane * 8;
    const bf16* src = x + row * K * (SWIGLU ? 2 : 1) + col0;
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const bool in = row < M && col0 + 256 * i < K;
      a[i] = in ? __ldg(reinterpret_cast<const uint4*>(src + 256 * i)) : make_uint4(0, 0, 0, 0);
      if constexpr (SWIGLU)
        b[i] = in ? __ldg(reinterpret_cast<const uint4*>(src + K + 256 * i))
                  : make_uint4(0, 0, 0, 0);
    }
  };
  load();
  while (row < M) {
    const int col0 = seg * (256 * U) + lane * 8;
    uint4 ca[U], cb[SWIGLU ? U : 1];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      ca[i] = a[i];
      if constexpr (SWIGLU) cb[i] = b[i];
    }
    uint8_t* dst = q8 + row * K + col0;
    float* sc = scale + row * G + col0 / 128;
    row += step_row;
    seg += step_seg;
    if (seg >= segs) {
      seg -= segs;
      ++row;
    }
    load();  // the next unit's, while this one is worked on
#pragma unroll
    for (int i = 0; i < U; ++i) {
      float z[8];
      unpack8(ca[i], z);
      float m = 0.f;  // max |z|, or NaN
      if constexpr (SWIGLU) {
        float u[8];
        unpack8(cb[i], u);
        swiglu8(z, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max_nan(m, z[j]);
      } else {
        // as bf16 pairs: the bits without the sign order as the values, NaN on top
        uint32_t t = __vmaxu2(ca[i].x & 0x7fff7fffu, ca[i].y & 0x7fff7fffu);
        t = __vmaxu2(t, ca[i].z & 0x7fff7fffu);
        t = __vmaxu2(t, ca[i].w & 0x7fff7fffu);
        m = __uint_as_float(max(t << 16, t & 0xffff0000u));
      }
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
      const bool fast = m >= 1e-27f && m <= 1e30f;
      float s, r = 0.f;
      if (fast) {
        s = div_fixed(m, 448.0f, 1.0f / 448.0f);
        r = __frcp_rn(s);
      } else {
        // (0 also where z, held in fp32, is below 448 times half of fp32's smallest number)
        s = __fdiv_rn(m, 448.0f);
        if (s == 0.f) s = 1.0f;
      }
      if (col0 + 256 * i < K) {
        *reinterpret_cast<uint2*>(dst + 256 * i) = e4m3_codes8(z, s, r, fast);
        if ((lane & 15) == 0) sc[2 * i] = s;
      }
    }
  }
}

struct DenseParams {
  const float* a_scale;
  const float* w_scale;
  const bf16* bias;
  void* out;
  int64_t M;
  int K, N, out_f32;
  int32_t* error_word;
};

// ---- shared by both products ----
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
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[32]) {
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

// c += (a0, a1) * b on a pair of sums kept packed, so that no pair is taken apart
// and put together again in every block.
__device__ __forceinline__ void fma_pair(uint64_t& c, uint32_t a0, uint32_t a1, uint64_t b) {
  asm("{\n\t.reg .b64 a;\n\tmov.b64 a, {%1, %2};\n\tfma.rn.f32x2 %0, a, %3, %0;\n\t}"
      : "+l"(c)
      : "r"(a0), "r"(a1), "l"(b));
}

// ---- many rows: CTA pairs ----
// Tile of 256 rows by NT = 256 or 128 columns on a CTA pair (tcgen05
// cta_group::2), each CTA holding 128 rows.  A stage is 128 of K, one scale block:
// 128 rows of A and NT / 2 columns of the weight per CTA.  Each K block is an
// accumulation of its own in one of 512 / NT TMEM accumulators, scaled and added
// into registers by eight warps (32 rows x NT / 2 columns each) while the others
// are filled.  A K block of 256 columns takes 830 cycles (512 of MMA; the hand-off
// without the sums 700, loads and MMAs alone 590), one of 128 columns 590: the narrow
// tile is for products whose wide tiles would leave many pairs idle (512 x 7168 x 4096:
// 28.3 us in 32 wide tiles, 21.2 in 64 narrow ones; 8192 x 7168 x 4096: 172 and 237).
constexpr int kDpThreads = 128 + 256;  // TMA, 2 MMA, scale warp; 8 promotion warps
// Registers: the launch holds 168 per thread; for wide tiles the first warpgroup
// returns what it does not need and the promotion warps, with 128 sums each, take it.
constexpr int kDpRegsLaunch = 168, kDpRegsFew = 72, kDpRegsMany = 208;
static_assert(128 * kDpRegsFew + 256 * kDpRegsMany <= kDpThreads * kDpRegsLaunch,
              "register split within the launch's registers");
constexpr int kDpStaging = 8 * 4096;   // per promotion warp 32 rows x 128 bytes of output
constexpr int kDpGroupM = 8;           // row tiles of a raster group
template <int NT>  // columns of a tile
struct DpGeo {
  static constexpr int STAGES = NT == 256 ? 5 : 7;
  static constexpr int STAGE = 16384 + NT / 2 * 128;  // A 128 x 128 bytes, weight 128 x NT / 2
  static constexpr int ACCS = 512 / NT;               // TMEM accumulators
  static constexpr int SCALES = 2 * ACCS;             // scale slots (K blocks)
  static constexpr int AHEAD = NT == 256 ? 2 : 4;     // K blocks whose scales are loaded together
  static constexpr size_t SMEM = 1024 + STAGES * STAGE + kDpStaging;
};

template <int NT>
struct DpCtl {
  using G = DpGeo<NT>;
  uint64_t full[G::STAGES], empty[G::STAGES];
  uint64_t tmem_full[G::ACCS], tmem_empty[G::ACCS];
  float a_scale[G::SCALES][128], w_scale[G::SCALES][2];  // rows, column blocks of a K block
  uint32_t tmem_base;
  int32_t abort;
};
static_assert(DpGeo<256>::SMEM + sizeof(DpCtl<256>) <= 232448 &&
                  DpGeo<128>::SMEM + sizeof(DpCtl<128>) <= 232448,
              "shared memory budget");

// The two halves of a cluster barrier; this arrival orders nothing (a releasing
// one waits for the thread's loads in flight).
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
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

// One 128-byte row piece of the output (64 bf16 or 32 fp32 columns) into row
// `lane` of a 128-byte-swizzled staging block.
template <bool F32>
__device__ __forceinline__ void stage_row(uint8_t* buf, int lane, const uint64_t* v) {
  // (opaque: the eight addresses would otherwise be kept in registers all
  // through the promotion loop)
  asm volatile("" : "+r"(lane));
#pragma unroll
  for (int j = 0; j < 8; ++j) {  // 16-byte units
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 4); ++i) {
      const float2 o = unpair(v[(F32 ? 2 : 4) * j + i]);
      if constexpr (F32) {
        u[2 * i] = __float_as_uint(o.x);
        u[2 * i + 1] = __float_as_uint(o.y);
      } else {
        u[i] = pack2(o.x, o.y);
      }
    }
    *reinterpret_cast<uint4*>(buf + lane * 128 + ((j ^ (lane & 7)) << 4)) =
        make_uint4(u[0], u[1], u[2], u[3]);
  }
}

// As smem_desc_sw128 with the 64-byte swizzle (mode 4): MN-major rows of 64 bytes.
__device__ __forceinline__ uint64_t smem_desc_sw64(uint32_t saddr, uint32_t lbo, uint32_t sbo) {
  return (ptx::smem_desc_sw128(saddr, lbo, sbo) & ~(uint64_t(7) << 61)) | uint64_t(4) << 61;
}

template <bool TR, int NT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kDpThreads, 1)
    dense_fp8_pair_kernel(const __grid_constant__ CUtensorMap tmA,
                          const __grid_constant__ CUtensorMap tmB,
                          const __grid_constant__ CUtensorMap tmO, const DenseParams P) {
  using G = DpGeo<NT>;
  pdl_begin();
  extern __shared__ uint8_t smem_raw[];
  __shared__ DpCtl<NT> ctl;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = ptx::cluster_ctarank();
  uint8_t* tiles = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  uint8_t* staging = tiles + G::STAGES * G::STAGE;
  if (threadIdx.x == 0) {
    for (int i = 0; i < G::STAGES; ++i) {
      ptx::mbar_init(&ctl.full[i], 1);
      ptx::mbar_init(&ctl.empty[i], 1);
    }
    for (int i = 0; i < G::ACCS; ++i) {
      ptx::mbar_init(&ctl.tmem_full[i], 2);        // the MMA's commit, the scale warp
      ptx::mbar_init(&ctl.tmem_empty[i], 2 * 8);   // the promotion warps of both CTAs
    }
    ctl.abort = 0;
    ptx::fence_barrier_init();
    ptx::prefetch_tmap(&tmA);
    ptx::prefetch_tmap(&tmB);
    ptx::prefetch_tmap(&tmO);
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
  const int mt = static_cast<int>(ceil_div<int64_t>(P.M, 256)), nt = ceil_div(P.N, NT);
  const int total = mt * nt;
  const int unit = static_cast<int>(blockIdx.x >> 1), units = static_cast<int>(gridDim.x >> 1);
  const int64_t blocks =  // K blocks of this pair
      unit < total ? static_cast<int64_t>((total - 1 - unit) / units + 1) * KB : 0;

  if (warp < 4) {
    if constexpr (NT == 256) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kDpRegsFew));
    if (warp == 0 && lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int t = unit; t < total && ok; t += units) {
        const TileMN tl = dense_tile(t, mt, nt);
        const int row = tl.m * 256 + static_cast<int>(rank) * 128;
        const int col = tl.n * NT + static_cast<int>(rank) * (NT / 2);
        for (int kb = 0; kb < KB; ++kb) {
          if (!dense_wait(&ctl.empty[stage], phase ^ 1u, &ctl.abort, P.error_word)) {
            ok = false;
            break;
          }
          uint8_t* sa = tiles + stage * G::STAGE;
          uint8_t* sb = sa + 16384;
          // both CTAs' copies complete on the even CTA's barrier
          const uint32_t full0 = ptx::mapa_shared(ptx::smem_u32(&ctl.full[stage]), 0);
          if (rank == 0) ptx::mbar_arrive_expect_tx(&ctl.full[stage], 2 * G::STAGE);
          ptx::tma_load_2d_pair(sa, &tmA, full0, kb * 128, row);
          ptx::tma_load_2d_pair(sb, &tmB, full0, TR ? kb * 128 : col, TR ? col : kb * 128);
          if (++stage == G::STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
      }
    } else if (warp <= 2) {
      // two issuing threads, of every second block: while one is held up by the
      // MMAs queued ahead of its own, the other's waits and commits go on
      // (8192 x 7168 x 4096, before later steps: 194 us with one thread, 180 with two)
      if (lane == 0 && rank == 0) {
        uint32_t acc = warp - 1;
        constexpr uint32_t idesc = ptx::idesc_e4m3_f32(256, NT, false, !TR);
        int stage = acc;  // blocks warp - 1, warp + 1, ...
        uint32_t phase = 0, turn = 0;
        for (int64_t g = acc; g < blocks; g += 2) {
          if (!dense_wait(&ctl.full[stage], phase, &ctl.abort, P.error_word) ||
              !dense_wait(&ctl.tmem_empty[acc], turn ^ 1u, &ctl.abort, P.error_word))
            break;
          ptx::tc_fence_after();
          const uint32_t sa = ptx::smem_u32(tiles + stage * G::STAGE), sb = sa + 16384;
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            const uint64_t ad = ptx::smem_desc_sw128(sa + ks * 32, 16, 1024);
            const uint64_t bd = TR ? ptx::smem_desc_sw128(sb + ks * 32, 16, 1024)
                                   : NT == 256
                                         ? ptx::smem_desc_sw128(sb + ks * 4096, 16384, 1024)
                                         : smem_desc_sw64(sb + ks * 2048, 8192, 512);
            ptx::mma_e4m3_pair(tmem + acc * NT, ad, bd, idesc, ks != 0);
          }
          // (the accumulator's barrier first: the other order took a K-rows
          // weight from 182 to 206 us at 8192 x 7168 x 4096, before later steps)
          ptx::mma_commit_pair(&ctl.tmem_full[acc], 0x3);
          ptx::mma_commit_pair(&ctl.empty[stage], 0x3);
          stage += 2;
          if (stage >= G::STAGES) {
            stage -= G::STAGES;
            phase ^= 1u;
          }
          acc += 2;
          if (acc >= G::ACCS) {
            acc -= G::ACCS;
            turn ^= 1u;
          }
        }
      }
    } else {
      // scales of the promotion warps' next blocks: four rows per lane, of A K
      // blocks at a time and loaded A blocks ahead (across tiles too; narrow tiles with
      // two ahead: 25.0 us for 512 x 7168 x 4096, 21.5 with four, for which the wide
      // tiles' kernel has no registers).  In the promotion warps, short of registers
      // to hold them, these loads' latency came into every group of blocks.
      constexpr int A = G::AHEAD;
      float nx[4][A], nw[A];  // (w: lanes 0 and 1, one column block each)
      auto load = [&](int t, int kb0) {
        const TileMN tl = dense_tile(t, mt, nt);
        const int64_t m = static_cast<int64_t>(tl.m) * 256 + rank * 128 + lane;
        const int nb = min(NT == 256 ? tl.n * 2 + (lane & 1) : tl.n, NB - 1);
        const float* pw = P.w_scale + (TR ? static_cast<int64_t>(nb) * KB : nb);
#pragma unroll
        for (int j = 0; j < A; ++j) {
          const int kb = min(kb0 + j, KB - 1);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            nx[r][j] = __ldg(P.a_scale + min(m + 32 * r, P.M - 1) * KB + kb);
          nw[j] = __ldg(pw + (TR ? kb : static_cast<int64_t>(kb) * NB));
        }
      };
      if (unit < total) load(unit, 0);
      uint32_t g = 0;  // K blocks so far
      bool ok = true;
      for (int t = unit; t < total && ok; t += units) {
        for (int kb = 0; kb < KB && ok; kb += A) {
          float c[4][A], cw[A];
#pragma unroll
          for (int j = 0; j < A; ++j) {
#pragma unroll
            for (int r = 0; r < 4; ++r) c[r][j] = nx[r][j];
            cw[j] = nw[j];
          }
          if (kb + A < KB)
            load(t, kb + A);
          else if (t + units < total)
            load(t + units, 0);
#pragma unroll
          for (int j = 0; j < A; ++j) {
            if (kb + j >= KB) break;
            // block g - ACCS complete means that block g - 2 ACCS, whose slot this
            // is, has left the accumulators and the slot: the MMA of g - ACCS waited
            // for its release
            bool got = true;
            const int acc = g % G::ACCS;
            if (g >= G::ACCS)
              got = dense_wait(&ctl.tmem_full[acc], (g / G::ACCS & 1) ^ 1u, &ctl.abort,
                               P.error_word);
            if (!__all_sync(0xffffffffu, got)) {
              ok = false;
              break;
            }
            const int slot = g % G::SCALES;
#pragma unroll
            for (int r = 0; r < 4; ++r) ctl.a_scale[slot][lane + 32 * r] = c[r][j];
            if (lane < 2) ctl.w_scale[slot][lane] = cw[j];
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(&ctl.tmem_full[acc]);
            ++g;
          }
        }
      }
    }
  } else {
    if constexpr (NT == 256) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kDpRegsMany));
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(q * 32) << 16) + half * (NT / 2);
    const uint32_t empty0 = ptx::mapa_shared(ptx::smem_u32(&ctl.tmem_empty[0]), 0);
    uint8_t* buf = staging + (warp - 4) * 4096;
    uint32_t g = 0;  // K blocks so far
    bool ok = true;
    for (int t = unit; t < total && ok; t += units) {
      uint64_t sum[NT / 4];  // NT / 2 columns
      const int n0 = dense_tile(t, mt, nt).n * NT + half * (NT / 2);
      if (P.bias != nullptr) {
#pragma unroll
        for (int j = 0; j < NT / 2; j += 8) {  // (N is a multiple of 16)
          float b[8] = {};
          if (n0 + j < P.N) unpack8(__ldg(reinterpret_cast<const uint4*>(P.bias + n0 + j)), b);
#pragma unroll
          for (int i = 0; i < 8; i += 2) sum[(j + i) / 2] = pair_of(b[i], b[i + 1]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < NT / 4; ++j) sum[j] = 0;
      }
      // (two blocks of the loop's body at a time, so that a block's last sums run
      // under the next one's wait: 172-175 us at 8192 x 7168 x 4096, 182 without, 180
      // with four)
#pragma unroll 2
      for (int kb = 0; kb < KB; ++kb, ++g) {
        const uint32_t acc = g % G::ACCS;
        const bool got =
            dense_wait(&ctl.tmem_full[acc], g / G::ACCS & 1, &ctl.abort, P.error_word);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        ptx::tc_fence_after();
        const uint32_t ta = lane_addr + acc * NT;
        uint32_t v[2][16];
        ptx::tmem_ld_16cols(ta, v[0]);
        const int slot = g % G::SCALES;
        const float f = ctl.a_scale[slot][q * 32 + lane] * ctl.w_scale[slot][NT == 256 ? half : 0];
        const uint64_t sc = pair_of(f, f);
#pragma unroll
        for (int i = 0; i < NT / 32; ++i) {
          tmem_wait(v[i & 1]);
          if (i < NT / 32 - 1) {
            ptx::tmem_ld_16cols(ta + 16 * (i + 1), v[(i + 1) & 1]);
          } else {  // the accumulator is in registers
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) arrive_relaxed(empty0 + acc * 8);
          }
#pragma unroll
          for (int j = 0; j < 16; j += 2)
            fma_pair(sum[8 * i + j / 2], v[i & 1][j], v[i & 1][j + 1], sc);
        }
      }
      if (!ok) break;
      // the tile's rows through the warp's staging block, 128 bytes of each
      // at a time, and out by TMA (which clips what lies past M and N): lanes
      // storing their own rows would take a sector per lane and store, 6000
      // cycles per tile
      const int m = dense_tile(t, mt, nt).m * 256 + static_cast<int>(rank) * 128 + q * 32;
      auto put = [&](auto f32) {
        constexpr bool F32 = decltype(f32)::value;
        constexpr int W = F32 ? 32 : 64;
#pragma unroll
        for (int i = 0; i < NT / 2 / W; ++i) {
          const int n = n0 + i * W;
          if (n < P.N && m < P.M) {
            if (lane == 0) ptx::bulk_wait_read0();
            __syncwarp();
            stage_row<F32>(buf, lane, sum + i * W / 2);
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              ptx::tma_store_2d(&tmO, buf, n, m);
              ptx::bulk_commit();
            }
          }
        }
      };
      if (P.out_f32)
        put(std::true_type{});
      else
        put(std::false_type{});
    }
    if (lane == 0) ptx::bulk_wait0();
  }
  __syncwarp();
  ptx::cluster_sync();
  // the commits of the last use of every stage, which nothing else waits for, have
  // to arrive before the barriers' memory goes: each of them (commits of one thread
  // complete in order, but nothing says that their arrivals do)
  if (threadIdx.x < G::STAGES && blocks > static_cast<int>(threadIdx.x)) {
    const int64_t g = blocks - 1 - threadIdx.x;
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


// ---- few rows: the weight's columns as the MMA's rows, K split over a cluster ----
// The weight's bytes bound these products, so that every SM has to stream
// them: a CTA takes 128 weight columns (the MMA's M) and one of S parts of K
// for T rows of A (the MMA's N).  TMEM lane = weight column, TMEM column = row of
// A, so a thread's sums are one output column for T rows.  The S CTAs of a
// cluster each own every S-th group of four rows: they store their sums into
// the owners' shared memory (reading the others' instead was a chain of remote
// loads, 8 of 17 us at 77 x 2048 x 7168), and the owner adds the S parts in order.
constexpr int kDsThreads = 64 + 128;   // TMA warp, MMA warp, 4 promotion warps
constexpr int kDsScaleBlocks = 16;     // K blocks whose scales are held at a time
template <int T>
struct DsGeo {
  static constexpr int STAGE = 16384 + T * 128;
  static constexpr int STAGES = T <= 32 ? 8 : T == 64 ? 7 : T == 96 ? 5 : 4;
  static constexpr int ACCS = T >= 96 ? 4 : 8;  // TMEM accumulators of T columns
  static constexpr int COLS = T == 96 ? 512 : ACCS * T;  // (allocated: a power of two)
  // sums of S parts for the T / 4 row groups (up to 7 more slots than groups: the
  // groups of an owner are rounded up)
  static constexpr int PARTS = (T / 4 + 8) * 128 * 16;
  static constexpr size_t SMEM = 1024 + STAGES * STAGE + PARTS;
};
template <int T>
struct DsCtl {
  uint64_t full[DsGeo<T>::STAGES], empty[DsGeo<T>::STAGES];
  uint64_t tmem_full[DsGeo<T>::ACCS], tmem_empty[DsGeo<T>::ACCS];
  uint64_t scale_free, scale_ready;
  // row scale times the block's weight scale (padded: stored a column at a time)
  alignas(16) float scale[kDsScaleBlocks][T + 4];
  uint32_t tmem_base;
  int32_t abort;
};
static_assert(DsGeo<16>::SMEM + sizeof(DsCtl<16>) <= 232448 &&
                  DsGeo<32>::SMEM + sizeof(DsCtl<32>) <= 232448 &&
                  DsGeo<64>::SMEM + sizeof(DsCtl<64>) <= 232448 &&
                  DsGeo<96>::SMEM + sizeof(DsCtl<96>) <= 232448 &&
                  DsGeo<128>::SMEM + sizeof(DsCtl<128>) <= 232448,
              "shared memory budget");

__device__ __forceinline__ void st_cluster_f32x4(uint32_t addr, float a, float b, float c, float d) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b),
               "f"(c), "f"(d)
               : "memory");
}

template <int T, bool TR>
__global__ void __launch_bounds__(kDsThreads, 1)
    dense_fp8_split_kernel(const __grid_constant__ CUtensorMap tmA,
                           const __grid_constant__ CUtensorMap tmB, const DenseParams P,
                           const int S) {
  using G = DsGeo<T>;
  pdl_begin();
  extern __shared__ uint8_t smem_raw[];
  __shared__ DsCtl<T> ctl;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(ptx::cluster_ctarank());  // the part of K
  uint8_t* tiles = smem_raw + ((1024u - (ptx::smem_u32(smem_raw) & 1023u)) & 1023u);
  float4* parts = reinterpret_cast<float4*>(tiles + G::STAGES * G::STAGE);
  const int groups = ceil_div(T / 4, S);  // row groups of an owner; parts [S][groups][128]
  const int KB = ceil_div(P.K, 128), NB = ceil_div(P.N, 128);
  const int nb = static_cast<int>(blockIdx.x) / S;
  const int64_t m0 = static_cast<int64_t>(blockIdx.y) * T;
  const int kb0 = static_cast<int>(static_cast<int64_t>(KB) * rank / S);
  const int kb1 = static_cast<int>(static_cast<int64_t>(KB) * (rank + 1) / S);
  // Scales of the next kDsScaleBlocks blocks, from block kb on: thread p of the
  // promotion warps takes block p % 16 of rows p / 16, p / 16 + 8, ... (a warp's
  // load is two rows' 64 bytes); the first ones are loaded ahead of everything
  // else (they were 2000 cycles of latency between the first MMA and its
  // promotion).  Rows past M count as 0.
  static_assert(kDsScaleBlocks == 16, "one block per thread");
  const int p = static_cast<int>(threadIdx.x) - 64;
  const int sb = p & 15, sr = p >> 4;
  auto load_scale = [&](int kb, int j) {  // (the block's for j < 0)
    const int64_t m = m0 + sr + 8 * j;
    if (sb >= kb1 - kb || m >= P.M) return 0.f;
    if (j < 0)
      return __ldg(P.w_scale + (TR ? static_cast<int64_t>(nb) * KB + kb + sb
                                   : static_cast<int64_t>(kb + sb) * NB + nb));
    return __ldg(P.a_scale + m * KB + kb + sb);
  };
  float ra[T / 8], rw = 0.f;
  if (warp >= 2) {
    rw = load_scale(kb0, -1);
#pragma unroll
    for (int j = 0; j < T / 8; ++j) ra[j] = load_scale(kb0, j);
  }
  if (threadIdx.x == 0) {
    for (int i = 0; i < G::STAGES; ++i) {
      ptx::mbar_init(&ctl.full[i], 1);
      ptx::mbar_init(&ctl.empty[i], 1);
    }
    for (int i = 0; i < G::ACCS; ++i) {
      ptx::mbar_init(&ctl.tmem_full[i], 1);
      ptx::mbar_init(&ctl.tmem_empty[i], 4);
    }
    ptx::mbar_init(&ctl.scale_free, 4);
    ptx::mbar_init(&ctl.scale_ready, 4);
    ctl.abort = 0;
    ptx::fence_barrier_init();
    ptx::prefetch_tmap(&tmA);
    ptx::prefetch_tmap(&tmB);
  }
  if (warp == 1) {
    ptx::tmem_alloc(&ctl.tmem_base, G::COLS);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  cluster_arrive_relaxed();  // (waited for ahead of the stores to the others' memory)
  ptx::tc_fence_after();
  const uint32_t tmem = ctl.tmem_base;

  bool ok = true;
  if (warp == 0) {
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!dense_wait(&ctl.empty[stage], phase ^ 1u, &ctl.abort, P.error_word)) break;
        uint8_t* sw = tiles + stage * G::STAGE;
        ptx::mbar_arrive_expect_tx(&ctl.full[stage], G::STAGE);
        ptx::tma_load_2d(sw, &tmB, &ctl.full[stage], TR ? kb * 128 : nb * 128,
                         TR ? nb * 128 : kb * 128);
        ptx::tma_load_2d(sw + 16384, &tmA, &ctl.full[stage], kb * 128, static_cast<int>(m0));
        if (++stage == G::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
      // the last stages' commits, which no load waits for, have to arrive
      // before the barriers' memory goes
      for (int i = max(0, kb1 - kb0 - G::STAGES); i < kb1 - kb0; ++i)
        if (!dense_wait(&ctl.empty[i % G::STAGES], static_cast<uint32_t>(i / G::STAGES) & 1u,
                        &ctl.abort, P.error_word))
          break;
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = ptx::idesc_e4m3_f32(128, T, !TR, false);
      int stage = 0, acc = 0;
      uint32_t phase = 0, turn = 0;
      for (int kb = kb0; kb < kb1; ++kb) {
        if (!dense_wait(&ctl.tmem_empty[acc], turn ^ 1u, &ctl.abort, P.error_word) ||
            !dense_wait(&ctl.full[stage], phase, &ctl.abort, P.error_word))
          break;
        ptx::tc_fence_after();
        const uint32_t sw = ptx::smem_u32(tiles + stage * G::STAGE), sx = sw + 16384;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
          const uint64_t wd = TR ? ptx::smem_desc_sw128(sw + ks * 32, 16, 1024)
                                 : ptx::smem_desc_sw128(sw + ks * 4096, 16384, 1024);
          ptx::mma_e4m3(tmem + acc * T, wd, ptx::smem_desc_sw128(sx + ks * 32, 16, 1024), idesc,
                        ks != 0);
        }
        ptx::mma_commit(&ctl.empty[stage]);
        ptx::mma_commit(&ctl.tmem_full[acc]);
        if (++stage == G::STAGES) {
          stage = 0;
          phase ^= 1u;
        }
        if (++acc == G::ACCS) {
          acc = 0;
          turn ^= 1u;
        }
      }
    }
  } else {
    const int q = warp & 3;
    const int col = q * 32 + lane;       // weight column of the tile
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>(q * 32) << 16);
    uint64_t sum[T / 2];
#pragma unroll
    for (int j = 0; j < T / 2; ++j) sum[j] = 0;
    // all four promotion warps meet (a bounded wait, unlike a named barrier)
    auto meet = [&](uint64_t* bar, uint32_t parity) {
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar);
      const bool got = dense_wait(bar, parity, &ctl.abort, P.error_word);
      return __all_sync(0xffffffffu, got) != 0;
    };
    int acc = 0;
    uint32_t turn = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      const int slot = (kb - kb0) % kDsScaleBlocks;
      if (slot == 0) {
        // the next blocks' scales, by all four warps; rows past M count as 0
        const uint32_t chunk = static_cast<uint32_t>(kb - kb0) / kDsScaleBlocks;
        if (chunk > 0 && !meet(&ctl.scale_free, (chunk - 1) & 1)) {
          ok = false;
          break;
        }
        if (chunk == 0) {
#pragma unroll
          for (int j = 0; j < T / 8; ++j) ctl.scale[sb][sr + 8 * j] = ra[j] * rw;
        } else {
          const float w = load_scale(kb, -1);
#pragma unroll 4
          for (int j = 0; j < T / 8; ++j) ctl.scale[sb][sr + 8 * j] = load_scale(kb, j) * w;
        }
        if (!meet(&ctl.scale_ready, chunk & 1)) {
          ok = false;
          break;
        }
      }
      const bool got = dense_wait(&ctl.tmem_full[acc], turn, &ctl.abort, P.error_word);
      if (!__all_sync(0xffffffffu, got)) {
        ok = false;
        break;
      }
      ptx::tc_fence_after();
      const ulonglong2* sc = reinterpret_cast<const ulonglong2*>(ctl.scale[slot]);
      constexpr int W = T < 32 ? T : 32;  // columns per TMEM load
#pragma unroll
      for (int c = 0; c < T; c += W) {
        uint32_t v[W];
        if constexpr (W == 32) ptx::tmem_ld_32cols(lane_addr + acc * T + c, v);
        else ptx::tmem_ld_16cols(lane_addr + acc * T + c, v);
        tmem_wait(v);
        if (c + W == T) {  // the accumulator is in registers
          ptx::tc_fence_before();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&ctl.tmem_empty[acc]);
        }
#pragma unroll
        for (int j = 0; j < W; j += 4) {
          const ulonglong2 s4 = sc[(c + j) / 4];
          fma_pair(sum[(c + j) / 2], v[j], v[j + 1], s4.x);
          fma_pair(sum[(c + j) / 2 + 1], v[j + 2], v[j + 3], s4.y);
        }
      }
      if (++acc == G::ACCS) {
        acc = 0;
        turn ^= 1u;
      }
    }
    __syncwarp();
    cluster_wait();
    if (ok) {
      uint32_t slot = ptx::smem_u32(parts + rank * groups * 128 + col);
      int owner = 0;
#pragma unroll
      for (int g = 0; g < T / 4; ++g) {
        const float2 a = unpair(sum[2 * g]), b = unpair(sum[2 * g + 1]);
        st_cluster_f32x4(ptx::mapa_shared(slot, owner), a.x, a.y, b.x, b.y);
        if (++owner == S) {
          owner = 0;
          slot += 128 * 16;
        }
      }
    }
  }
  __syncwarp();
  if (warp < 2) cluster_wait();
  ptx::cluster_sync();
  if (warp >= 2) {
    const int col = (warp & 3) * 32 + lane;
    const int n = nb * 128 + col;
    const float b = P.bias != nullptr && n < P.N ? __bfloat162float(P.bias[n]) : 0.f;
    const int rows = static_cast<int>(min(static_cast<int64_t>(T), P.M - m0));
    auto put = [&](auto* out) {
      using O = std::remove_pointer_t<decltype(out)>;
      const int64_t ld = P.N;
      out += (m0 + 4 * rank) * ld + n;
      const float4* mine = parts + col;
      auto add = [&](int i) {
        float4 v = make_float4(b, b, b, b);
#pragma unroll 4
        for (int s = 0; s < S; ++s) {
          const float4 o = mine[(s * groups + i) * 128];
          v.x += o.x;
          v.y += o.y;
          v.z += o.z;
          v.w += o.w;
        }
        return v;
      };
      // whole groups of this owner, then the one the rows end in
      const int whole = rows / 4 > rank ? (rows / 4 - rank - 1) / S + 1 : 0;
#pragma unroll 4
      for (int i = 0; i < whole; ++i) {
        const float4 v = add(i);
        O* d = out + i * (4 * S) * ld;
        d[0] = static_cast<O>(v.x);
        d[ld] = static_cast<O>(v.y);
        d[2 * ld] = static_cast<O>(v.z);
        d[3 * ld] = static_cast<O>(v.w);
      }
      if (rows % 4 != 0 && rows / 4 % S == rank) {
        const float4 v = add(rows / 4 / S);
        O* d = out + rows / 4 / S * (4 * S) * ld;
        d[0] = static_cast<O>(v.x);
        if (rows % 4 > 1) d[ld] = static_cast<O>(v.y);
        if (rows % 4 > 2) d[2 * ld] = static_cast<O>(v.z);
      }
    };
    if (n < P.N) {
      if (P.out_f32)
        put(static_cast<float*>(P.out));
      else
        put(static_cast<bf16*>(P.out));
    }
  }
  if (*reinterpret_cast<volatile int32_t*>(&ctl.abort)) {
    // copies and MMAs in flight get time to land before their memory goes
    const uint64_t t0 = ptx::globaltimer_ns();
    while (ptx::globaltimer_ns() - t0 < 2000000ull) __nanosleep(1000);
  }
  __syncthreads();
  if (warp == 1) {
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem, G::COLS);
  }
}

// Tensor maps of A [M, K], in boxes of a_rows x 128 bytes, and of the weight,
// in boxes of 128 x 128 bytes.
moe_status_t dense_maps(const MatmulFp8Args& a, uint32_t a_rows, uint32_t w_cols, CUtensorMap* tmA,
                        CUtensorMap* tmB) {
  const uint64_t K = a.K, N = a.N;
  const uint64_t da[2] = {K, static_cast<uint64_t>(a.M)}, sa[1] = {K};
  const uint32_t ba[2] = {128, a_rows};
  const uint32_t bb[2] = {a.transposed ? 128 : w_cols, a.transposed ? w_cols : 128};
  if (moe_status_t st = encode_tensor_map(tmA, a.a, 2, da, sa, ba, CU_TENSOR_MAP_DATA_TYPE_UINT8,
                                          CU_TENSOR_MAP_SWIZZLE_128B))
    return st;
  const uint64_t db[2] = {a.transposed ? K : N, a.transposed ? N : K}, sb[1] = {db[0]};
  return encode_tensor_map(tmB, a.w, 2, db, sb, bb, CU_TENSOR_MAP_DATA_TYPE_UINT8,
                           bb[0] == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B);
}

// Tensor map of the output, boxes of 32 rows x 128 bytes.
moe_status_t dense_out_map(const MatmulFp8Args& a, CUtensorMap* tmO) {
  const uint64_t eb = a.out_f32 ? 4 : 2;
  const uint64_t d[2] = {static_cast<uint64_t>(a.N), static_cast<uint64_t>(a.M)};
  const uint64_t st[1] = {static_cast<uint64_t>(a.N) * eb};
  const uint32_t box[2] = {static_cast<uint32_t>(128 / eb), 32};
  return encode_tensor_map(
      tmO, a.out, 2, d, st, box,
      a.out_f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
      CU_TENSOR_MAP_SWIZZLE_128B);
}

template <bool TR, int NT>
moe_status_t launch_pair(const MatmulFp8Args& a, const DenseParams& P, cudaStream_t s) {
  static PerDevice attr;
  int regs = 0;
  if (attr.get(
          [](int* v) {
            cudaFuncAttributes fa;
            const cudaError_t e = cudaFuncGetAttributes(&fa, dense_fp8_pair_kernel<TR, NT>);
            if (e != cudaSuccess) return e;
            *v = fa.numRegs;
            return cudaFuncSetAttribute(dense_fp8_pair_kernel<TR, NT>,
                                        cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        static_cast<int>(DpGeo<NT>::SMEM));
          },
          &regs) != cudaSuccess)
    return set_error(MOE_ERR_CUDA, "attributes of matmul_fp8: %s",
                     cudaGetErrorString(cudaGetLastError()));
  // fewer registers at launch would leave the promotion warps waiting for more
  if (NT == 256 && regs < kDpRegsLaunch)
    return set_error(MOE_ERR_CUDA, "matmul_fp8 was compiled to %d registers, %d needed", regs,
                     kDpRegsLaunch);
  CUtensorMap tmA, tmB, tmO;
  if (moe_status_t st = dense_maps(a, 128, NT / 2, &tmA, &tmB)) return st;
  if (moe_status_t st = dense_out_map(a, &tmO)) return st;
  const int64_t tiles = ceil_div<int64_t>(a.M, 256) * ceil_div(a.N, NT);
  const unsigned grid = 2u * static_cast<unsigned>(std::min<int64_t>(tiles, a.num_sms / 2));
  const char* name = NT == 256 ? "matmul_fp8_pairs256" : "matmul_fp8_pairs128";
  prof_before(name, s);
  launch_kernel(dense_fp8_pair_kernel<TR, NT>, grid, kDpThreads, DpGeo<NT>::SMEM, s, tmA, tmB, tmO, P);
  prof_after(name, s);
  return check_launch("matmul_fp8");
}

// A launch of the split kernel with clusters of S (cfg.attrs: room for two).
template <int T, bool TR>
void split_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute* at, int S, int nt, int64_t mt) {
  cfg.gridDim = dim3(static_cast<unsigned>(nt * S), static_cast<unsigned>(mt));
  cfg.blockDim = dim3(kDsThreads);
  cfg.dynamicSmemBytes = DsGeo<T>::SMEM;
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = pdl_enabled() ? 1 : 0;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = static_cast<unsigned>(S);
  at[1].val.clusterDim.y = 1;
  at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
}

// Parts of K for the split kernel: the most whose clusters are all resident at
// once (one cluster too many makes a second wave: 17 clusters of 8 took 20.7 us
// for 128 x 4096 x 2064, 17 of 7 11.7).  What fits is asked once per host thread
// and device (dev: the current one).
template <int T, bool TR>
int split_parts(int dev, int64_t clusters, int KB) {
  constexpr int MAX_S = 8;  // a portable cluster
  thread_local int room_dev = -1, room[MAX_S + 1];
  if (dev != room_dev) {
    if (cudaFuncSetAttribute(dense_fp8_split_kernel<T, TR>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(DsGeo<T>::SMEM)) != cudaSuccess) {
      cudaGetLastError();
      return 1;
    }
    for (int c = 2; c <= MAX_S; ++c) {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute at[2];
      split_config<T, TR>(cfg, at, c, 1, 1);
      if (cudaOccupancyMaxActiveClusters(&room[c], dense_fp8_split_kernel<T, TR>, &cfg) !=
          cudaSuccess) {
        cudaGetLastError();
        room[c] = 0;
      }
    }
    room_dev = dev;
  }
  int S = 1;
  for (int c = 2; c <= std::min(MAX_S, KB) && clusters <= room[c]; ++c) S = c;
  return S;
}

template <int T, bool TR>
moe_status_t launch_split(const MatmulFp8Args& a, const DenseParams& P, int S, cudaStream_t s) {
  CUtensorMap tmA, tmB;
  if (moe_status_t st = dense_maps(a, T, 128, &tmA, &tmB)) return st;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[2];
  split_config<T, TR>(cfg, at, S, ceil_div(a.N, 128), ceil_div<int64_t>(a.M, T));
  cfg.stream = s;
  const char* name = T == 16   ? "matmul_fp8_split16"
                     : T == 32 ? "matmul_fp8_split32"
                     : T == 64 ? "matmul_fp8_split64"
                     : T == 96 ? "matmul_fp8_split96"
                               : "matmul_fp8_split128";
  prof_before(name, s);
  cudaLaunchKernelEx(&cfg, dense_fp8_split_kernel<T, TR>, tmA, tmB, P, S);
  prof_after(name, s);
  return check_launch("matmul_fp8");
}

// The kernel for a call: the least of the times estimated from a fixed part
// and one per K block of a CTA, as measured on GB300 (us; K x N of 7168 x 4096,
// 2048 x 7168, 4096 x 2064 and 1024 x 1024, 1 to 2048 rows):
//   split, 16 rows a tile: 3.5 + 0.35    32 rows: 3.7 + 0.36
//          64 rows: 4.2 + 0.39           96 rows: 5.0 + 0.43
//         128 rows: 5.7 + 0.52
//   pairs, 256 columns a tile: 4.8 + 0.43    128 columns: 4.7 + 0.295
// e.g. 77 x 7168 x 4096: 12.3 (128), 11.1 (96); 192 x 4096 x 2064: 9.8, 8.6; 65 x 1024 x
// 1024: 4.6 (64), 5.4 (96); 256 x 7168 x 4096: 25.7 (64), 20.8 (128), 28.3 (wide pairs);
// 256 x 2048 x 7168: 13.7 (128), 11.6 (wide), 9.4 (narrow pairs); 512 x 7168 x 4096: 28.3
// (wide), 21.2; 1999 x 4096 x 2064: 20.1, 25.2; 512 x 1024 x 1024: 5.9 (64), 7.3 (128).
template <bool TR>
moe_status_t launch_matmul(const MatmulFp8Args& a, const DenseParams& P, cudaStream_t s) {
  const int nt = ceil_div(a.N, 128), KB = ceil_div(a.K, 128);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess)
    return set_error(MOE_ERR_CUDA, "matmul_fp8: %s", cudaGetErrorString(cudaGetLastError()));
  // T: rows of a split kernel's tile; 512 and 256 stand for the wide and narrow pairs
  const int64_t mt2 = ceil_div<int64_t>(a.M, 256), nt2 = ceil_div(a.N, 256);
  const auto pairs = [&](float fixed, float per_block, int64_t tiles) {
    return fixed + per_block * KB * static_cast<float>(ceil_div<int64_t>(tiles, a.num_sms / 2));
  };
  float best = pairs(4.8f, 0.43f, mt2 * nt2);
  int T = 512, S = 1;
  if (const float t = pairs(4.7f, 0.295f, mt2 * nt); t < best) {
    best = t;
    T = 256;
  }
  auto consider = [&](auto rows, float fixed, float per_block) {
    constexpr int R = decltype(rows)::value;
    const int64_t mt = ceil_div<int64_t>(a.M, R);
    if (mt > 64) return;  // the pairs' case, and a bound of the grid's y
    const int parts = split_parts<R, TR>(dev, nt * mt, KB);
    const int64_t waves = ceil_div<int64_t>(nt * mt * parts, a.num_sms);
    const float t = fixed + per_block * ceil_div(KB, parts) * static_cast<float>(waves);
    if (t < best) {
      best = t;
      T = R;
      S = parts;
    }
  };
  consider(std::integral_constant<int, 128>{}, 5.7f, 0.52f);
  consider(std::integral_constant<int, 96>{}, 5.0f, 0.43f);
  consider(std::integral_constant<int, 64>{}, 4.2f, 0.39f);
  consider(std::integral_constant<int, 32>{}, 3.7f, 0.36f);
  consider(std::integral_constant<int, 16>{}, 3.5f, 0.35f);
  if (T == 16) return launch_split<16, TR>(a, P, S, s);
  if (T == 32) return launch_split<32, TR>(a, P, S, s);
  if (T == 64) return launch_split<64, TR>(a, P, S, s);
  if (T == 96) return launch_split<96, TR>(a, P, S, s);
  if (T == 128) return launch_split<128, TR>(a, P, S, s);
  if (T == 256) return launch_pair<TR, 128>(a, P, s);
  return launch_pair<TR, 256>(a, P, s);
}

}  // namespace

moe_status_t launch_quant_groups_fp8(const QuantGroupsArgs& a, cudaStream_t s) {
  const int64_t units = a.M * ceil_div(a.K, a.swiglu ? 512 : 1024);
  const unsigned grid =
      static_cast<unsigned>(std::min<int64_t>(ceil_div<int64_t>(units, kQgWarps), a.num_sms * kQgBlocks));
  prof_before("quant_groups_fp8", s);
  launch_kernel(a.swiglu ? quant_groups_kernel<true> : quant_groups_kernel<false>, grid,
                kQgWarps * 32, 0, s, a.x, a.M, a.K, a.q8, a.scale);
  prof_after("quant_groups_fp8", s);
  return check_launch("quant_groups_fp8");
}

moe_status_t launch_matmul_fp8(const MatmulFp8Args& a, cudaStream_t s) {
  const DenseParams P{a.a_scale, a.w_scale, a.bias, a.out, a.M, a.K, a.N, a.out_f32, a.error_word};
  return a.transposed ? launch_matmul<true>(a, P, s) : launch_matmul<false>(a, P, s);
}

}  // namespace gbmoe
