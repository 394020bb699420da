// What the dense and grouped products share: packed fp32 pairs, SiLU on them,
// bounded waits, TMEM loads tied to their wait.
#pragma once
#include "common.cuh"
#include "fp8q.cuh"
#include "ptx.cuh"

namespace gbmoe {

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
constexpr float kFastGate = 80.f;  // gates below it in size take the fast form
// -(1 + e^-x) of a pair, and approximate reciprocals of 1 + e^-x.
__device__ __forceinline__ uint64_t neg_one_plus_exp2(uint64_t x, uint64_t& r) {
  const uint64_t minus1 = pair_of(-1.0f, -1.0f);
  const uint64_t h = mul2(x, pair_of(kLog2E, kLog2E));
  const uint64_t t = fma2(h, pair_of(-kLn2Lo, -kLn2Lo), fma2(h, pair_of(-kLn2Hi, -kLn2Hi), x));
  const float2 h1 = unpair(h);
  float p0, p1, r0, r1;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p0) : "f"(-h1.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p1) : "f"(-h1.y));
  const uint64_t nden = fma2(pair_of(p0, p1), add2(t, minus1), minus1);
  const float2 d = unpair(nden);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r0) : "f"(-d.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r1) : "f"(-d.y));
  r = pair_of(r0, r1);
  return nden;
}
__device__ __forceinline__ void swiglu8(float (&g)[8], const float (&u)[8]) {
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(g[j]));
  if (top < kFastGate) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      const uint64_t x = pair_of(g[j], g[j + 1]);
      uint64_t r;
      const uint64_t nden = neg_one_plus_exp2(x, r);
      const float2 z = unpair(mul2(div_fixed2(x, nden, r), pair_of(u[j], u[j + 1])));
      g[j] = z.x;
      g[j + 1] = z.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = g[j] / (1.0f + expf(-g[j])) * u[j];
  }
}

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

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}

__device__ __forceinline__ void st_cluster_f32x4(uint32_t addr, float a, float b, float c, float d) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "f"(a), "f"(b),
               "f"(c), "f"(d)
               : "memory");
}

// The two halves of a cluster barrier; this arrival orders nothing (a releasing
// one waits for the thread's loads in flight).
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

}  // namespace gbmoe
