// Routing with a per-expert bias for load balance, and the gradient of the
// routing weights.
//
// Scores p (softmax over the experts or sigmoid) as in moe_route; the choice
// of experts is by c_e = p_e + b_e, the weights are the chosen experts' p.
// c is compared as in 64-bit arithmetic: two fp32 values of c closer than
// their rounding say nothing about the order of the exact ones, and the ids
// are integers, right or wrong.
#include <algorithm>

#include "common.cuh"

namespace gbmoe {
namespace {

constexpr int kRbWarps = 4;  // tokens (one per warp) of a block

__device__ __forceinline__ float rb_f32(float v) { return v; }
__device__ __forceinline__ float rb_f32(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void rb_store(float* p, float v) { *p = v; }
__device__ __forceinline__ void rb_store(bf16* p, float v) { *p = __float2bfloat16(v); }

__device__ __forceinline__ float rb_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <typename T>
__device__ __forceinline__ T rb_sum(T v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

struct RbParams {
  int64_t M;
  int E, top_k, method, renormalize, k_group, group_count, group_select_mode;
  float scale;
  int gs, gs_inv;   // experts of a group; ceil(2^20 / gs): e / gs = e gs_inv >> 20 for e < 1024
  int lpg_log;      // WHOLE (below): log2 of the lanes that hold a group
};

// Order-preserving map of a double to an unsigned key, and back; NaN goes with
// -inf, and 0 is below every key.  (Comparisons of doubles run at this GPU's
// FP64 rate: the choice below took 30 us per token with them.)
__device__ __forceinline__ uint64_t rb_key64(double v) {
  if (!(v == v)) v = -INFINITY;
  const uint64_t b = static_cast<uint64_t>(__double_as_longlong(v));
  return (b >> 63) ? ~b : (b | (uint64_t(1) << 63));
}
__device__ __forceinline__ double rb_value64(uint64_t k) {
  return __longlong_as_double(
      static_cast<long long>((k >> 63) ? k & ~(uint64_t(1) << 63) : ~k));
}

// A score in 64 bits: sigmoid, or exp(l - m).  (One warp-wide FP64 operation
// takes 64 cycles here, a sigmoid about 2000: the paths below call this for as
// few experts as they can.)
__device__ __noinline__ double rb_score64(float l, bool softmax, float m) {
  const double e = exp(softmax ? static_cast<double>(l) - m : -static_cast<double>(l));
  return softmax ? e : 1.0 / (1.0 + e);
}

// Largest key over the warp; i: the lowest index among the lanes that have it.
__device__ __forceinline__ uint64_t rb_warp_best(uint64_t v, int& i) {
  const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(v >> 32));
  const uint32_t lo = __reduce_max_sync(
      0xffffffffu, static_cast<uint32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u);
  const uint64_t best = static_cast<uint64_t>(hi) << 32 | lo;
  i = static_cast<int>(
      __reduce_min_sync(0xffffffffu, v == best ? static_cast<uint32_t>(i) : 0x7fffffffu));
  return best;
}

// The largest of keys c[first], c[first + 32], ... below n, and its index
// (the lowest of equals).
__device__ __forceinline__ uint64_t rb_scan(const uint64_t* c, int first, int n, int& i) {
  uint64_t v = 0;
  i = 0x7fffffff;
#pragma unroll 4
  for (int e = first; e < n; e += 32)
    if (c[e] > v) {
      v = c[e];
      i = e;
    }
  return v;
}

// One token's choice in 64 bits, by one warp.  c: E + group_count keys in
// shared memory.  Lane j receives chosen experts j and j + 32.  A candidate
// that is out (its group not kept, or chosen) has key 0; a masked expert
// (logit -inf) or a NaN score has that of -inf and comes last.
template <typename T>
__device__ __noinline__ int2 rb_choose64(const T* row, const float* bias, const RbParams& P,
                                         uint64_t* c) {
  const int lane = threadIdx.x & 31;
  const int E = P.E;
  const bool softmax = P.method == MOE_ROUTE_SOFTMAX;
  float m = 0.f;
  double inv = 1.0;
  if (softmax) {
    m = -INFINITY;
    for (int e = lane; e < E; e += 32) m = fmaxf(m, rb_f32(row[e]));
    m = rb_max(m);
    double s = 0.0;
#pragma unroll 1
    for (int e = lane; e < E; e += 32) {
      const double x = rb_score64(rb_f32(row[e]), true, m);
      c[e] = static_cast<uint64_t>(__double_as_longlong(x));  // (for the loop below)
      s += x;
    }
    inv = 1.0 / rb_sum(s);
  }
#pragma unroll 1
  for (int e = lane; e < E; e += 32) {
    const float l = rb_f32(row[e]);
    const double x = softmax ? __longlong_as_double(static_cast<long long>(c[e]))
                             : rb_score64(l, false, m);
    c[e] = rb_key64(l == -INFINITY ? -INFINITY
                                   : fma(x, inv, static_cast<double>(bias[e])) + 0.0);
  }
  __syncwarp();
  if (P.group_count > 1) {
    const int G = P.group_count, gs = E / G;
    uint64_t* gk = c + E;
    for (int g = lane; g < G; g += 32) {
      uint64_t b1 = 0, b2 = 0;
#pragma unroll 4
      for (int j = 0; j < gs; ++j) {
        const uint64_t v = c[g * gs + j];
        b2 = max(b2, min(b1, v));
        b1 = max(b1, v);
      }
      gk[g] = P.group_select_mode == 0 ? b1 : rb_key64(rb_value64(b1) + rb_value64(b2));
    }
    __syncwarp();
    // the k_group best groups leave gk (0); what is left there is dropped
    for (int r = 0; r < P.k_group; ++r) {
      int i;
      rb_warp_best(rb_scan(gk, lane, G, i), i);
      if (lane == 0) gk[i] = 0;
      __syncwarp();
    }
    for (int e = lane; e < E; e += 32)
      if (gk[e / gs] != 0) c[e] = 0;
    __syncwarp();
  }
  int2 id = make_int2(0, 0);
  int mine;
  uint64_t v = rb_scan(c, lane, E, mine);
  for (int j = 0; j < P.top_k; ++j) {
    int i = mine;
    rb_warp_best(v, i);
    if (lane == (j & 31)) (j < 32 ? id.x : id.y) = i;
    if (i == mine) {  // this lane's: the next best of its experts
      c[i] = 0;
      v = rb_scan(c, lane, E, mine);
    }
  }
  return id;
}

// A sigmoid, over e^top where the largest chosen logit top is below 0: scores that
// underflow by themselves, and those below -88 where 1 / (1 + e^-l) is 0, keep their
// ratio to the others.  (top is the token's: its lanes go one way.)
__device__ __forceinline__ float rb_sigmoid_over(float l, float top) {
  if (top >= 0.f) {
    const float a = expf(-fabsf(l));
    return (l < 0.f ? a : 1.0f) / (1.0f + a);
  }
  return expf(l - top) / (1.0f + expf(l));
}

// Weights of the chosen experts (lane j: chosen j and j + 32), in fp32.
// Ratios of the chosen scores come from the logits' differences where the
// scores themselves would underflow; a masked expert's weight is 0, and a
// token with nothing but masked experts has weights of 0.
template <typename T>
__device__ __noinline__ void rb_weights(const T* row, const RbParams& P, int id0, int id1,
                                        float* out_w, int32_t* out_ids) {
  const int lane = threadIdx.x & 31;
  // softmax: the row's largest logit and the sum of exp(l - mx) over it (NaN
  // where the row holds a NaN or +inf)
  float mx = -INFINITY, sum = 0.f;
  if (P.method == MOE_ROUTE_SOFTMAX) {
    for (int e = lane; e < P.E; e += 32) mx = fmaxf(mx, rb_f32(row[e]));
    mx = rb_max(mx);
    for (int e = lane; e < P.E; e += 32) sum += expf(rb_f32(row[e]) - mx);
    sum = rb_sum(sum);
  }
  const bool h0 = lane < P.top_k, h1 = lane + 32 < P.top_k;
  const float l0 = h0 ? rb_f32(row[id0]) : -INFINITY, l1 = h1 ? rb_f32(row[id1]) : -INFINITY;
  const bool masked = __all_sync(0xffffffffu, l0 == -INFINITY && l1 == -INFINITY);
  const bool bad = P.method == MOE_ROUTE_SOFTMAX && sum != sum;
  const bool renorm = P.method == MOE_ROUTE_SIGMOID || P.renormalize;
  if (renorm) mx = rb_max(fmaxf(l0, l1));
  float p0, p1;
  if (P.method == MOE_ROUTE_SIGMOID) {
    p0 = rb_sigmoid_over(l0, mx);
    p1 = rb_sigmoid_over(l1, mx);
  } else {
    p0 = expf(l0 - mx);
    p1 = expf(l1 - mx);
  }
  if (renorm) sum = rb_sum((h0 ? p0 : 0.f) + (h1 ? p1 : 0.f));
  const float f = bad ? NAN : 1.0f;
  if (h0) {
    out_ids[lane] = id0;
    out_w[lane] = masked ? 0.f : p0 / sum * P.scale * f;
  }
  if (h1) {
    out_ids[lane + 32] = id1;
    out_w[lane + 32] = masked ? 0.f : p1 / sum * P.scale * f;
  }
}

// Every token by the 64-bit choice: more than 30 experts per token, or more
// groups than a warp has lanes.
template <typename T>
__global__ void __launch_bounds__(kRbWarps * 32)
    route_biased_exact_kernel(const T* __restrict__ logits, const float* __restrict__ bias, RbParams P,
                        float* __restrict__ out_w, int32_t* __restrict__ out_ids) {
  pdl_begin();
  extern __shared__ uint64_t rb_smem[];
  const int warp = threadIdx.x >> 5;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp;
  if (t >= P.M) return;
  const T* row = logits + t * P.E;
  const int2 id = rb_choose64(row, bias, P, rb_smem + warp * (P.E + P.group_count));
  rb_weights(row, P, id.x, id.y, out_w + t * P.top_k, out_ids + t * P.top_k);
}

// Order-preserving map of a float (neither NaN nor -0) to an unsigned key, and back.
__device__ __forceinline__ uint32_t rb_key(float f) {
  const uint32_t b = __float_as_uint(f);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float rb_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// 2^x (within 2^-22 of it) and 1 / x (within 2^-23), relative.
__device__ __forceinline__ float rb_ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rb_rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float kLog2e = 1.44269504f;

// The N largest keys of a lane in descending order, from EPL of them.
__device__ __forceinline__ void rb_order(uint32_t& a, uint32_t& b) {
  const uint32_t hi = max(a, b);
  b = min(a, b);
  a = hi;
}
__device__ __forceinline__ void rb_sort4(uint32_t (&t)[4]) {
  rb_order(t[0], t[1]);
  rb_order(t[2], t[3]);
  rb_order(t[0], t[2]);
  rb_order(t[1], t[3]);
  rb_order(t[1], t[2]);
}
template <int EPL>
__device__ __forceinline__ void rb_top4(const uint32_t (&key)[EPL], uint32_t (&t)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) t[i] = i < EPL ? key[i] : 0u;
  rb_sort4(t);
#pragma unroll
  for (int q = 4; q < EPL; q += 4) {
    uint32_t u[4] = {key[q], key[q + 1], key[q + 2], key[q + 3]};
    rb_sort4(u);
    // the larger half of two sorted quads, a bitonic sequence again
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = max(t[i], u[3 - i]);
    rb_order(t[0], t[2]);
    rb_order(t[1], t[3]);
    rb_order(t[0], t[1]);
    rb_order(t[2], t[3]);
  }
}

template <int LPT, typename F>
__device__ __forceinline__ F rb_seg_max(F v) {
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}
template <int LPT>
__device__ __forceinline__ float rb_seg_sum(float v) {
#pragma unroll
  for (int o = LPT / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The largest key of a segment, by the warp's reduction (one for each half of the
// warp: 5 instructions where exchanges take 8, and the shorter chain).
template <int LPT>
__device__ __forceinline__ uint32_t rb_seg_top(uint32_t v, int seg0) {
  if constexpr (LPT == 32) return __reduce_max_sync(0xffffffffu, v);
  const uint32_t first = __reduce_max_sync(0xffffffffu, seg0 == 0 ? v : 0u);
  const uint32_t second = __reduce_max_sync(0xffffffffu, seg0 == 0 ? 0u : v);
  return seg0 == 0 ? first : second;
}

// N consecutive logits as floats; vec: N elements at p are there and aligned.
template <int N>
__device__ __forceinline__ void rb_load(const float* p, float (&l)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
      l[i] = v.x;
      l[i + 1] = v.y;
      l[i + 2] = v.z;
      l[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 v = __ldg(reinterpret_cast<const float2*>(p + i));
      l[i] = v.x;
      l[i + 1] = v.y;
    }
  }
}
__device__ __forceinline__ void rb_pair(uint32_t u, float& a, float& b) {
  a = __uint_as_float(u << 16);
  b = __uint_as_float(u & 0xffff0000u);
}
template <int N>
__device__ __forceinline__ void rb_load(const bf16* p, float (&l)[N]) {
  if constexpr (N % 8 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 8) {
      const uint4 v = __ldg(reinterpret_cast<const uint4*>(p + i));
      rb_pair(v.x, l[i], l[i + 1]);
      rb_pair(v.y, l[i + 2], l[i + 3]);
      rb_pair(v.z, l[i + 4], l[i + 5]);
      rb_pair(v.w, l[i + 6], l[i + 7]);
    }
  } else if constexpr (N == 4) {
    const uint2 v = __ldg(reinterpret_cast<const uint2*>(p));
    rb_pair(v.x, l[0], l[1]);
    rb_pair(v.y, l[2], l[3]);
  } else {
    rb_pair(__ldg(reinterpret_cast<const uint32_t*>(p)), l[0], l[1]);
  }
}

// The choice in fp32 where fp32 decides it.
//
// LPT lanes per token, EPL experts per lane.  A candidate is one 32-bit key: c in
// order-preserving form with its low bits replaced by the expert (complemented: the
// lower id wins), so that a maximum over the lanes is a chosen expert; each lane
// offers its four largest in turn, and past those its largest below the last one it
// gave.  top_k + 2 rounds leave a candidate per lane.  Their exact fp32 c (the keys'
// low bits back) puts them in order, and the choice stands if no two neighbours down to
// the (top_k + 1)-th are closer than the error of c, nor the top_k-th and what was not a
// candidate; equal logits with equal biases are ties for certain.  Candidates that are
// too close (a token in a thousand of normally distributed scores) are ranked in 64 bits
// by the lanes, after as many rounds as there are lanes if the rest is too near as well;
// groups that are too close likewise, from their two best experts.  Where that does not
// settle it, or a score is NaN, the warp takes the token by rb_choose64 (20 us for one
// token of 512 experts, which is why the steps before it are there: 10804 x 336 softmax,
// 13 of 4 of 8 groups, with two such tokens 80 us, now 25).
//
// WHOLE: lanes hold EPL consecutive experts or none, of one group (a power of two of
// lanes to a group).  Otherwise every LPT-th expert, so that loads of rows of any length
// are whole lines.
//
// Bound: latency.  A warp takes its tokens one after the other with nothing loaded ahead,
// and the blocks of many tokens are little more than are resident: 8192 x 256 are 1.12
// waves (6 blocks of four warps per SM at 80 registers), issue slots 44 % busy, loads the
// largest stall; 16384 x 128 are 1.92 waves (7 per SM at 72), 57 %.  The last warp is often
// one whose token needed 64 bits.  In a graph, over 24 seeds: 8192 tokens x 256 experts, 8
// of 4 of 8 groups, 9.5 to 13.0 us (every token by rb_choose64: 281); 16384 x 128 bf16
// softmax, 8 chosen, 10.1 to 17.2 (298); one token of 256 experts 3.0.
template <int EPL, int LPT, bool WHOLE, typename T>
__global__ void __launch_bounds__(kRbWarps * 32, EPL <= 16 ? 6 : 1)  // (six: 72-80 registers)
    route_biased_kernel(const T* __restrict__ logits, const float* __restrict__ bias, RbParams P,
                        int vec, float* __restrict__ out_w, int32_t* __restrict__ out_ids) {
  pdl_begin();
  extern __shared__ uint64_t rb_smem[];
  constexpr int TPW = 32 / LPT;
  constexpr uint32_t MASK = LPT * EPL - 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sl = lane % LPT, seg0 = lane - sl;
  const int E = P.E, G = P.group_count, k = P.top_k, gs = P.gs;
  const bool softmax = P.method == MOE_ROUTE_SOFTMAX, grouped = P.k_group < G;
  const int e0 = sl * EPL;
  auto expert = [&](int i) { return WHOLE ? e0 + i : sl + LPT * i; };
  auto exists = [&](int i) { return WHOLE ? e0 < E : expert(i) < E; };
  uint64_t* sm = rb_smem + warp * (E + G);
  float b[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) b[i] = exists(i) ? __ldg(bias + expert(i)) : 0.f;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (blockDim.x >> 5) * TPW;
  for (int64_t t0 = (static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp) * TPW; t0 < P.M;
       t0 += step) {
    const bool live = t0 + seg0 / LPT < P.M;
    const int64_t t = live ? t0 + seg0 / LPT : P.M - 1;
    const T* row = logits + t * E;
    float c[EPL];
    if (WHOLE && vec && e0 < E) {
      rb_load<EPL>(row + e0, c);
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) c[i] = exists(i) ? rb_f32(row[expert(i)]) : -INFINITY;
    }
    // ---- c = p + b (p = exp(l - mx) cf for softmax) ----
    float lo = c[0], mx = c[0], sum = 0.f, cf = 1.f;
#pragma unroll
    for (int i = 1; i < EPL; ++i) lo = fminf(lo, c[i]);
    if (softmax) {
#pragma unroll
      for (int i = 1; i < EPL; ++i) mx = fmaxf(mx, c[i]);
      mx = rb_seg_max<LPT>(mx);
      // (the difference first, as in the weights' numerator: l log2 e - mx log2 e with a
      // rounded second term scales every exp by 2^(its error), which the numerator does
      // not see, and for large logits lowers cf below the largest p)
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        c[i] = rb_ex2((c[i] - mx) * kLog2e);
        sum += c[i];
      }
      sum = rb_seg_sum<LPT>(sum);
      cf = 1.0f / sum;
#pragma unroll
      for (int i = 0; i < EPL; ++i) c[i] = fmaf(c[i], cf, b[i]);
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) c[i] = rb_rcp(1.0f + rb_ex2(-kLog2e * c[i])) + b[i];
    }
    if (lo == -INFINITY) {  // masked experts of this lane, or none at all here
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (!exists(i) || rb_f32(row[expert(i)]) == -INFINITY) c[i] = -INFINITY;
    }
    const float p1 = softmax ? cf : 1.0f;
    // error of a difference of two c, over p1.  Sigmoid: the exponential's
    // 2^-22 + |l| 2^-23.5 times p (1 - p) (at most 2^-23.5), the sum's 2^-24, the
    // reciprocal's 2^-23, twice.  Softmax, in 2^-24, with d = mx - l: an exponential's 4
    // and its argument's 2.25 d (d e^-d is below 0.4), twice; once, as it is common to
    // the row, the sum's: its terms' 4 and 2.25 times their mean d (below 4.5 for 1024
    // experts), EPL + 5 additions, the reciprocal: EPL + 30 of the 2 EPL + 36 here.
    // The rounding of the bias' addition is in the comparisons.
    const float kerr = softmax ? 2.0f * (18 + EPL) * 5.9604645e-8f : 6e-7f;
    bool hard = false;  // needs rb_choose64
#pragma unroll
    for (int i = 0; i < EPL; ++i) hard |= c[i] != c[i];
    // softmax: 1 / sum of exp(l - mx) for what is compared in 64 bits.  The sum stays in
    // pairs of fp32: a term is expf (2 ulp, 4 in 2^-24) with what l - mx lost in its
    // rounding put back (a rounding, 1), the additions' errors are kept.  5 in all, below
    // sum_err: common to all scores, it moves a difference of two c by as much of that
    // of their p.  (The tokens that this leaves open are what a call's end waits for.)
    constexpr float sum_err = 3.2e-7f;
    auto inv64 = [&]() {
      float s = 0.f, comp = 0.f;
      auto add = [&](float x, float more) {  // (the same bits with its operands exchanged:
        const float y = s + x;               // all lanes get one inverse)
        comp = (comp + more) + (s >= x ? (s - y) + x : (x - y) + s);
        s = y;
      };
#pragma unroll 1
      for (int i = sl; i < E; i += LPT) {
        const float l = rb_f32(row[i]), d = l - mx, back = d + mx;
        // l - mx - d, exactly (Knuth's sum of two)
        const float r = d > -200.f ? (l - back) + ((back - d) - mx) : 0.f;
        const float x = expf(d);
        add(fmaf(x, r, x), 0.f);
      }
#pragma unroll
      for (int o = LPT / 2; o > 0; o >>= 1)
        add(__shfl_xor_sync(0xffffffffu, s, o), __shfl_xor_sync(0xffffffffu, comp, o));
      return 1.0 / (static_cast<double>(s) + comp);
    };
    // such a difference dc is open where the sum's error could turn it
    auto undecided = [&](double dc, double dp) {
      return softmax && dp != 0.0 && !(fabsf(static_cast<float>(dc)) > sum_err * fabsf(static_cast<float>(dp)));
    };
    // ---- groups: kept ones as a mask of the segment ----
    uint32_t kept = 0xffffffffu;
    if (grouped) {
      // lane g: group g's score, and the size of what it is the sum of; -1 for a score
      // that is -inf exactly (its experts masked, or all but one of those that it sums)
      float gk = -INFINITY, mag = -1.f;
      const bool sum2 = P.group_select_mode != 0;
      auto size = [&](float b1, float b2) {
        return (sum2 ? b2 : b1) == -INFINITY ? -1.f : sum2 ? fabsf(b1) + fabsf(b2) : fabsf(b1);
      };
      auto score = [&](float b1, float b2) {  // (inf - inf counts as -inf)
        return !sum2 ? b1 : b2 == -INFINITY ? -INFINITY : b1 + b2;
      };
      float* row_c = reinterpret_cast<float*>(sm) + (seg0 / LPT) * E;
      auto store_c = [&]() {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (exists(i)) row_c[expert(i)] = c[i];
        __syncwarp();
      };
      const int lpg = 1 << P.lpg_log;  // WHOLE: lanes of a group
      if constexpr (WHOLE) {
        float b1 = c[0], b2 = -INFINITY;
#pragma unroll
        for (int i = 1; i < EPL; ++i) {
          b2 = fmaxf(b2, fminf(b1, c[i]));
          b1 = fmaxf(b1, c[i]);
        }
        for (int o = 1; o < lpg; o <<= 1) {
          const float o1 = __shfl_xor_sync(0xffffffffu, b1, o);
          const float o2 = __shfl_xor_sync(0xffffffffu, b2, o);
          b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));
          b1 = fmaxf(b1, o1);
        }
        const int from = seg0 + min(sl * lpg, LPT - 1);
        gk = __shfl_sync(0xffffffffu, score(b1, b2), from);
        mag = __shfl_sync(0xffffffffu, size(b1, b2), from);
      } else {
        // by parts of a group per lane, joined in lane g
        const int parts = LPT / G, part = sl / G, g = sl - part * G;
        float b1 = -INFINITY, b2 = -INFINITY;
        store_c();
        if (part < parts) {
#pragma unroll 4
          for (int j = part; j < gs; j += parts) {
            const float v = row_c[g * gs + j];
            b2 = fmaxf(b2, fminf(b1, v));
            b1 = fmaxf(b1, v);
          }
        }
        for (int p = 1; p < parts; ++p) {
          const int from = seg0 + min(sl + p * G, LPT - 1);
          const float o1 = __shfl_sync(0xffffffffu, b1, from);
          const float o2 = __shfl_sync(0xffffffffu, b2, from);
          if (sl < G) {
            b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));
            b1 = fmaxf(b1, o1);
          }
        }
        gk = score(b1, b2);
        mag = size(b1, b2);
      }
      if (sl >= G) gk = -INFINITY;
      // rank among the groups, and the groups too close to tell apart: each of the two c
      // and their sum are rounded, 2^-24 of each, so that c of both signs leave an error
      // that their sum's size says nothing of (the lane of the larger ones sees it)
      const float gerr = 3.0f * (kerr * p1 + 1.2e-7f * mag);
      int rank = 0;
      uint32_t near = 0;
      for (int h = 0; h < G; ++h) {
        const float o = __shfl_sync(0xffffffffu, gk, seg0 + h);
        rank += (o > gk || (o == gk && h < sl)) ? 1 : 0;
        if (!(fabsf(o - gk) > gerr)) near |= 1u << h;
      }
      // (-inf is below all others and the index settles its ties.  Sums that only fp32
      // takes to -inf are near every other by their own lane, where mag is inf)
      if (mag < 0.f) near = 0u;
      const uint32_t all = __ballot_sync(0xffffffffu, sl < G && rank < P.k_group);
      kept = LPT == 32 ? all : (all >> seg0) & ((1u << (LPT & 31)) - 1u);
      // (a group's own bit is never on the other side)
      const bool unsure = sl < G && (((kept >> sl) & 1u) ? near & ~kept : near & kept) != 0u;
      if (const uint32_t which = __ballot_sync(0xffffffffu, unsure && live)) {
        // group scores in 64 bits (lane g: group g's) from the two best experts of each
        // lane or part, where its third is no rival of them
        const bool seg_unsure =
            (LPT == 32 ? which : (which >> seg0) & ((1u << (LPT & 31)) - 1u)) != 0u;
        const double inv = softmax ? inv64() : 1.0;
        float v1 = -INFINITY, v2 = -INFINITY, v3 = -INFINITY;
        int i1 = 0, i2 = 0;
        auto place = [&](float v, int i) {
          if (v > v1) {
            v3 = v2;
            v2 = v1;
            i2 = i1;
            v1 = v;
            i1 = i;
          } else if (v > v2) {
            v3 = v2;
            v2 = v;
            i2 = i;
          } else {
            v3 = fmaxf(v3, v);
          }
        };
        if constexpr (WHOLE) {
#pragma unroll
          for (int i = 0; i < EPL; ++i) place(c[i], e0 + i);
        } else if (sl < G) {
#pragma unroll 4
          for (int i = sl * gs; i < sl * gs + gs; ++i) place(row_c[i], i);
        }
        const bool holds = WHOLE ? e0 < E : sl < G;
        const float least = sum2 ? v2 : v1;  // v3's rival, if it is not as masked as v3
        if (seg_unsure && holds && least != -INFINITY)
          hard |= !(least - v3 > kerr * p1 + 1.2e-7f * fabsf(least));
        // the best two: keys of c and p
        uint64_t q1 = 0, q2 = 0;
        double pa = 0.0, pb = 0.0;
        if (holds) {
          pa = rb_score64(rb_f32(row[i1]), softmax, mx) * inv;
          pb = rb_score64(rb_f32(row[i2]), softmax, mx) * inv;
          q1 = rb_key64(v1 == -INFINITY ? -INFINITY : pa + __ldg(bias + i1) + 0.0);
          q2 = rb_key64(v2 == -INFINITY ? -INFINITY : pb + __ldg(bias + i2) + 0.0);
        }
        auto order = [](uint64_t& a, double& x, uint64_t& b, double& y) {
          if (a < b) {
            const uint64_t t = a;
            a = b;
            b = t;
            const double z = x;
            x = y;
            y = z;
          }
        };
        order(q1, pa, q2, pb);
        uint64_t q3 = 0;  // the best that the group's two leave out
        if constexpr (WHOLE) {
          for (int o = 1; o < 1 << P.lpg_log; o <<= 1) {
            uint64_t o1 = __shfl_xor_sync(0xffffffffu, q1, o), o2 = __shfl_xor_sync(0xffffffffu, q2, o);
            double oa = __shfl_xor_sync(0xffffffffu, pa, o), ob = __shfl_xor_sync(0xffffffffu, pb, o);
            order(q1, pa, o1, oa);
            order(q2, pb, o1, oa);
            order(q2, pb, o2, ob);
            q3 = max(max(q3, __shfl_xor_sync(0xffffffffu, q3, o)), max(o1, o2));
          }
        }
        // softmax: the sum's error could have put another one among them
        if (softmax) {
          if (!sum2) q3 = max(q2, q3);
          if (seg_unsure && q3 > rb_key64(-INFINITY))
            hard |= !(static_cast<float>(rb_value64(sum2 ? q2 : q1) - rb_value64(q3)) > sum_err * p1);
        }
        double c64 = rb_value64(q1), p64 = pa;
        if (P.group_select_mode == 1) {
          c64 += rb_value64(q2);
          p64 += pb;
        }
        if constexpr (WHOLE) {
          const int from = seg0 + min(sl << P.lpg_log, LPT - 1);
          c64 = __shfl_sync(0xffffffffu, c64, from);
          p64 = __shfl_sync(0xffffffffu, p64, from);
        }
        const uint64_t g64 = sl < G ? rb_key64(c64) : 0;
        rank = 0;
        uint32_t other = 0;  // near groups that these scores do not tell from this one
#pragma unroll 1
        for (int h = 0; h < G; ++h) {
          const uint64_t o = __shfl_sync(0xffffffffu, g64, seg0 + h);
          rank += (o > g64 || (o == g64 && h < sl)) ? 1 : 0;
          if (softmax) {
            const double op = __shfl_sync(0xffffffffu, p64, seg0 + h);
            if (((near >> h) & 1u) && h != sl && undecided(rb_value64(o) - c64, op - p64))
              other |= 1u << h;
          }
        }
        const uint32_t all64 = __ballot_sync(0xffffffffu, sl < G && rank < P.k_group);
        if (seg_unsure) {
          kept = LPT == 32 ? all64 : (all64 >> seg0) & ((1u << (LPT & 31)) - 1u);
          if (sl < G && (((kept >> sl) & 1u) ? other & ~kept : other & kept) != 0u) hard = true;
        }
      }
    }
    // ---- keys, the lane's four largest ----
    uint32_t key[EPL];
    uint32_t top4[4];
    if constexpr (WHOLE) {
      // (e0 is a multiple of EPL: MASK - e0 - i is (MASK - e0) ^ i)
#pragma unroll
      for (int i = 0; i < EPL; ++i) key[i] = ((rb_key(c[i]) & ~MASK) | (MASK - e0)) ^ i;
      rb_top4<EPL>(key, top4);
      if (e0 >= E || !((kept >> (grouped ? sl >> P.lpg_log : 0)) & 1u)) top4[0] = top4[1] = top4[2] = top4[3] = 0u;
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const bool in =
            exists(i) && (!grouped || ((kept >> (expert(i) * P.gs_inv >> 20)) & 1u));
        key[i] = in ? (rb_key(c[i]) & ~MASK) | (MASK - expert(i)) : 0u;
      }
      rb_top4<EPL>(key, top4);
    }
    // ---- top_k + 2 rounds ----
    uint32_t mine = 0, last = 0;
    int left = 4;  // of the lane's four
    auto round = [&](int r) {
      last = rb_seg_top<LPT>(top4[0], seg0);
      if (sl == r) mine = last;
      if (top4[0] == last) {
        top4[0] = top4[1];
        top4[1] = top4[2];
        top4[2] = top4[3];
        top4[3] = 0u;
        --left;
      }
      if (EPL > 4 && r >= 3 && __any_sync(0xffffffffu, left == 0)) {
        // a lane gave all four: its largest key below the last one.  (The
        // differences wrap, so that the nearest one below is the largest;
        // nothing left comes out as 0.)
        if (left == 0) {
          uint32_t d = key[0] - last;
#pragma unroll
          for (int i = 1; i < EPL; ++i) d = max(d, key[i] - last);
          top4[0] = last + d < last ? last + d : 0u;
          left = 1;
        }
      }
    };
    for (int r = 0; r < k + 2; ++r) round(r);
    // ---- the candidates' own c, in order ----
    int e;
    float l, be, ce;
    auto candidate = [&]() {
      e = mine ? static_cast<int>(MASK - (mine & MASK)) : 0x7fffffff;
      l = mine ? rb_f32(row[e]) : -INFINITY;
      be = mine ? __ldg(bias + e) : 0.f;
      ce = -INFINITY;
      if (l != -INFINITY)
        ce = softmax ? fmaf(rb_ex2((l - mx) * kLog2e), cf, be)
                     : rb_rcp(1.0f + rb_ex2(-kLog2e * l)) + be;
    };
    candidate();
    float cn = __shfl_down_sync(0xffffffffu, ce, 1, LPT);
    // (keys with the same high bits may come out in the wrong order)
    if (__any_sync(0xffffffffu, sl < k + 1 && cn > ce)) {
#pragma unroll 1
      for (int pass = 0; pass < 3; ++pass) {
        const int other = pass == 1 ? ((sl + 1) ^ 1) - 1 : sl ^ 1;
        const int from = seg0 + min(max(other, 0), LPT - 1);
        const float co = __shfl_sync(0xffffffffu, ce, from), lo2 = __shfl_sync(0xffffffffu, l, from),
                    bo = __shfl_sync(0xffffffffu, be, from);
        const int eo = __shfl_sync(0xffffffffu, e, from);
        const bool front = other > sl;  // this lane keeps the better of the two
        const bool better = co > ce || (co == ce && eo < e);
        const bool worse = co < ce || (co == ce && eo > e);
        if (other >= 0 && other < LPT && (front ? better : worse)) {
          ce = co;
          l = lo2;
          be = bo;
          e = eo;
        }
      }
      cn = __shfl_down_sync(0xffffffffu, ce, 1, LPT);
    }
    const float ln = __shfl_down_sync(0xffffffffu, l, 1, LPT);
    const float bn = __shfl_down_sync(0xffffffffu, be, 1, LPT);
    const int en = __shfl_down_sync(0xffffffffu, e, 1, LPT);
    const float err = kerr * p1 + 1.2e-7f * fabsf(ce);
    const bool tie = l == ln && be == bn && e < en;
    // (what three passes left out of order could hide near ties of others)
    const bool close = (sl < k && !(ce - cn > err) && !tie) || (sl == k && cn > ce);
    // what is no candidate has to be below the top_k first for certain (below a c of
    // -inf it is: of equal c the keys themselves put the lower id first)
    auto reached = [&]() {
      return last != 0u && ce != -INFINITY && !(ce - rb_value(last | MASK) > err);
    };
    int rank = sl;  // of the lane's candidate
    bool open = false;
    int n = k + 2;
    // (what another token of the warp needs changes nothing here, the order of the
    // weights' sum neither: a token's results do not depend on its neighbours)
    const uint32_t own_lanes = LPT == 32 ? 0xffffffffu : ((1u << (LPT & 31)) - 1u) << seg0;
    const uint32_t mores = __ballot_sync(0xffffffffu, sl < k && reached() && live);
    const bool more = (mores & own_lanes) != 0u;
    if (mores != 0u) {  // as many candidates as lanes
      for (; n < LPT; ++n) round(n);
      if (sl < k && reached()) hard = true;
      if (more) candidate();
    }
    const uint32_t closes = __ballot_sync(0xffffffffu, close && live) | mores;
    if (closes != 0u) {
      // in 64 bits among the candidates
      const double inv = softmax ? inv64() : 1.0;
      const double p64 = rb_score64(l, softmax, mx) * inv;
      const double c64 = l == -INFINITY ? -INFINITY : p64 + be + 0.0;
      const uint64_t mykey = mine != 0u && (more || sl < k + 2) ? rb_key64(c64) : 0;
      uint64_t next = 0;  // the largest key below this lane's, and its p
      const uint64_t pbits = static_cast<uint64_t>(__double_as_longlong(p64));
      uint64_t pnext = 0, peq = 0;  // peq: the largest p among equal c of different p
      rank = 0;
#pragma unroll 1
      for (int j = 0; j < n; ++j) {
        const uint64_t o = __shfl_sync(0xffffffffu, mykey, seg0 + j);
        const int oe = __shfl_sync(0xffffffffu, e, seg0 + j);
        // (p are positive: their bits order as they do, off the slow FP64 unit)
        const uint64_t op = __shfl_sync(0xffffffffu, pbits, seg0 + j);
        rank += (o > mykey || (o == mykey && oe < e)) ? 1 : 0;
        if (o < mykey && o > next) {
          next = o;
          pnext = op;
        }
        if (o == mykey && op != pbits) peq = max(peq, max(op, pbits));
      }
      // All pairs are decided if each candidate is from the next below it, the ones
      // that are not chosen too: gaps and differences of p add up along the order.
      // Equal c of different p are equal by this inverse only, unless both p vanish in c
      // (below half a step of a bias, whatever the inverse).
      if (softmax && mykey > rb_key64(-INFINITY)) {
        if (peq != 0)
          open = static_cast<float>(__longlong_as_double(static_cast<long long>(peq))) >
                 5e-17f * fabsf(static_cast<float>(c64));
        if (next != 0)
          open |= undecided(c64 - rb_value64(next),
                            p64 - __longlong_as_double(static_cast<long long>(pnext)));
      }
      if (mykey == 0) rank = LPT;
      if ((closes & own_lanes) == 0u) {
        rank = sl;
        open = false;
      }
    }
    const uint32_t hards = __ballot_sync(0xffffffffu, (hard || open) && live);
    // ---- weights (as rb_weights) ----
    const bool chosen = rank < k;
    const bool renorm = !softmax || P.renormalize;
    const float top = renorm ? rb_seg_max<LPT>(chosen ? l : -INFINITY) : mx;
    const bool none = top == -INFINITY;  // nothing chosen that is not masked
    float p = softmax ? expf(l - top) : rb_sigmoid_over(l, top);
    if (!chosen || none) p = 0.f;
    float total = renorm ? rb_seg_sum<LPT>(p) : sum;
    if (none) total = 1.0f;
    const uint32_t seg_hard = LPT == 32 ? hards : (hards >> seg0) & ((1u << (LPT & 31)) - 1u);
    if (chosen && live && seg_hard == 0u) {
      out_w[t * k + rank] = p / total * P.scale;
      out_ids[t * k + rank] = e;
    }
    if (hards != 0u) {
#pragma unroll 1
      for (int s = 0; s < TPW; ++s) {
        const uint32_t part = LPT == 32 ? hards : (hards >> (s * LPT)) & ((1u << (LPT & 31)) - 1u);
        if (part == 0u) continue;
        const int64_t tb = t0 + s;
        __syncwarp();
        const int2 id = rb_choose64(logits + tb * E, bias, P, sm);
        rb_weights(logits + tb * E, P, id.x, id.y, out_w + tb * k, out_ids + tb * k);
        __syncwarp();
      }
    }
  }
}

// Gradient with respect to the logits of sum_j gw_j w_j.
// With v_j = w_j / scale and u_j the chosen log scores,
//   renormalised:  v = softmax(u),  du_j = scale v_j (gw_j - sum_i v_i gw_i)
//     softmax: dl = du at the chosen logits (the row's own sum cancels)
//     sigmoid: dl = du sigma(-l)
//   softmax as it is: v_j = p_j,  dl_e = scale (sum_j [id_j = e] gw_j p_e - p_e sum_i gw_i p_i)
//
// Registers hold a token's row: LPT lanes per token (two tokens per warp up to
// 256 experts and 16 items, else one), EPL experts per lane.  The
// row goes out in 16-byte stores with what every entry has (0, or -p_e times
// the dot product), then the lanes of the items store their experts' entries
// over it.
template <int N>
__device__ __forceinline__ void rg_store(float* p, const float (&v)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2) *reinterpret_cast<float2*>(p + i) = make_float2(v[i], v[i + 1]);
  }
}
__device__ __forceinline__ uint32_t rg_pack(float a, float b) {
  __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<uint32_t*>(&v);
}
template <int N>
__device__ __forceinline__ void rg_store(bf16* p, const float (&v)[N]) {
  if constexpr (N % 8 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 8)
      *reinterpret_cast<uint4*>(p + i) =
          make_uint4(rg_pack(v[i], v[i + 1]), rg_pack(v[i + 2], v[i + 3]),
                     rg_pack(v[i + 4], v[i + 5]), rg_pack(v[i + 6], v[i + 7]));
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 2)
      *reinterpret_cast<uint32_t*>(p + i) = rg_pack(v[i], v[i + 1]);
  }
}

template <int EPL, int LPT, typename T>
__global__ void __launch_bounds__(kRbWarps * 32)
    route_backward_kernel(const float* __restrict__ gw, const T* __restrict__ logits,
                          const int32_t* __restrict__ ids, RbParams P, int vec,
                          T* __restrict__ out, int32_t* error_word) {
  pdl_begin();
  const int lane = threadIdx.x & 31, sl = lane % LPT;
  const int64_t warp0 = static_cast<int64_t>(blockIdx.x) * kRbWarps + (threadIdx.x >> 5);
  const int64_t token = warp0 * (32 / LPT) + lane / LPT;
  const bool live = token < P.M;
  const int64_t t = live ? token : P.M - 1;
  const int E = P.E, k = P.top_k;
  // EPL consecutive experts, or every LPT-th where rows are no multiples of them (by
  // the sizes alone: a tensor's alignment must not change the order of its sums)
  const bool apart = E % EPL != 0;
  const int e0 = apart ? sl : sl * EPL, es = apart ? LPT : 1;
  const T* row = logits + t * E;
  // the lane's item
  int id = sl < k ? ids[t * k + sl] : -1;
  if (sl < k && (id < 0 || id >= E)) {
    if (live) record_error(error_word, MOE_ERR_BAD_EXPERT_ID);
    id = -1;
  }
  const float l = id >= 0 ? rb_f32(row[id]) : -INFINITY;
  // (a masked expert's weight is 0 whatever came back for it: its item takes no part.
  // Loaded all the same, together with l: 5.64 us at 16384 x 128, 5.78 after it)
  float g = id >= 0 ? gw[t * k + sl] : 0.f;
  if (l == -INFINITY) g = 0.f;
  float v[EPL];
  float d;            // the item's own part of its expert's entry
  float base = 0.f;   // what the entry has without it
  if (P.method == MOE_ROUTE_SOFTMAX && !P.renormalize) {
    if (vec && e0 < E) {
      rb_load<EPL>(row + e0, v);
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) v[i] = e0 + i * es < E ? rb_f32(row[e0 + i * es]) : -INFINITY;
    }
    float mx = v[0], s = 0.f;
#pragma unroll
    for (int i = 1; i < EPL; ++i) mx = fmaxf(mx, v[i]);
    mx = rb_seg_max<LPT>(mx);
    const bool none = mx == -INFINITY;  // nothing but masked experts (or NaN, which stays)
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      v[i] = none && v[i] == -INFINITY ? 0.f : expf(v[i] - mx);
      s += v[i];
    }
    s = rb_seg_sum<LPT>(s);
    const float inv = s == 0.f ? 0.f : 1.0f / s;
    const float p = l == -INFINITY ? 0.f : expf(l - mx) * inv;
    d = P.scale * p * g;
    const float dot = rb_seg_sum<LPT>(d);
    base = -p * dot;
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = -(v[i] * inv) * dot;
  } else {
    const bool sigmoid = P.method == MOE_ROUTE_SIGMOID;
    const float u = sigmoid ? fminf(l, 0.f) - log1pf(expf(-fabsf(l))) : l;
    const float mx = rb_seg_max<LPT>(u);
    const float e = (id < 0 || mx == -INFINITY) && !(l != l) ? 0.f : expf(u - mx);
    const float s = rb_seg_sum<LPT>(e);
    const float w = e * (s == 0.f ? 0.f : 1.0f / s);
    const float dot = rb_seg_sum<LPT>(w * g);
    d = P.scale * w * (g - dot);
    if (sigmoid) d *= 1.0f / (1.0f + expf(l));
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[i] = 0.f;
  }
  // an expert named twice: its first item's lane adds the others' parts, in order
  const unsigned same =
      __match_any_sync(0xffffffffu, id >= 0 ? id | (lane / LPT) << 16 : -1 - lane);
  if (__any_sync(0xffffffffu, __popc(same) > 1)) {
    float all = 0.f;
    for (int j = 0; j < 32; ++j) {
      const float o = __shfl_sync(0xffffffffu, d, j);
      if ((same >> j) & 1u) all += o;
    }
    d = all;
  }
  T* dst = out + t * E;
  if (live) {
    if (vec) {
      if (e0 < E) rg_store<EPL>(dst + e0, v);
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (e0 + i * es < E) rb_store(dst + e0 + i * es, v[i]);
    }
  }
  __syncwarp();
  if (live && id >= 0 && lane == __ffs(same) - 1) rb_store(dst + id, base + d);
}

// More than 32 items per token: one warp per token, the row in shared memory.
template <typename T>
__global__ void __launch_bounds__(kRbWarps * 32)
    route_backward_wide_kernel(const float* __restrict__ gw, const T* __restrict__ logits,
                          const int32_t* __restrict__ ids, RbParams P, T* __restrict__ out,
                          int32_t* error_word) {
  pdl_begin();
  extern __shared__ float rg_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kRbWarps + warp;
  if (t >= P.M) return;
  const int E = P.E, k = P.top_k;
  const T* row = logits + t * E;
  float* acc = rg_smem + warp * E;
  int id[2];
  float l[2], g[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int j = lane + 32 * h;
    id[h] = j < k ? ids[t * k + j] : -1;
    if (j < k && (id[h] < 0 || id[h] >= E)) {
      record_error(error_word, MOE_ERR_BAD_EXPERT_ID);
      id[h] = -1;
    }
    l[h] = id[h] >= 0 ? rb_f32(row[id[h]]) : -INFINITY;
    g[h] = id[h] >= 0 && l[h] != -INFINITY ? gw[t * k + j] : 0.f;
  }
  float d[2];
  if (P.method == MOE_ROUTE_SOFTMAX && !P.renormalize) {
    float mx = -INFINITY, s = 0.f;
    for (int e = lane; e < E; e += 32) mx = fmaxf(mx, rb_f32(row[e]));
    mx = rb_max(mx);
    for (int e = lane; e < E; e += 32) {
      acc[e] = mx == -INFINITY ? 0.f : expf(rb_f32(row[e]) - mx);
      s += acc[e];
    }
    s = rb_sum(s);
    const float inv = s > 0.f ? P.scale / s : (s == 0.f ? 0.f : s);
    __syncwarp();
#pragma unroll
    for (int h = 0; h < 2; ++h) d[h] = id[h] >= 0 ? g[h] * (acc[id[h]] * inv) : 0.f;
    const float dot = rb_sum(d[0] + d[1]) * (s > 0.f ? 1.0f / s : 0.f);
    __syncwarp();
    for (int e = lane; e < E; e += 32) acc[e] = -acc[e] * dot;
  } else {
    float u[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      u[h] = P.method == MOE_ROUTE_SIGMOID ? fminf(l[h], 0.f) - log1pf(expf(-fabsf(l[h]))) : l[h];
    const float mx = rb_max(fmaxf(u[0], u[1]));
    float v[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      v[h] = (id[h] < 0 || mx == -INFINITY) ? 0.f : expf(u[h] - mx);
    const float s = rb_sum(v[0] + v[1]);
    const float inv = s == 0.f ? 0.f : 1.0f / s;
    v[0] *= inv;
    v[1] *= inv;
    const float dot = rb_sum(v[0] * g[0] + v[1] * g[1]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      d[h] = P.scale * v[h] * (g[h] - dot);
      if (P.method == MOE_ROUTE_SIGMOID) d[h] *= 1.0f / (1.0f + expf(l[h]));
    }
    for (int e = lane; e < E; e += 32) acc[e] = 0.f;
  }
  __syncwarp();
  // item by item, so that an expert named twice gets a sum in a fixed order
  for (int j = 0; j < k; ++j) {
    const int e = __shfl_sync(0xffffffffu, j < 32 ? id[0] : id[1], j & 31);
    const float v = __shfl_sync(0xffffffffu, j < 32 ? d[0] : d[1], j & 31);
    if (e >= 0 && lane == (e & 31)) acc[e] += v;
  }
  for (int e = lane; e < E; e += 32) rb_store(out + t * E + e, acc[e]);
}

// Blocks and shared memory of a launch over the tokens: warps per block so
// that 48 KB hold their 64-bit values.
int rb_warps(const RouteArgs& a) { return a.E + a.group_count <= 1536 ? kRbWarps : kRbWarps / 2; }

template <int EPL, int LPT, typename T>
void launch_fast(const RouteArgs& a, const float* bias, RbParams P, cudaStream_t s) {
  const int warps = rb_warps(a);
  const size_t smem = static_cast<size_t>(warps) * (a.E + a.group_count) * sizeof(uint64_t);
  const int64_t blocks = ceil_div<int64_t>(a.M, warps * (32 / LPT));
  // 16-byte (for few experts narrower) aligned loads of a lane's experts
  const int bytes = EPL * static_cast<int>(sizeof(T)) < 16 ? EPL * static_cast<int>(sizeof(T)) : 16;
  const int vec = a.E % EPL == 0 && (a.E * sizeof(T)) % bytes == 0 &&
                  reinterpret_cast<uintptr_t>(a.logits) % bytes == 0;
  const int gs = P.gs, lpg = gs / EPL;
  while ((2 << P.lpg_log) <= lpg) ++P.lpg_log;
  const bool whole =
      a.E % EPL == 0 && (a.k_group == a.group_count ||
                         (gs == lpg * EPL && (lpg & (lpg - 1)) == 0));
  // (a bound of 16 blocks for each of 152 SMs, of which 6 to 8 are resident at 64 to 80
  // registers: warps of larger calls go through several tokens, their biases loaded once)
  launch_kernel(whole ? route_biased_kernel<EPL, LPT, true, T>
                      : route_biased_kernel<EPL, LPT, false, T>,
                static_cast<unsigned>(std::min<int64_t>(blocks, 152 * 16)), warps * 32, smem, s,
                static_cast<const T*>(a.logits), bias, P, vec, a.weights, a.ids);
}

template <typename T>
void launch_biased(const RouteArgs& a, const float* bias, cudaStream_t s) {
  const RbParams P{a.M, a.E, a.top_k, a.method, a.renormalize, a.k_group, a.group_count,
                   a.group_select_mode, a.scale,
                   a.E / a.group_count, ceil_div(1 << 20, a.E / a.group_count), 0};
  const bool grouped = a.k_group < a.group_count;
  // A candidate per lane (two beyond top_k), a group per lane.  Half a warp per token
  // halves the instructions, a whole one shortens a token's chain and, from 65 experts
  // on, wins up to 4096 tokens (half, whole; 256 experts: 1 token 3.3, 2.9 us; 4096: 8.4,
  // 8.2; 16384: 15.1, 18.0; 128: 2.7, 2.2; 5.7, 5.4; 10.5, 11.0; 64: 2.2, 2.2; 4.9, 5.5).
  const bool whole_warp = a.E > 64 && a.M <= 4096;
  if (!whole_warp && a.E <= 256 && a.top_k <= 14 && (!grouped || a.group_count <= 16)) {
    if (a.E <= 32) return launch_fast<2, 16, T>(a, bias, P, s);
    if (a.E <= 64) return launch_fast<4, 16, T>(a, bias, P, s);
    if (a.E <= 128) return launch_fast<8, 16, T>(a, bias, P, s);
    return launch_fast<16, 16, T>(a, bias, P, s);
  }
  if (a.top_k <= 30 && (!grouped || a.group_count <= 32)) {
    if (a.E <= 128) return launch_fast<4, 32, T>(a, bias, P, s);
    if (a.E <= 256) return launch_fast<8, 32, T>(a, bias, P, s);
    if (a.E <= 512) return launch_fast<16, 32, T>(a, bias, P, s);
    return launch_fast<32, 32, T>(a, bias, P, s);
  }
  const int warps = rb_warps(a);
  launch_kernel(route_biased_exact_kernel<T>, static_cast<unsigned>(ceil_div<int64_t>(a.M, warps)),
                warps * 32, static_cast<size_t>(warps) * (a.E + a.group_count) * sizeof(uint64_t), s,
                static_cast<const T*>(a.logits), bias, P, a.weights, a.ids);
}

template <int EPL, int LPT, typename T>
void launch_rg(const RouteBackwardArgs& a, const RbParams& P, cudaStream_t s) {
  const int bytes = EPL * static_cast<int>(sizeof(T)) < 16 ? EPL * static_cast<int>(sizeof(T)) : 16;
  const int vec = a.E % EPL == 0 && (a.E * sizeof(T)) % bytes == 0 &&
                  reinterpret_cast<uintptr_t>(a.logits) % bytes == 0 &&
                  reinterpret_cast<uintptr_t>(a.grad_logits) % bytes == 0;
  launch_kernel(route_backward_kernel<EPL, LPT, T>,
                static_cast<unsigned>(ceil_div<int64_t>(a.M, kRbWarps * (32 / LPT))), kRbWarps * 32,
                0, s, a.grad_weights, static_cast<const T*>(a.logits), a.ids, P, vec,
                static_cast<T*>(a.grad_logits), a.error_word);
}

template <typename T>
void launch_backward(const RouteBackwardArgs& a, cudaStream_t s) {
  RbParams P{};
  P.M = a.M;
  P.E = a.E;
  P.top_k = a.top_k;
  P.method = a.method;
  P.renormalize = a.renormalize;
  P.scale = a.scale;
  if (a.top_k <= 16 && a.E <= 256) {
    if (a.E <= 32) return launch_rg<2, 16, T>(a, P, s);
    if (a.E <= 128) return launch_rg<8, 16, T>(a, P, s);
    return launch_rg<16, 16, T>(a, P, s);
  }
  if (a.top_k <= 32) {
    if (a.E <= 256) return launch_rg<8, 32, T>(a, P, s);
    if (a.E <= 512) return launch_rg<16, 32, T>(a, P, s);
    return launch_rg<32, 32, T>(a, P, s);
  }
  launch_kernel(route_backward_wide_kernel<T>,
                static_cast<unsigned>(ceil_div<int64_t>(a.M, kRbWarps)), kRbWarps * 32,
                static_cast<size_t>(kRbWarps) * a.E * sizeof(float), s, a.grad_weights,
                static_cast<const T*>(a.logits), a.ids, P, static_cast<T*>(a.grad_logits),
                a.error_word);
}

}  // namespace

moe_status_t launch_route_biased(const RouteArgs& a, const float* bias, cudaStream_t s) {
  prof_before("route_biased", s);
  if (a.logits_bf16)
    launch_biased<bf16>(a, bias, s);
  else
    launch_biased<float>(a, bias, s);
  prof_after("route_biased", s);
  return check_launch("route_biased");
}

moe_status_t launch_route_backward(const RouteBackwardArgs& a, cudaStream_t s) {
  prof_before("route_backward", s);
  if (a.logits_bf16)
    launch_backward<bf16>(a, s);
  else
    launch_backward<float>(a, s);
  prof_after("route_backward", s);
  return check_launch("route_backward");
}

}  // namespace gbmoe
