// Routing with a per-expert bias for load balance, and the gradient of the
// routing weights.
//
// Scores p (softmax over the experts or sigmoid) as in moe_route; the choice
// of experts is by c_e = p_e + b_e, the weights are the chosen experts' p.
// c is compared as in 64-bit arithmetic: two fp32 values of c closer than
// their rounding say nothing about the order of the exact ones, and the ids
// are integers, right or wrong.
#include <cfloat>

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
};

// Best (value, index) over the warp, ties to the lower index.
__device__ __forceinline__ void rb_warp_best(double& v, int& i) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double v2 = __shfl_xor_sync(0xffffffffu, v, o);
    const int i2 = __shfl_xor_sync(0xffffffffu, i, o);
    if (v2 > v || (v2 == v && i2 < i)) {
      v = v2;
      i = i2;
    }
  }
}

// One token's choice in 64 bits, by one warp.  c: E + group_count doubles of
// shared memory.  Lane j receives chosen experts j and j + 32.  A candidate
// that is out (its group not kept, or chosen) is marked by NaN; a masked
// expert (logit -inf) or a NaN score has c = -inf and comes last.
template <typename T>
__device__ void rb_choose64(const T* row, const float* bias, const RbParams& P, double* c, int& id0,
                            int& id1) {
  const int lane = threadIdx.x & 31;
  const int E = P.E;
  double m = 0.0, inv = 1.0;
  if (P.method == MOE_ROUTE_SOFTMAX) {
    float mf = -INFINITY;
    for (int e = lane; e < E; e += 32) mf = fmaxf(mf, rb_f32(row[e]));
    m = rb_max(mf);
    double s = 0.0;
    for (int e = lane; e < E; e += 32) s += exp(static_cast<double>(rb_f32(row[e])) - m);
    inv = 1.0 / rb_sum(s);
  }
  for (int e = lane; e < E; e += 32) {
    const double l = rb_f32(row[e]);
    const double p = P.method == MOE_ROUTE_SOFTMAX ? exp(l - m) * inv : 1.0 / (1.0 + exp(-l));
    const double v = p + static_cast<double>(bias[e]);
    c[e] = (l == -INFINITY || !(v == v)) ? -INFINITY : v;
  }
  __syncwarp();
  if (P.group_count > 1) {
    const int G = P.group_count, gs = E / G;
    double* gk = c + E;
    for (int g = lane; g < G; g += 32) {
      double b1 = -INFINITY, b2 = -INFINITY;
      for (int j = 0; j < gs; ++j) {
        const double v = c[g * gs + j];
        if (v > b1) {
          b2 = b1;
          b1 = v;
        } else if (v > b2) {
          b2 = v;
        }
      }
      gk[g] = P.group_select_mode == 0 ? b1 : b1 + b2;
    }
    __syncwarp();
    // the k_group best groups leave gk (NaN); what is left there is dropped
    for (int r = 0; r < P.k_group; ++r) {
      double v = -INFINITY;
      int i = 0x7fffffff;
      for (int g = lane; g < G; g += 32)
        if (gk[g] > v || (gk[g] == v && g < i)) {
          v = gk[g];
          i = g;
        }
      rb_warp_best(v, i);
      if (lane == 0) gk[i] = NAN;
      __syncwarp();
    }
    for (int e = lane; e < E; e += 32)
      if (gk[e / gs] == gk[e / gs]) c[e] = NAN;
    __syncwarp();
  }
  for (int j = 0; j < P.top_k; ++j) {
    double v = -INFINITY;
    int i = 0x7fffffff;
    for (int e = lane; e < E; e += 32)
      if (c[e] > v || (c[e] == v && e < i)) {
        v = c[e];
        i = e;
      }
    rb_warp_best(v, i);
    if (lane == 0) c[i] = NAN;
    if (lane == (j & 31)) (j < 32 ? id0 : id1) = i;
    __syncwarp();
  }
}

// Weights of the chosen experts (lane j: chosen j and j + 32), in fp32.
// Ratios of the chosen scores come from the logits' differences where the
// scores themselves would underflow; a masked expert's weight is 0, and a
// token with nothing but masked experts has weights of 0.
// softmax: mx the row's largest logit and sum that of exp(l - mx) over it
// (NaN where the row holds a NaN or +inf).
template <typename T>
__device__ __forceinline__ void rb_weights(const T* row, const RbParams& P, int id0, int id1,
                                           float mx, float sum, float* out_w, int32_t* out_ids) {
  const int lane = threadIdx.x & 31;
  const bool h0 = lane < P.top_k, h1 = lane + 32 < P.top_k;
  const float l0 = h0 ? rb_f32(row[id0]) : -INFINITY, l1 = h1 ? rb_f32(row[id1]) : -INFINITY;
  const bool masked = __all_sync(0xffffffffu, l0 == -INFINITY && l1 == -INFINITY);
  const bool bad = P.method == MOE_ROUTE_SOFTMAX && sum != sum;
  const bool renorm = P.method == MOE_ROUTE_SIGMOID || P.renormalize;
  if (renorm) mx = rb_max(fmaxf(l0, l1));
  float p0, p1;
  // sigmoid below -60 is exp to fp32 precision
  if (P.method == MOE_ROUTE_SIGMOID && mx >= -60.f) {
    p0 = 1.0f / (1.0f + expf(-l0));
    p1 = 1.0f / (1.0f + expf(-l1));
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

template <typename T>
__global__ void __launch_bounds__(kRbWarps * 32)
    route_biased_kernel(const T* __restrict__ logits, const float* __restrict__ bias, RbParams P,
                        float* __restrict__ out_w, int32_t* __restrict__ out_ids) {
  pdl_begin();
  extern __shared__ double rb_smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (blockDim.x >> 5) + warp;
  if (t >= P.M) return;
  const T* row = logits + t * P.E;
  int id0 = 0, id1 = 0;
  rb_choose64(row, bias, P, rb_smem + warp * (P.E + P.group_count), id0, id1);
  float mx = -INFINITY, sum = 0.f;
  if (P.method == MOE_ROUTE_SOFTMAX) {
    for (int e = lane; e < P.E; e += 32) mx = fmaxf(mx, rb_f32(row[e]));
    mx = rb_max(mx);
    for (int e = lane; e < P.E; e += 32) sum += expf(rb_f32(row[e]) - mx);
    sum = rb_sum(sum);
  }
  rb_weights(row, P, id0, id1, mx, sum, out_w + t * P.top_k, out_ids + t * P.top_k);
}

// Gradient with respect to the logits of sum_j gw_j w_j, one warp per token.
// With v_j = w_j / scale and u_j the chosen log scores,
//   renormalised:  v = softmax(u),  du_j = scale v_j (gw_j - sum_i v_i gw_i)
//     softmax: dl = du at the chosen logits (the row's own sum cancels)
//     sigmoid: dl = du sigma(-l)
//   softmax as it is: v_j = p_j,  dl_e = scale (sum_j [id_j = e] gw_j p_e - p_e sum_i gw_i p_i)
template <typename T>
__global__ void __launch_bounds__(kRbWarps * 32)
    route_backward_kernel(const float* __restrict__ gw, const T* __restrict__ logits,
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
    g[h] = id[h] >= 0 ? gw[t * k + j] : 0.f;
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

}  // namespace

moe_status_t launch_route_biased(const RouteArgs& a, const float* bias, cudaStream_t s) {
  // 48 KB of shared memory hold the four warps' values up to 1536 of them each
  const int warps = a.E + a.group_count <= 1536 ? kRbWarps : kRbWarps / 2;
  const int64_t blocks = ceil_div<int64_t>(a.M, warps);
  const RbParams P{a.M, a.E, a.top_k, a.method, a.renormalize, a.k_group, a.group_count,
                   a.group_select_mode, a.scale};
  const size_t smem = static_cast<size_t>(warps) * (a.E + a.group_count) * sizeof(double);
  prof_before("route_biased", s);
  if (a.logits_bf16)
    launch_kernel(route_biased_kernel<bf16>, static_cast<unsigned>(blocks), warps * 32, smem, s,
                  static_cast<const bf16*>(a.logits), bias, P, a.weights, a.ids);
  else
    launch_kernel(route_biased_kernel<float>, static_cast<unsigned>(blocks), warps * 32, smem, s,
                  static_cast<const float*>(a.logits), bias, P, a.weights, a.ids);
  prof_after("route_biased", s);
  return check_launch("route_biased");
}

moe_status_t launch_route_backward(const RouteBackwardArgs& a, cudaStream_t s) {
  const int64_t blocks = ceil_div<int64_t>(a.M, kRbWarps);
  RbParams P{};
  P.M = a.M;
  P.E = a.E;
  P.top_k = a.top_k;
  P.method = a.method;
  P.renormalize = a.renormalize;
  P.scale = a.scale;
  const size_t smem = static_cast<size_t>(kRbWarps) * a.E * sizeof(float);
  prof_before("route_backward", s);
  if (a.logits_bf16)
    launch_kernel(route_backward_kernel<bf16>, static_cast<unsigned>(blocks), kRbWarps * 32, smem, s,
                  a.grad_weights, static_cast<const bf16*>(a.logits), a.ids, P,
                  static_cast<bf16*>(a.grad_logits), a.error_word);
  else
    launch_kernel(route_backward_kernel<float>, static_cast<unsigned>(blocks), kRbWarps * 32, smem,
                  s, a.grad_weights, static_cast<const float*>(a.logits), a.ids, P,
                  static_cast<float*>(a.grad_logits), a.error_word);
  prof_after("route_backward", s);
  return check_launch("route_backward");
}

}  // namespace gbmoe
