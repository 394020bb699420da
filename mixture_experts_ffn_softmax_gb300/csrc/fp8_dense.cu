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
                      a.out_f32};
  const dim3 grid(static_cast<unsigned>(ceil_div<int64_t>(a.M, 64)),
                  static_cast<unsigned>(ceil_div(a.N, 64)));
  prof_before("matmul_fp8", s);
  launch_kernel(dense_fp8_simt_kernel, grid, 256, 0, s, P);
  prof_after("matmul_fp8", s);
  return check_launch("matmul_fp8");
}

}  // namespace gbmoe
