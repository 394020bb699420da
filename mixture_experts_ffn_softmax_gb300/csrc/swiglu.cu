// SiLU(gate) * up of each routed row with the row's routing weight, and its
// gradient: what stands between the two products of the experts in training.
//
//   z[r, i] = w[r] SiLU(g) u,   SiLU(g) = g sig(g),  sig(g) = 1 / (1 + e^-g)
//   dg = w dz u sig(g) (1 + g (1 - sig(g))),  du = w dz SiLU(g)
//   dw[r] = sum_i dz[r, i] SiLU(g) u
// With the weight on the second product's input instead of its output (the
// same layer: y = sum_j w_j z_j W2), dw comes from dz = dy W2^T, and no expert's
// output has to be kept for it.
#include "common.cuh"
#include "dense.cuh"

namespace gbmoe {
namespace {

constexpr int kSwThreads = 256;

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}

// W warps per row, eight columns per lane and step, for both directions (a warp up to 2048
// columns, else a block).  Bound: HBM (backward: 131064 x 768 in 144 us, 7.0 TB/s; forward
// in 89 us, 6.8).  Blocks of a few rows each, not resident ones stepping through the tensor: those
// took 111 us for the forward's 131064 x 768.
template <int W>
__global__ void __launch_bounds__(kSwThreads)
    swiglu_kernel(const bf16* __restrict__ gate_up, const float* __restrict__ weights, int64_t R,
                  int I, bf16* __restrict__ z) {
  pdl_begin();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kSwThreads / 32 / W) + warp / W;
  if (row >= R) return;
  const float w = weights != nullptr ? __ldg(weights + row) : 1.0f;
  const bf16* src = gate_up + row * 2 * I;
  for (int c = ((warp % W) * 32 + lane) * 8; c < I; c += W * 256) {
    float g[8], u[8];
    unpack8(__ldg(reinterpret_cast<const uint4*>(src + c)), g);
    unpack8(__ldg(reinterpret_cast<const uint4*>(src + I + c)), u);
    swiglu8(g, u);
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] *= w;
    *reinterpret_cast<uint4*>(z + row * I + c) = pack8(g);
  }
}

// The gradient's eight columns: dz, gate and up in, dgate and dup (times w)
// out; returns sum dz SiLU(g) u.
__device__ __forceinline__ float swiglu_grad8(const float (&dz)[8], float (&g)[8], float (&u)[8],
                                              float w) {
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(g[j]));
  float s[8];
  if (top < kFastGate) {
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
      uint64_t r;
      const uint64_t nden = neg_one_plus_exp2(pair_of(g[j], g[j + 1]), r);
      const float2 v = unpair(div_fixed2(pair_of(1.0f, 1.0f), nden, r));
      s[j] = v.x;
      s[j + 1] = v.y;
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) s[j] = 1.0f / (1.0f + expf(-g[j]));
  }
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float silu = g[j] * s[j];
    const float d = dz[j] * w;
    sum = fmaf(dz[j] * silu, u[j], sum);
    g[j] = d * u[j] * (s[j] * fmaf(g[j], 1.0f - s[j], 1.0f));
    u[j] = d * silu;
  }
  return sum;
}

// d_gate_up may be gate_up: a thread reads its columns before it
// writes them, and no other thread reads them.
template <int W>
__global__ void __launch_bounds__(kSwThreads)
    swiglu_backward_kernel(const bf16* __restrict__ dz, const bf16* gate_up,
                           const float* __restrict__ weights, int64_t R, int I, bf16* d_gate_up,
                           float* __restrict__ d_weights) {
  pdl_begin();
  constexpr int ROWS = kSwThreads / 32 / W;  // of a block
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * ROWS + warp / W;
  float sum = 0.f;
  if (row < R) {
    const float w = weights != nullptr ? __ldg(weights + row) : 1.0f;
    const bf16* src = gate_up + row * 2 * I;
    bf16* dst = d_gate_up + row * 2 * I;
    for (int c = ((warp % W) * 32 + lane) * 8; c < I; c += W * 256) {
      float d[8], g[8], u[8];
      unpack8(__ldg(reinterpret_cast<const uint4*>(dz + row * I + c)), d);
      unpack8(*reinterpret_cast<const uint4*>(src + c), g);
      unpack8(*reinterpret_cast<const uint4*>(src + I + c), u);
      sum += swiglu_grad8(d, g, u, w);
      *reinterpret_cast<uint4*>(dst + c) = pack8(g);
      *reinterpret_cast<uint4*>(dst + I + c) = pack8(u);
    }
  }
  if (d_weights == nullptr) return;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  if constexpr (W == 1) {
    if (lane == 0 && row < R) d_weights[row] = sum;
  } else {
    __shared__ float parts[kSwThreads / 32];
    if (lane == 0) parts[warp] = sum;
    __syncthreads();
    if (lane == 0 && warp % W == 0 && row < R) {
      float t = 0.f;
#pragma unroll
      for (int i = 0; i < W; ++i) t += parts[warp + i];
      d_weights[row] = t;
    }
  }
}

}  // namespace

moe_status_t launch_swiglu(const SwigluArgs& a, cudaStream_t s) {
  auto go = [&](auto kernel, int rows) {
    launch_kernel(kernel, static_cast<unsigned>(ceil_div<int64_t>(a.R, rows)), kSwThreads, 0, s,
                  a.gate_up, a.weights, a.R, a.I, a.z);
  };
  prof_before("swiglu", s);
  if (a.I <= 2048)
    go(swiglu_kernel<1>, 8);
  else
    go(swiglu_kernel<8>, 1);
  prof_after("swiglu", s);
  return check_launch("swiglu");
}

moe_status_t launch_swiglu_backward(const SwigluBackwardArgs& a, cudaStream_t s) {
  auto go = [&](auto kernel, int rows) {
    launch_kernel(kernel, static_cast<unsigned>(ceil_div<int64_t>(a.R, rows)), kSwThreads, 0, s, a.dz,
                  a.gate_up, a.weights, a.R, a.I, a.d_gate_up, a.d_weights);
  };
  prof_before("swiglu_backward", s);
  if (a.I <= 2048)
    go(swiglu_backward_kernel<1>, 8);
  else
    go(swiglu_backward_kernel<8>, 1);
  prof_after("swiglu_backward", s);
  return check_launch("swiglu_backward");
}

}  // namespace gbmoe
