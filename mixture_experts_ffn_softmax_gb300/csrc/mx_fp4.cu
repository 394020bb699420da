// MX FP4 (OCP Microscaling Formats v1.0): E2M1 elements, one power-of-two
// scale (UE8M0) per block of 32 along the row.
//
//   scale = 2^(floor(log2 max|z|) - 2), its exponent stored with a bias of 127 and
//           held at 0 from below (2^-127);
//   code  = nearest E2M1 value (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives) of
//           z / scale, ties to the even code, magnitudes above 6 at 6.
// 2 is E2M1's largest exponent.  z / scale is exact, so that a code is one rounding of z.
#include <cuda_fp4.h>

#include <algorithm>

#include "common.cuh"
#include "dense.cuh"

namespace gbmoe {
namespace {

constexpr int kQ4Threads = 256;
constexpr int quant4_blocks(bool swiglu) { return swiglu ? 3 : 4; }  // resident blocks of an SM

// Four lanes per block of 32, 8 columns per lane.  Rows are whole blocks, so that x, the
// codes and the scales are taken as flat arrays; only gate and up are apart by row.  Bound:
// HBM for a tensor (8192 x 7168 with the values 43.7 us, 6.1 TB/s), issue slots for SiLU(gate) *
// up, whose next loads are in flight while it works (8191 x 2048 with the values: 20.6 us, 22.0
// without; a tensor 46.9 with them ahead and three blocks, 43.7 in four without).
template <bool SWIGLU>
__global__ void __launch_bounds__(kQ4Threads, quant4_blocks(SWIGLU))
    quant_mx_fp4_kernel(const bf16* __restrict__ x, int64_t M, int K, uint8_t* __restrict__ q4,
                        uint8_t* __restrict__ scale, bf16* __restrict__ values) {
  pdl_begin();
  constexpr int U = SWIGLU ? 2 : 4;  // units in flight
  const int per = K / 8;
  const int64_t total = M * per;  // a multiple of 4
  const int64_t threads = static_cast<int64_t>(gridDim.x) * kQ4Threads;
  const int64_t first = static_cast<int64_t>(blockIdx.x) * kQ4Threads + threadIdx.x;
  int64_t row = 0, step_row = 0;
  int unit = 0, step_unit = 0;
  if constexpr (SWIGLU) {  // stepped without a division in the loop
    row = first / per;
    unit = static_cast<int>(first - row * per);
    step_row = threads / per;
    step_unit = static_cast<int>(threads - step_row * per);
  }
  uint4 na[U], nb[SWIGLU ? U : 1];
  auto load = [&](int64_t base) {  // (SWIGLU: of the units that follow those loaded last)
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t f = base + (threadIdx.x & 31) + i * threads;
      const bool in = f < total;
      if constexpr (SWIGLU) {
        const bf16* src = x + row * 2 * K + unit * 8;
        na[i] = in ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0, 0, 0, 0);
        nb[i] = in ? __ldg(reinterpret_cast<const uint4*>(src + K)) : make_uint4(0, 0, 0, 0);
        row += step_row;
        unit += step_unit;
        if (unit >= per) {
          unit -= per;
          ++row;
        }
      } else {
        na[i] = in ? __ldg(reinterpret_cast<const uint4*>(x + f * 8)) : make_uint4(0, 0, 0, 0);
      }
    }
  };
  const int64_t base0 = first - (threadIdx.x & 31);
  if constexpr (SWIGLU) load(base0);
  // (whole warps stay in the loop for the shuffles)
  for (int64_t base = base0; base < total; base += U * threads) {
    uint4 a[U], b[SWIGLU ? U : 1];
    if constexpr (!SWIGLU) load(base);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      a[i] = na[i];
      if constexpr (SWIGLU) b[i] = nb[i];
    }
    if constexpr (SWIGLU) load(base + U * threads);
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int64_t f = base + (threadIdx.x & 31) + i * threads;
      float z[8];
      unpack8(a[i], z);
      uint32_t top;  // max |z|, by its bits (they order as the values, NaN on top)
      if constexpr (SWIGLU) {
        float u[8];
        unpack8(b[i], u);
        swiglu8(z, u);
        top = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(z[j]) & 0x7fffffffu);
      } else {
        uint32_t t = __vmaxu2(a[i].x & 0x7fff7fffu, a[i].y & 0x7fff7fffu);
        t = __vmaxu2(t, a[i].z & 0x7fff7fffu);
        t = __vmaxu2(t, a[i].w & 0x7fff7fffu);
        top = max(t << 16, t & 0xffff0000u);
      }
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const uint32_t e = top >> 23;  // floor(log2 max) + 127; 255: an infinity or NaN
      const uint32_t s = e == 255u ? 255u : e > 2u ? e - 2u : 0u;
      // 1 / scale = 2^(127 - s), normal for s up to 252
      const float inv = e == 255u ? 0.f : __uint_as_float((254u - s) << 23);
      uint32_t codes = 0;
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        float2 v = make_float2(z[j] * inv, z[j + 1] * inv);
        if (e == 255u) v = make_float2(0.f, 0.f);
        codes |= static_cast<uint32_t>(
                     __nv_cvt_float2_to_fp4x2(v, __NV_E2M1, cudaRoundNearest))
                 << (4 * j);
      }
      if (f < total) {
        *reinterpret_cast<uint32_t*>(q4 + f * 4) = codes;
        if ((threadIdx.x & 3) == 0) scale[f / 4] = static_cast<uint8_t>(s);
        if (values != nullptr) {
          // 2^(s - 127): subnormal for s = 0, NaN for 255
          const float sc = __uint_as_float(s == 255u ? 0x7fffffffu : s == 0u ? 0x00400000u : s << 23);
          float v[8];
#pragma unroll
          for (int j = 0; j < 8; j += 2) {
            const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(
                static_cast<__nv_fp4x2_storage_t>(codes >> (4 * j) & 0xffu), __NV_E2M1);
            const float2 p = __half22float2(__half2(h));
            v[j] = p.x * sc;
            v[j + 1] = p.y * sc;
          }
          *reinterpret_cast<uint4*>(values + f * 8) = make_uint4(
              pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
        }
      }
    }
  }
}

}  // namespace

moe_status_t launch_quant_mx_fp4(const QuantMxFp4Args& a, cudaStream_t s) {
  const int64_t units = a.M * (a.K / 8);
  const unsigned grid = static_cast<unsigned>(
      std::min<int64_t>(ceil_div<int64_t>(units, kQ4Threads), int64_t(a.num_sms) * quant4_blocks(a.swiglu)));
  prof_before("quant_mx_fp4", s);
  launch_kernel(a.swiglu ? quant_mx_fp4_kernel<true> : quant_mx_fp4_kernel<false>, grid, kQ4Threads,
                0, s, a.x, a.M, a.K, a.q4, a.scale, a.values);
  prof_after("quant_mx_fp4", s);
  return check_launch("quant_mx_fp4");
}

}  // namespace gbmoe
