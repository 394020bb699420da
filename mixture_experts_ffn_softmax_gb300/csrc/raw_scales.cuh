// Which bytes of MX FP4 scales a tile's bulk copies take where rows of scales are not whole
// 16 bytes (grouped.cu).  Host code as well as device code: the ranges are tested without a GPU.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define GBMOE_HOST_DEVICE __host__ __device__
#else
#define GBMOE_HOST_DEVICE
#endif

namespace gbmoe {

// `bulk` bytes from `begin` on, both multiples of 16, then the bytes up to `end` one by one.
struct RawSpan {
  int64_t begin, end;
  uint32_t bulk;
};

// The span of bytes [from, to) of a tensor of `total` bytes: from a multiple of 16 bytes on
// and to one, but not past the tensor.  Nothing where from == to, which may lie behind the tensor.
GBMOE_HOST_DEVICE inline RawSpan raw_span(int64_t from, int64_t to, int64_t total) {
  if (to <= from) return RawSpan{from, from, 0u};
  const int64_t a = from & ~int64_t(15), past = (to + 15) & ~int64_t(15), last = total & ~int64_t(15);
  const int64_t z = past < last ? past : last;
  return RawSpan{a, to, z > a ? static_cast<uint32_t>(z - a) : 0u};
}

// Scales of expert e's columns n.. of the weight [E, N, K / 32], KG = K / 32 a row: a CTA's
// 128, as far as they are there (a tile's second CTA may have none).
GBMOE_HOST_DEVICE inline RawSpan weight_scale_span(int E, int N, int KG, int e, int n) {
  const int64_t row = static_cast<int64_t>(e) * N + n;
  const int rows = N - n < 128 ? (N - n > 0 ? N - n : 0) : 128;
  return raw_span(row * KG, (row + rows) * KG, static_cast<int64_t>(E) * N * KG);
}

// Scales of the T rows from c0 on, of R.
GBMOE_HOST_DEVICE inline RawSpan row_scale_span(int64_t R, int KG, int64_t c0, int T) {
  return raw_span(c0 * KG, (c0 + T < R ? c0 + T : R) * KG, R * KG);
}

}  // namespace gbmoe
