// gdn_linear_tc32.cuh -- products with fp32 precision on the tensor cores, for the kernels of gdn_linear_tc32.cu and
// gdn_linear_bwd.cu.
//
// An fp32 value is the sum of three bf16 values to its last bit or so (8 bits each); a product of two such sums keeps
// the six of its nine terms that reach 2^-24 of it, each exact in the fp32 accumulators (a bf16 input is its own first
// term).  Six bf16 products cost a sixth of 1.89 PFLOP/s, against 74 TFLOP/s of fp32 FMAs.  The accumulators drop bits
// that small products add to large sums (an output summed over 128 was off by 6e-7 instead of 1.5e-7): the smaller
// products come first, or, where a sum goes on from tile to tile, have an accumulator of their own.
//
// Tiles are rows of 64 bf16 (128 bytes, swizzled) as the tensors have them, whatever their part in a product; those of
// 64 rows or columns are read as 128 where they stand in A, and the lanes behind them are ignored.
#pragma once

#include "gdn_linear_tc.cuh"

namespace gdn {
namespace lin {

template <typename T>
constexpr int kTerms = sizeof(T) == 4 ? 3 : 1;

// N threads: ROWS x COLS values, four neighbours a thread at a time -> `TERMS` tiles of 64-column atom columns, row r
// times w[r]; zeros past `rows`.
template <int ROWS, int COLS, int N, typename T>
__device__ __forceinline__ void fetch(float4 (&x)[ROWS * COLS / 4 / N], const T* src, int64_t ld, int rows) {
#pragma unroll
  for (int u = 0; u < ROWS * COLS / 4 / N; ++u) {
    const int quad = threadIdx.x + u * N, r = quad / (COLS / 4), c = quad % (COLS / 4) * 4;
    x[u] = r < rows ? load4(src + r * ld + c) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
}
template <int ROWS, int COLS, int TERMS, int N>
__device__ __forceinline__ void place(uint8_t* sm, const float4 (&x)[ROWS * COLS / 4 / N], const float* w) {
  constexpr uint32_t tile = ROWS * COLS * 2;
#pragma unroll
  for (int u = 0; u < ROWS * COLS / 4 / N; ++u) {
    const int quad = threadIdx.x + u * N, r = quad / (COLS / 4), c = quad % (COLS / 4) * 4;
    float4 y = x[u];
    if (w) {
      const float f = w[r];
      y.x *= f, y.y *= f, y.z *= f, y.w *= f;
    }
    uint8_t* to = sm + (c >> 6) * (ROWS * 128) + sw128_chunk(r, (c & 63) >> 3) + (c & 4) * 2;
    if (TERMS == 1) {
      *reinterpret_cast<uint2*>(to) = make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
    } else {
      uint32_t w0[2], w1[2], w2[2];
      split3(y, w0, w1, w2);
      *reinterpret_cast<uint2*>(to) = make_uint2(w0[0], w0[1]);
      *reinterpret_cast<uint2*>(to + tile) = make_uint2(w1[0], w1[1]);
      *reinterpret_cast<uint2*>(to + 2 * tile) = make_uint2(w2[0], w2[1]);
    }
  }
}

// The products of A's and B's terms, the smallest first: f(term of A, term of B, 0 for the first one of all).
template <int A, int B, typename F>
__device__ __forceinline__ void products(F f) {
  uint32_t more = 0;
#pragma unroll
  for (int sum = 2; sum >= 0; --sum)
#pragma unroll
    for (int a = 2; a >= 0; --a)
      if (a < A && a <= sum && sum - a < B) f(a, sum - a, more), more = 1;
}

// mbar_wait with the whole warp's verdict (TMEM loads want whole warps).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int32_t* status) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, status));
}

}  // namespace lin
}  // namespace gdn
