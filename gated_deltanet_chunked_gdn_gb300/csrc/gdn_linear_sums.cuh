// gdn_linear_sums.cuh -- sums along a sequence of what its chunks (or segments) add to the state, and over the value
// heads of a q/k head.
#pragma once

#include <string.h>

#include "gdn_linear.cuh"

namespace gdn {
namespace lin {

// Head dims and row strides of a problem.
struct Shape {
  int Hqk, Hv, K, V, g_per_head;
  int64_t ldq, ldk, ldv;
};

inline Shape shape_of(const gdn_linear_problem& p) {
  return {p.Hqk, p.Hv, p.K, p.V, p.g_per_head, p.ld_q, p.ld_k, p.ld_v};
}

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 x = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(x.x << 16), __uint_as_float(x.x & 0xffff0000u), __uint_as_float(x.y << 16),
                     __uint_as_float(x.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float* p, const float (&v)[4]) {
  *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store4(__nv_bfloat16* p, const float (&v)[4]) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2*>(p) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// A sum along every sequence (sums_kernel, gdn_linear.cu).
struct Sum {
  const float* init;
  float* S;
  float* fin;
  const int32_t* idx;
  int slots;
  bool rev;
};

// What a chunk adds to the state behind it, sum_j e^{b_last - b_j} x_j y_j^T (x = k, y = v), or, for the adjoint, to
// the one before it, factor sum_i e^{b_i} x_i y_i^T (x = q, y = do), and its whole decay; the outputs of every chunk
// from the state before it (gdn_linear_tc32.cu).
template <typename T>
struct Side {
  const T *x, *y;
  int64_t ldx, ldy;
  float factor;
  float* S;
  bool adj;
};
// One launch for the states, or for them and the adjoint's (sides 1 or 2).
template <typename T>
gdn_status launch_states(const Shape& d, const Side<T>& first, const Side<T>& second, int sides, const float* g,
                         const Pieces& pc, int most, Two* total, int32_t* status, cudaStream_t s);
gdn_status launch_outputs(const Shape& d, const float* q, const float* k, const float* v, const float* g,
                          const Pieces& pc, int most, float scale, const float* S0, float* o, int32_t* status,
                          cudaStream_t s);

// Final states (or a pool's rows by idx), or, with rev, the adjoints before the sequences, go to fin.
gdn_status launch_sums(const Shape& d, const Pieces& pc, int N, const Two* total, const Sum& first, const Sum& second,
                       int sides, cudaStream_t s);
inline gdn_status launch_sums(const Shape& d, const Pieces& pc, int N, const Two* total, const Sum& one,
                              cudaStream_t s) {
  return launch_sums(d, pc, N, total, one, one, 1, s);
}

// dst[row][hq][:] = sum over the R value heads of a q/k head, in their order (row: a token); dq and dk
template <typename T>
__global__ void __launch_bounds__(256) heads_kernel(const float* __restrict__ src0, const float* __restrict__ src1,
                                                    int64_t quads, int R, int K4, const int32_t* __restrict__ nc,
                                                    T* __restrict__ dst0, T* __restrict__ dst1) {
  if (nc && *nc < 0) return;
  const float* src = blockIdx.y ? src1 : src0;
  T* dst = blockIdx.y ? dst1 : dst0;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= quads) return;
  const int64_t head = at / K4;
  const float* p = src + ((head * R) * K4 + (at - head * K4)) * 4;
  float4 s = load4(p);
  for (int r = 1; r < R; ++r) {
    const float4 x = load4(p + (int64_t)r * K4 * 4);
    s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
  }
  const float v[4] = {s.x, s.y, s.z, s.w};
  store4(dst + at * 4, v);
}

// dq and dk: fp32 [B, T, Hv, K] -> [B, T, Hqk, K].
template <typename T>
gdn_status launch_heads(const gdn_linear_problem& p, const float* own_dq, const float* own_dk, const int32_t* nc, T* dq,
                        T* dk, cudaStream_t s) {
  const int64_t quads = (int64_t)p.B * p.T * p.Hqk * (p.K / 4);
  const dim3 grid((unsigned)ceil_div(quads, 256), 2);
  heads_kernel<T><<<grid, 256, 0, s>>>(own_dq, own_dk, quads, p.Hv / p.Hqk, p.K / 4, nc, dq, dk);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

// dg of fixed decays from the chunks' sums [chunks][Hv] (gdn_linear_bwd.cu).
gdn_status launch_head_decays(const gdn_linear_problem& p, const float* part, const int32_t* nc, float* dg,
                              cudaStream_t s);

}  // namespace lin
}  // namespace gdn
