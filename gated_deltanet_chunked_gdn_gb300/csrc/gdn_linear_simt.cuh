// gdn_linear_simt.cuh -- fp32 tiles of decayed linear attention: 64 x 64 x 64 products by 256 threads (4 x 4 results a
// thread, operands in shared memory with the summed dimension outermost), and the sums along a sequence.
#pragma once

#include <string.h>

#include "gdn_linear.cuh"

namespace gdn {
namespace lin {

constexpr int kThreads = 256;
constexpr int kLd = 68;   // row length of a tile in shared memory: 16-byte rows, transposed stores without conflicts

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

__device__ __forceinline__ void zero(float (&a)[4][4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) a[i][j] = 0.f;
}

// dst[row][col] = src[row][col] * w[row] for 64 x 64 elements; rows past `rows` are zeros.
template <typename T>
__device__ __forceinline__ void load_n(float* dst, const T* src, int64_t ld, int rows, const float* w) {
  const int c = 4 * (threadIdx.x & 15);
#pragma unroll
  for (int r = threadIdx.x >> 4; r < kC; r += kThreads / 16) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows) {
      x = load4(src + r * ld + c);
      if (w) {
        const float f = w[r];
        x.x *= f, x.y *= f, x.z *= f, x.w *= f;
      }
    }
    *reinterpret_cast<float4*>(dst + r * kLd + c) = x;
  }
}

// dst[col][row] = src[row][col] * w[row].
template <typename T>
__device__ __forceinline__ void load_t(float* dst, const T* src, int64_t ld, int rows, const float* w) {
  const int r = threadIdx.x & 63;
  const float f = w ? w[r] : 1.f;
#pragma unroll
  for (int c = 4 * (threadIdx.x >> 6); c < kC; c += 16) {
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows) {
      x = load4(src + r * ld + c);
      if (w) x.x *= f, x.y *= f, x.z *= f, x.w *= f;
    }
    dst[c * kLd + r] = x.x, dst[(c + 1) * kLd + r] = x.y, dst[(c + 2) * kLd + r] = x.z, dst[(c + 3) * kLd + r] = x.w;
  }
}

// acc[r][u] += sum_kk A[kk][4 ty + r] B[kk][4 tx + u] over 64 kk, two columns an instruction
__device__ __forceinline__ void fma_tile(float (&acc)[4][4], const float* A, const float* B, int ty, int tx) {
  float2 c[4][2];
#pragma unroll
  for (int r = 0; r < 4; ++r) c[r][0] = make_float2(acc[r][0], acc[r][1]), c[r][1] = make_float2(acc[r][2], acc[r][3]);
#pragma unroll 16
  for (int kk = 0; kk < kC; ++kk) {
    const float4 a = *reinterpret_cast<const float4*>(A + kk * kLd + 4 * ty);
    const float4 b = *reinterpret_cast<const float4*>(B + kk * kLd + 4 * tx);
    const float av[4] = {a.x, a.y, a.z, a.w};
    const float2 b0 = make_float2(b.x, b.y), b1 = make_float2(b.z, b.w);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float2 ar = make_float2(av[r], av[r]);
      c[r][0] = __ffma2_rn(ar, b0, c[r][0]);
      c[r][1] = __ffma2_rn(ar, b1, c[r][1]);
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) acc[r][0] = c[r][0].x, acc[r][1] = c[r][0].y, acc[r][2] = c[r][1].x, acc[r][3] = c[r][1].y;
}

// Along every sequence, in place: S_c (what chunk c adds) becomes the state before chunk c (REV: the adjoint of the
// state behind it); four elements of a state a thread, the next chunks' loads in flight.
template <bool REV>
__global__ void __launch_bounds__(256) sums_kernel(Shape d, Pieces pc, const float* __restrict__ total,
                                                   const float* __restrict__ init, float* __restrict__ S,
                                                   float* __restrict__ fin, const int32_t* __restrict__ idx,
                                                   int slots) {
  const int64_t kv = (int64_t)d.K * d.V;
  const int per = (int)(kv / 1024);   // CTAs a state
  const int nh = blockIdx.x / per, n = nh / d.Hv, h = nh % d.Hv;
  const int64_t at = ((int64_t)(blockIdx.x % per) * 256 + threadIdx.x) * 4;
  if (pc.seq && *pc.nc < 0) return;
  const int c0 = pc.seq ? pc.first[n] : n * pc.per, c1 = pc.seq ? pc.first[n + 1] : c0 + pc.per;
  float4 run = init ? load4(init + nh * kv + at) : make_float4(0.f, 0.f, 0.f, 0.f);
  // the next four chunks' loads are under way while these are added up
  constexpr int AHEAD = 4;
  float4 x[2][AHEAD];
  float a[2][AHEAD];
  auto chunk = [&](int i) { return REV ? c1 - 1 - i : c0 + i; };
  auto fetch = [&](float4 (&y)[AHEAD], float (&f)[AHEAD], int base) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (base + i < c1 - c0) {
        y[i] = __ldcs(reinterpret_cast<const float4*>(S + ((int64_t)chunk(base + i) * d.Hv + h) * kv + at));
        f[i] = total[(int64_t)chunk(base + i) * d.Hv + h];
      }
  };
  auto add = [&](const float4 (&y)[AHEAD], const float (&f)[AHEAD], int base) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (base + i < c1 - c0) {
        *reinterpret_cast<float4*>(S + ((int64_t)chunk(base + i) * d.Hv + h) * kv + at) = run;
        run.x = fmaf(f[i], run.x, y[i].x), run.y = fmaf(f[i], run.y, y[i].y);
        run.z = fmaf(f[i], run.z, y[i].z), run.w = fmaf(f[i], run.w, y[i].w);
      }
  };
  fetch(x[0], a[0], 0);
  for (int base = 0; base < c1 - c0; base += 2 * AHEAD) {
    fetch(x[1], a[1], base + AHEAD);
    add(x[0], a[0], base);
    fetch(x[0], a[0], base + 2 * AHEAD);
    add(x[1], a[1], base + AHEAD);
  }
  if (fin) {
    int64_t row = n;
    if (idx) {
      row = idx[n];
      if (row < 0 || row >= slots) return;
    }
    *reinterpret_cast<float4*>(fin + (row * d.Hv + h) * kv + at) = run;
  }
}

// What a chunk adds to the state behind it, sum_j e^{b_last - b_j} x_j y_j^T (x = k, y = v), or, for the adjoint, to
// the one before it, factor sum_i e^{b_i} x_i y_i^T (x = q, y = do), and its whole decay; the outputs of every chunk
// from the state before it (gdn_linear_tc32.cu).
template <typename T, bool ADJ>
gdn_status launch_states(const Shape& d, const T* x, int64_t ldx, const T* y, int64_t ldy, const float* g,
                         const Pieces& pc, int most, float factor, float* S, float* total, int32_t* status,
                         cudaStream_t s);
gdn_status launch_outputs(const Shape& d, const float* q, const float* k, const float* v, const float* g,
                          const Pieces& pc, int most, float scale, const float* S0, float* o, int32_t* status,
                          cudaStream_t s);

template <bool REV>
gdn_status launch_sums(const Shape& d, const Pieces& pc, int N, const float* total, const float* init, float* S,
                       float* fin, const int32_t* idx, int slots, cudaStream_t s) {
  const int64_t grid = (int64_t)N * d.Hv * ((int64_t)d.K * d.V / 1024);
  sums_kernel<REV><<<(unsigned)grid, 256, 0, s>>>(d, pc, total, init, S, fin, idx, slots);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

// dst[row][hq][:] = sum over the R value heads of a q/k head, in their order (row: a token)
template <typename T>
__global__ void __launch_bounds__(256) heads_kernel(const float* __restrict__ src, int64_t quads, int R, int K4,
                                                    const int32_t* __restrict__ nc, T* __restrict__ dst) {
  if (nc && *nc < 0) return;
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

// src: fp32 [B, T, Hv, K]; dst [B, T, Hqk, K].
template <typename T>
gdn_status launch_heads(const gdn_linear_problem& p, const float* src, const int32_t* nc, T* dst, cudaStream_t s) {
  const int64_t quads = (int64_t)p.B * p.T * p.Hqk * (p.K / 4);
  heads_kernel<T><<<(unsigned)ceil_div(quads, 256), 256, 0, s>>>(src, quads, p.Hv / p.Hqk, p.K / 4, nc, dst);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

// dg of fixed decays from the chunks' sums [chunks][Hv] (gdn_linear_bwd.cu).
gdn_status launch_head_decays(const gdn_linear_problem& p, const float* part, const int32_t* nc, float* dg,
                              cudaStream_t s);

}  // namespace lin
}  // namespace gdn
