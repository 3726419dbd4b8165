// gdn_norms.cu -- norms around a mixer, forward and backward, one pass over the rows:
//
//   gated norm     y = silu(z) * w * xhat,  xhat = x r,  r = 1 / sqrt(mean(x^2) + eps)   (a row: one head of a token)
//   residual norm  u = w_post * y r1 (or y),  h = residual + scale * gate * u,  n = w * h r2 (or none)
//
// Backward of xhat = x r for an upstream gradient a: dx = r (a - xhat mean(a xhat)).  The residual norm's backward
// forms h again from its inputs in fp32 (reading y and the residual costs what reading h would, and h may have been
// rounded to bf16).  Statistics and sums are fp32; every output is rounded once.
//
// All of it is bound by HBM traffic.  A row is held in registers by 16 or 32 lanes (several rows a CTA, sums by
// shuffles) or by the threads of a CTA, in 16-byte vectors where rows are 16-byte aligned, in single elements
// otherwise.  The gradients of the weights are summed by column: every CTA takes rows at a fixed stride, adds each into
// fp32 columns of its own (registers or shared memory), and a second launch adds the CTAs' columns in a fixed order.
// Measured, of the bytes that have to move: gated norm, 16384 x 32 rows of 128 in bf16: forward 71 us (5.7 TB/s),
// backward 115 (5.8); residual norm, 8192 x 4096 in bf16: forward 57 us (4.7); 4099 x 2500 in fp32 with a gate of its own
// for each element: forward 37 us (5.5), backward 100 (3.3).  Wide rows' backwards hold more than a thread's registers:
// residual norm above 4096 bf16 elements (4096 x 8192 214 us, 1.9 TB/s; 2048 x 16384 473, 0.9), gated norm above 8192
// (2048 x 16384 in bf16 618 us, 0.5 TB/s, in fp32 398, 1.7; 4096 x 8192 in bf16 87, 3.9).
#include "gdn_internal.h"

namespace gdn {
namespace {

// VEC elements as they lie in memory: 16 bytes or a multiple, or one element.
template <typename T, int VEC>
struct Raw {
  uint4 v[VEC * sizeof(T) / 16];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)(VEC * sizeof(T) / 16); ++i) v[i] = reinterpret_cast<const uint4*>(p)[i];
  }
  __device__ __forceinline__ void get(float (&f)[VEC]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < VEC / 4; ++i) {
        f[4 * i] = __uint_as_float(v[i].x), f[4 * i + 1] = __uint_as_float(v[i].y);
        f[4 * i + 2] = __uint_as_float(v[i].z), f[4 * i + 3] = __uint_as_float(v[i].w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < VEC / 8; ++i) {
        const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          f[8 * i + 2 * j] = __uint_as_float(w[j] << 16), f[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    }
  }
};
template <typename T>
struct Raw<T, 1> {
  T v;
  __device__ __forceinline__ void load(const T* p) { v = *p; }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = to_f(v); }
};

template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[VEC]) {
  Raw<T, VEC> r;
  r.load(p);
  r.get(f);
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename T, int VEC>
__device__ __forceinline__ void store_vec(T* p, const float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    *p = from_f<T>(v[0]);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
  }
}

// A row's threads: GROUP lanes of a warp (16 or 32), or all of a CTA (GROUP 0).
constexpr int kGroupThreads = 256;

template <int GROUP>
__device__ __forceinline__ int row_threads() {
  return GROUP ? GROUP : (int)blockDim.x;
}

// Sum over a row's threads.  A CTA's: one barrier, the warps' sums in alternating halves of sm[2][32] (a half is
// written again only after the next sum's barrier, which every reader of it has passed), added in one order.
template <int GROUP>
__device__ __forceinline__ float row_sum(float v, float* sm, int& phase) {
#pragma unroll
  for (int o = (GROUP == 16 ? 16 : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (GROUP == 0) {
    float* s = sm + 32 * phase;
    phase ^= 1;
    const int lane = threadIdx.x & 31;
    if (lane == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < (int)(blockDim.x >> 5) ? s[lane] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  }
  return v;
}

// 1 / (1 + e^-z), and what it lacks to 1.  For bf16 rows by the exponential and reciprocal units: within 2^-21 + |z| 2^-24
// of it, relatively (far out it is 0 or 1), which the outputs' rounding covers.  fp32 rows keep their bits, within 2^-22 of
// each: e^-|z| by expf, whose argument is not rounded, and both values as quotients by 1 + e^-|z|.
template <typename T>
__device__ __forceinline__ float sigmoid_f(float z, float& rest) {
  if constexpr (sizeof(T) == 4) {
    const float e = expf(-fabsf(z)), r = __fdividef(1.f, 1.f + e), er = e * r;
    rest = z >= 0.f ? er : r;
    return z >= 0.f ? r : er;
  }
  const float s = __fdividef(1.f, 1.f + __expf(-z));
  rest = 1.f - s;
  return s;
}

// ------------------------------------------------------------- gated norm
template <typename T, int VEC, int NV, int GROUP>
__global__ void __launch_bounds__(GROUP ? kGroupThreads : 512) gated_fwd_kernel(
    const T* __restrict__ x, int64_t ldx, const T* __restrict__ z, int64_t ldz, const float* __restrict__ w, int rows,
    int H, int V, float eps, T* __restrict__ y, float* __restrict__ rstd) {
  __shared__ float sm[64];
  int phase = 0;
  constexpr bool AHEAD = NV * VEC <= 8;   // rows that leave registers for the next one's loads
  const int tpr = row_threads<GROUP>();
  constexpr int RPB = GROUP ? kGroupThreads / GROUP : 1;
  const int t = GROUP ? threadIdx.x % GROUP : threadIdx.x, grp = GROUP ? threadIdx.x / GROUP : 0;
  Raw<T, VEC> nx[NV], nz[NV];
  auto fetch = [&](int64_t row) {
    const int64_t token = (int)row / H, head = (int)row - token * H;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + t) * VEC;
      if (e < V) {
        nx[i].load(x + token * ldx + head * V + e);
        if (z) nz[i].load(z + token * ldz + head * V + e);
      }
    }
  };
  const int64_t step = (int64_t)gridDim.x * RPB;
  if (AHEAD && (int64_t)blockIdx.x * RPB + grp < rows) fetch((int64_t)blockIdx.x * RPB + grp);
  for (int64_t base = (int64_t)blockIdx.x * RPB; base < rows; base += step) {
    const int64_t row = base + grp;
    const bool live = row < rows;
    if (!AHEAD && live) fetch(row);
    float a[NV][VEC];
    Raw<T, VEC> cz[NV];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + t) * VEC;
      const bool in = live && e < V;
      nx[i].get(a[i]);
      cz[i] = nz[i];
#pragma unroll
      for (int j = 0; j < VEC; ++j) ss += in ? a[i][j] * a[i][j] : 0.f;
    }
    if (AHEAD && row + step < rows) fetch(row + step);
    const float r = rsqrtf(row_sum<GROUP>(ss, sm, phase) / V + eps);
    if (!live) continue;
    if (rstd && t == 0) rstd[row] = r;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + t) * VEC;
      if (e >= V) continue;
      float c[VEC], g[VEC];
      load_vec<float, VEC>(w + e, c);
      if (z) cz[i].get(g);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float u = a[i][j] * r * c[j];
        float rest;
        a[i][j] = z ? u * (g[j] * sigmoid_f<T>(g[j], rest)) : u;
      }
      store_vec<T, VEC>(y + row * V + e, a[i]);
    }
  }
}

template <typename T, int VEC, int NV, int GROUP>
__global__ void __launch_bounds__(GROUP ? kGroupThreads : 512) gated_bwd_kernel(
    const T* __restrict__ x, int64_t ldx, const T* __restrict__ z, int64_t ldz, const float* __restrict__ w,
    const float* __restrict__ rstd, const T* __restrict__ dy, int rows, int H, int V, T* __restrict__ dx,
    T* __restrict__ dz, float* __restrict__ part) {
  __shared__ float sm[64];
  extern __shared__ float cols[];   // [RPB][V]
  int phase = 0;
  const int tpr = row_threads<GROUP>();
  constexpr int RPB = GROUP ? kGroupThreads / GROUP : 1;
  const int t = GROUP ? threadIdx.x % GROUP : threadIdx.x, grp = GROUP ? threadIdx.x / GROUP : 0;
  float dw[NV][VEC], wv[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (i * tpr + t) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) dw[i][j] = 0.f, wv[i][j] = 0.f;
    if (e < V) load_vec<float, VEC>(w + e, wv[i]);
  }
  constexpr bool AHEAD = NV * VEC <= 8;   // rows that leave registers for the next one's loads
  Raw<T, VEC> nx[NV], nd[NV], nz[NV];
  float nr = 0.f;
  auto fetch = [&](int64_t row) {
    const int64_t token = (int)row / H, head = (int)row - token * H;
    nr = rstd[row];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + t) * VEC;
      if (e < V) {
        nx[i].load(x + token * ldx + head * V + e);
        nd[i].load(dy + row * V + e);
        if (z) nz[i].load(z + token * ldz + head * V + e);
      }
    }
  };
  if (AHEAD && (int64_t)blockIdx.x * RPB + grp < rows) fetch((int64_t)blockIdx.x * RPB + grp);
  // whole groups of RPB rows: every thread of a row's warp takes part in its sums
  const int64_t step = (int64_t)gridDim.x * RPB;
  for (int64_t base = (int64_t)blockIdx.x * RPB; base < rows; base += step) {
    const int64_t row = base + grp;
    const bool live = row < rows;
    if (!AHEAD && live) fetch(row);
    const float r = live ? nr : 0.f;
    float xh[NV][VEC], d[NV][VEC], zz[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + t) * VEC;
      if (live && e < V) {
        nx[i].get(xh[i]);
        nd[i].get(d[i]);
        if (z) nz[i].get(zz[i]);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) xh[i][j] = 0.f, d[i][j] = 0.f, zz[i][j] = 0.f;
      }
    }
    if (AHEAD && row + step < rows) fetch(row + step);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + t) * VEC;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float h = xh[i][j] * r;
        xh[i][j] = h;
        float du = d[i][j];
        if (z) {
          float rest;
          const float zv = zz[i][j], sg = sigmoid_f<T>(zv, rest);
          zz[i][j] = du * h * wv[i][j] * (sg * fmaf(zv, rest, 1.f));
          du *= zv * sg;
        }
        dw[i][j] = fmaf(du, h, dw[i][j]);
        d[i][j] = du * wv[i][j];
        s = fmaf(d[i][j], h, s);
      }
      if (z && live && e < V) store_vec<T, VEC>(dz + row * V + e, zz[i]);
    }
    const float m = row_sum<GROUP>(s, sm, phase) / V;
    if (live) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = (i * tpr + t) * VEC;
        if (e >= V) continue;
#pragma unroll
        for (int j = 0; j < VEC; ++j) d[i][j] = r * (d[i][j] - xh[i][j] * m);
        store_vec<T, VEC>(dx + row * V + e, d[i]);
      }
    }
  }
  if constexpr (GROUP == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + t) * VEC;
      if (e < V) store_vec<float, VEC>(part + (int64_t)blockIdx.x * V + e, dw[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + t) * VEC;
      if (e < V) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) cols[grp * V + e + j] = dw[i][j];
      }
    }
    __syncthreads();
    for (int e = threadIdx.x; e < V; e += kGroupThreads) {
      float s = 0.f;
#pragma unroll
      for (int g = 0; g < RPB; ++g) s += cols[g * V + e];
      part[(int64_t)blockIdx.x * V + e] = s;
    }
  }
}

// ---------------------------------------------------------- residual norm
// gate: 0 none, 1 a vector of D fp32, 2 a value of type T for every element.  Rows of up to 8 elements a thread have the
// next row's loads in flight, and registers for two CTAs an SM.
template <typename T, typename R, int VEC, int NV, int GROUP>
__global__ void __launch_bounds__(GROUP ? kGroupThreads : 512, NV * VEC <= 8 ? (GROUP ? 4 : 2) : 1) residual_fwd_kernel(
    const T* __restrict__ y, int64_t ldy, const R* __restrict__ res, const float* __restrict__ pw,
    const void* __restrict__ gate, int gmode, float scale, const float* __restrict__ w, int rows, int D, float eps,
    R* __restrict__ hout, T* __restrict__ nout, float* __restrict__ rstd) {
  __shared__ float sm[64];
  int phase = 0;
  constexpr bool AHEAD = NV * VEC <= 8;
  const int tpr = row_threads<GROUP>();
  constexpr int RPB = GROUP ? kGroupThreads / GROUP : 1;
  const int t = GROUP ? threadIdx.x % GROUP : threadIdx.x, grp = GROUP ? threadIdx.x / GROUP : 0;
  Raw<T, VEC> ny[NV];
  Raw<R, VEC> nr[NV];
  auto fetch = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + t) * VEC;
      if (e < D) {
        ny[i].load(y + row * ldy + e);
        nr[i].load(res + row * D + e);
      }
    }
  };
  const int64_t step = (int64_t)gridDim.x * RPB;
  if (AHEAD && (int64_t)blockIdx.x * RPB + grp < rows) fetch((int64_t)blockIdx.x * RPB + grp);
  for (int64_t base = (int64_t)blockIdx.x * RPB; base < rows; base += step) {
    const int64_t row = base + grp;
    const bool live = row < rows;
    if (!AHEAD && live) fetch(row);
    float a[NV][VEC];
    Raw<R, VEC> cr[NV];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + t) * VEC;
      const bool in = live && e < D;
      ny[i].get(a[i]);
      cr[i] = nr[i];
#pragma unroll
      for (int j = 0; j < VEC; ++j) ss += in ? a[i][j] * a[i][j] : 0.f;
    }
    if (AHEAD && row + step < rows) fetch(row + step);
    float r1 = 1.f;
    if (pw) r1 = rsqrtf(row_sum<GROUP>(ss, sm, phase) / D + eps);
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + t) * VEC;
      if (!live || e >= D) continue;
      float f[VEC];
      if (pw) {
        load_vec<float, VEC>(pw + e, f);
#pragma unroll
        for (int j = 0; j < VEC; ++j) a[i][j] = a[i][j] * r1 * f[j];
      }
      if (gmode == 1) load_vec<float, VEC>(static_cast<const float*>(gate) + e, f);
      if (gmode == 2) load_vec<T, VEC>(static_cast<const T*>(gate) + row * D + e, f);
      if (gmode) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) a[i][j] *= f[j];
      }
      cr[i].get(f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        a[i][j] = fmaf(scale, a[i][j], f[j]);
        ss += a[i][j] * a[i][j];
      }
      store_vec<R, VEC>(hout + row * D + e, a[i]);
    }
    float r2 = 1.f;
    if (w) {
      r2 = rsqrtf(row_sum<GROUP>(ss, sm, phase) / D + eps);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = (i * tpr + t) * VEC;
        if (!live || e >= D) continue;
        float f[VEC];
        load_vec<float, VEC>(w + e, f);
#pragma unroll
        for (int j = 0; j < VEC; ++j) a[i][j] = a[i][j] * r2 * f[j];
        store_vec<T, VEC>(nout + row * D + e, a[i]);
      }
    }
    if (rstd && live && t == 0) rstd[2 * row] = r1, rstd[2 * row + 1] = r2;
  }
}

// Column sums of dweight, dpost_weight and dgate: in registers for rows of up to 8 elements a thread, else in shared
// memory ([RPB][3][D]; a thread adds to columns that no other thread of its row touches).  Where registers are left, the
// next row's loads are in flight.  The furthest of these kernels from the bytes' time: registers for one CTA an SM, whose
// 16 warps issue a third to half of the time (790 instructions a row and warp of 4096 fp32, and two sums over the CTA).
// Some of those registers and instructions go to sums for weights and gates that a call does not have: the kinds are not
// known where this is compiled, so all three are formed, and the second launch drops what nobody asked for.  Slower were,
// for 8192 x 4096 in bf16 (122 us), fewer threads a row (206), 64 registers and two CTAs (326, spills), the next three
// rows in a ring in shared memory (135); for 4099 x 2500 in fp32 (100), that ring (105) and twice the threads (116).
template <typename T, typename R, int VEC, int NV, int GROUP>
__global__ void __launch_bounds__(GROUP ? kGroupThreads : 512) residual_bwd_kernel(
    const T* __restrict__ y, int64_t ldy, const R* __restrict__ res, const float* __restrict__ rstd,
    const R* __restrict__ dh, const T* __restrict__ dn, const float* __restrict__ pw, const void* __restrict__ gate,
    int gmode, float scale, const float* __restrict__ w, int rows, int D, T* __restrict__ dy, R* __restrict__ dres,
    T* __restrict__ dgate, float* __restrict__ part) {
  __shared__ float sm[64];
  extern __shared__ __align__(16) float cols[];
  int phase = 0;
  constexpr bool KEEP = NV * VEC <= 8;
  constexpr bool AHEAD = NV * VEC * (int)sizeof(R) <= 16;
  constexpr int KV = KEEP ? NV : 1;
  const int tpr = row_threads<GROUP>();
  constexpr int RPB = GROUP ? kGroupThreads / GROUP : 1;
  const int t = GROUP ? threadIdx.x % GROUP : threadIdx.x, grp = GROUP ? threadIdx.x / GROUP : 0;
  float* cw = cols + (int64_t)grp * 3 * D;
  float* cp = cw + D;
  float* cg = cp + D;
  float aw[KV][VEC], ap[KV][VEC], ag[KV][VEC];   // KEEP: the sums
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < VEC; ++j) aw[i][j] = ap[i][j] = ag[i][j] = 0.f;
  } else {
    for (int e = threadIdx.x; e < RPB * 3 * D; e += blockDim.x) cols[e] = 0.f;
    __syncthreads();
  }
  auto add = [&](float* to, const float (&v)[VEC]) {
    if constexpr (VEC == 1) {
      *to += v[0];
    } else if ((D & 3) == 0) {   // 16-byte aligned columns
#pragma unroll
      for (int j = 0; j < VEC; j += 4) {
        float4 x = *reinterpret_cast<float4*>(to + j);
        x.x += v[j], x.y += v[j + 1], x.z += v[j + 2], x.w += v[j + 3];
        *reinterpret_cast<float4*>(to + j) = x;
      }
    } else {
#pragma unroll
      for (int j = 0; j < VEC; ++j) to[j] += v[j];
    }
  };
  auto gate_of = [&](int64_t row, int e, float (&f)[VEC]) {
    if (gmode == 1) load_vec<float, VEC>(static_cast<const float*>(gate) + e, f);
    if (gmode == 2) load_vec<T, VEC>(static_cast<const T*>(gate) + row * D + e, f);
  };
  Raw<T, VEC> ny[NV], nn[NV], ng[NV];
  Raw<R, VEC> nh[NV], ns[NV];
  float n1 = 0.f, n2 = 0.f;
  auto fetch = [&](int64_t row) {
    n1 = rstd[2 * row], n2 = rstd[2 * row + 1];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + t) * VEC;
      if (e >= D) continue;
      ny[i].load(y + row * ldy + e);
      if (dh) nh[i].load(dh + row * D + e);
      if (w) {
        ns[i].load(res + row * D + e);
        nn[i].load(dn + row * D + e);
      }
      if (KEEP && gmode == 2) ng[i].load(static_cast<const T*>(gate) + row * D + e);
    }
  };
  const int64_t step = (int64_t)gridDim.x * RPB;
  if (AHEAD && (int64_t)blockIdx.x * RPB + grp < rows) fetch((int64_t)blockIdx.x * RPB + grp);
  for (int64_t base = (int64_t)blockIdx.x * RPB; base < rows; base += step) {
    const int64_t row = base + grp;
    const bool live = row < rows;
    if (!AHEAD && live) fetch(row);
    const float r1 = live ? n1 : 0.f, r2 = live ? n2 : 0.f;
    float yh[NV][VEC], d[NV][VEC], hh[NV][VEC], aa[NV][VEC], gt[KV][VEC];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + t) * VEC;
      if (!live || e >= D) continue;
      ny[i].get(yh[i]);
      if (dh) {
        nh[i].get(d[i]);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) d[i][j] = 0.f;
      }
      if (w) {
        ns[i].get(hh[i]);
        nn[i].get(aa[i]);
      }
      if constexpr (KEEP) {
        if (gmode == 2) ng[i].get(gt[i]);
        else gate_of(row, e, gt[i]);
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) yh[i][j] *= r1;
    }
    if (AHEAD && row + step < rows) fetch(row + step);
    if (w) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = (i * tpr + t) * VEC;
        if (!live || e >= D) continue;
        float p[VEC], f[VEC], wv[VEC];
        if (pw) load_vec<float, VEC>(pw + e, p);
        if constexpr (!KEEP) gate_of(row, e, f);
        load_vec<float, VEC>(w + e, wv);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          float u = pw ? yh[i][j] * p[j] : yh[i][j];
          if (gmode) u *= KEEP ? gt[KEEP ? i : 0][j] : f[j];
          const float h = fmaf(scale, u, hh[i][j]) * r2;
          hh[i][j] = h;
          p[j] = aa[i][j] * h;
          aa[i][j] *= wv[j];
          s = fmaf(aa[i][j], h, s);
        }
        if constexpr (KEEP) {
#pragma unroll
          for (int j = 0; j < VEC; ++j) aw[i][j] += p[j];
        } else {
          add(cw + e, p);
        }
      }
      const float m = row_sum<GROUP>(s, sm, phase) / D;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = (i * tpr + t) * VEC;
        if (!live || e >= D) continue;
#pragma unroll
        for (int j = 0; j < VEC; ++j) d[i][j] += r2 * (aa[i][j] - hh[i][j] * m);
      }
    }
    s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + t) * VEC;
      if (!live || e >= D) continue;
      store_vec<R, VEC>(dres + row * D + e, d[i]);
      float p[VEC], f[VEC], dg[VEC], dp[VEC];
      if (pw) load_vec<float, VEC>(pw + e, p);
      if constexpr (!KEEP) gate_of(row, e, f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float du = scale * d[i][j];
        dg[j] = du * (pw ? yh[i][j] * p[j] : yh[i][j]);
        if (gmode) du *= KEEP ? gt[KEEP ? i : 0][j] : f[j];
        dp[j] = du * yh[i][j];
        if (pw) {
          du *= p[j];
          s = fmaf(du, yh[i][j], s);
        }
        d[i][j] = du;
      }
      if (gmode == 2) store_vec<T, VEC>(dgate + row * D + e, dg);
      if constexpr (KEEP) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) ag[i][j] += dg[j], ap[i][j] += dp[j];
      } else {
        if (gmode == 1) add(cg + e, dg);
        if (pw) add(cp + e, dp);
      }
    }
    float m = 0.f;
    if (pw) m = row_sum<GROUP>(s, sm, phase) / D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + t) * VEC;
      if (!live || e >= D) continue;
      if (pw) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) d[i][j] = r1 * (d[i][j] - yh[i][j] * m);
      }
      store_vec<T, VEC>(dy + row * D + e, d[i]);
    }
  }
  if constexpr (KEEP) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * tpr + t) * VEC;
      if (e >= D) continue;
#pragma unroll
      for (int j = 0; j < VEC; ++j) cw[e + j] = aw[i][j], cp[e + j] = ap[i][j], cg[e + j] = ag[i][j];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 3 * D; e += blockDim.x) {
    float s = 0.f;
#pragma unroll
    for (int g = 0; g < RPB; ++g) s += cols[(int64_t)g * 3 * D + e];
    part[(int64_t)blockIdx.x * 3 * D + e] = s;
  }
}

// out_k[c] = sum over the nb rows of part [nb][n * D] of column k D + c; 8 columns a CTA, 32 threads a column
__global__ void __launch_bounds__(256) columns_kernel(const float* __restrict__ part, int nb, int D, int n,
                                                      float* __restrict__ o0, float* __restrict__ o1,
                                                      float* __restrict__ o2) {
  __shared__ float sm[32][9];
  const int c = blockIdx.x * 8 + (threadIdx.x & 7), r = threadIdx.x >> 3;
  const int64_t width = (int64_t)n * D;
  float s = 0.f;
  if (c < width)
    for (int i = r; i < nb; i += 32) s += part[i * width + c];
  sm[r][threadIdx.x & 7] = s;
  __syncthreads();
  if (r == 0 && c < width) {
#pragma unroll
    for (int i = 1; i < 32; ++i) s += sm[i][threadIdx.x];
    float* o = c < D ? o0 : (c < 2 * D ? o1 : o2);
    if (o) o[c % D] = s;
  }
}

// How a row of D elements is held: vectors of `vec` elements, nv of them a thread; its threads are `group` lanes (16 or
// 32) or, for group 0, the `threads` of a CTA: as few vectors a thread as 512 threads can hold.
struct Shape {
  int vec, group, nv, threads;
  int rpb() const { return group ? kGroupThreads / group : 1; }
};

Shape shape_of(int D, int vec) {
  const int vectors = (int)ceil_div(D, vec), most = vec == 1 ? 8 : 16 / vec;   // vectors a lane
  Shape s{vec, 0, 1, kGroupThreads};
  if (vec > 1 && vectors <= 16) {
    s.group = 16;
  } else if (vectors <= 32 * most) {
    s.group = 32;
    while (32 * s.nv < vectors) s.nv *= 2;
  } else {
    while (512 * s.nv < vectors) s.nv *= 2;
    s.threads = 32 * (int)ceil_div(vectors, 32 * s.nv);
  }
  return s;
}

// CTAs of a pass whose CTAs take rows at a fixed stride: what the device holds at once, each of the backward's with
// columns of its own (kMostCtas an SM at most).
constexpr int kMostCtas = 8;

template <typename K>
int resident_ctas(K kernel, int threads, size_t smem, int64_t rows, int rpb) {
  const int64_t need = ceil_div(rows, rpb);
  if (need <= sm_count()) return (int)need;
  int per = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per, kernel, threads, smem) != cudaSuccess || per < 1) per = 1;
  if (per > kMostCtas) per = kMostCtas;
  const int64_t most = (int64_t)per * sm_count();
  return (int)(need < most ? need : most);
}

// Above 48 KB, the kernel's static part counted, shared memory has to be asked for.
template <typename K>
bool allow_smem(K kernel, size_t bytes) {
  return bytes <= 47 * 1024 ||
         cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess;
}

// The shapes that shape_of gives, and no others.
#define GDN_NORM_CASE(VEC, NV, GROUP, F)                                                                       \
  case NV:                                                                                                     \
    if constexpr ((NV) * (VEC) <= ((GROUP) == 0 ? 32 : ((VEC) == 1 ? 8 : 16))) F(VEC, NV, GROUP);              \
    break;
#define GDN_NORM_NV(VEC, GROUP, F)                                                                             \
  switch (s.nv) {                                                                                              \
    GDN_NORM_CASE(VEC, 1, GROUP, F)                                                                            \
    GDN_NORM_CASE(VEC, 2, GROUP, F)                                                                            \
    GDN_NORM_CASE(VEC, 4, GROUP, F)                                                                            \
    GDN_NORM_CASE(VEC, 8, GROUP, F)                                                                            \
    GDN_NORM_CASE(VEC, 16, GROUP, F)                                                                           \
    GDN_NORM_CASE(VEC, 32, GROUP, F)                                                                           \
  }
#define GDN_NORM_SHAPE(VEC, F)                                                                                 \
  switch (s.group) {                                                                                           \
    case 16: if constexpr (VEC > 1) F(VEC, 1, 16); break;                                                      \
    case 32: GDN_NORM_NV(VEC, 32, F) break;                                                                    \
    default: GDN_NORM_NV(VEC, 0, F)                                                                            \
  }

bool rows16(const void* p, int64_t row_bytes) {
  return p == nullptr || ((reinterpret_cast<uintptr_t>(p) | (uint64_t)row_bytes) & 15) == 0;
}

template <typename T>
gdn_status gated_fwd_t(const T* x, int64_t ldx, const T* z, int64_t ldz, const float* w, int tokens, int H, int V,
                       float eps, T* y, float* rstd, cudaStream_t st) {
  constexpr int VW = 16 / (int)sizeof(T);
  const int es = sizeof(T), rows = tokens * H;
  const bool wide = rows16(x, ldx * es) && rows16(z, ldz * es) && rows16(w, 0) && rows16(y, (int64_t)V * es);
  const Shape s = shape_of(V, wide ? VW : 1);
#define GDN_F(VEC, NV, GROUP)                                                                                       \
  {                                                                                                                 \
    auto kern = gated_fwd_kernel<T, VEC, NV, GROUP>;                                                                \
    kern<<<resident_ctas(kern, s.threads, 0, rows, s.rpb()), s.threads, 0, st>>>(x, ldx, z, ldz, w, rows, H, V, eps, \
                                                                                 y, rstd);                          \
  }
  if (wide) {
    GDN_NORM_SHAPE(VW, GDN_F)
  } else {
    GDN_NORM_SHAPE(1, GDN_F)
  }
#undef GDN_F
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

template <typename T>
gdn_status gated_bwd_t(const T* x, int64_t ldx, const T* z, int64_t ldz, const float* w, const float* rstd,
                       const T* dy, int tokens, int H, int V, T* dx, T* dz, float* dw, float* part, cudaStream_t st) {
  constexpr int VW = 16 / (int)sizeof(T);
  const int es = sizeof(T), rows = tokens * H;
  const bool wide = rows16(x, ldx * es) && rows16(z, ldz * es) && rows16(w, 0) && rows16(dy, (int64_t)V * es) &&
                    rows16(dx, 0) && rows16(dz, 0);
  const Shape s = shape_of(V, wide ? VW : 1);
  const size_t smem = s.group ? sizeof(float) * s.rpb() * V : 0;
  int grid = 0;
#define GDN_F(VEC, NV, GROUP)                                                                                       \
  {                                                                                                                 \
    auto kern = gated_bwd_kernel<T, VEC, NV, GROUP>;                                                                \
    grid = resident_ctas(kern, s.threads, smem, rows, s.rpb());                                                     \
    kern<<<grid, s.threads, smem, st>>>(x, ldx, z, ldz, w, rstd, dy, rows, H, V, dx, dz, part);                     \
  }
  if (wide) {
    GDN_NORM_SHAPE(VW, GDN_F)
  } else {
    GDN_NORM_SHAPE(1, GDN_F)
  }
#undef GDN_F
  if (cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
  columns_kernel<<<(unsigned)ceil_div(V, 8), 256, 0, st>>>(part, grid, V, 1, dw, nullptr, nullptr);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

template <typename T, typename R>
gdn_status residual_fwd_t(const T* y, int64_t ldy, const R* res, const float* pw, const void* gate, int gmode,
                          float scale, const float* w, int rows, int D, float eps, R* h, T* n, float* rstd,
                          cudaStream_t st) {
  constexpr int VW = 16 / (int)(sizeof(T) < sizeof(R) ? sizeof(T) : sizeof(R));
  const int64_t rt = (int64_t)D * sizeof(T), rr = (int64_t)D * sizeof(R);
  const bool wide = rows16(y, ldy * (int)sizeof(T)) && rows16(res, rr) && rows16(pw, 0) && rows16(w, 0) &&
                    rows16(gate, gmode == 2 ? rt : 0) && rows16(h, rr) && rows16(n, rt) && rt % 16 == 0;
  const Shape s = shape_of(D, wide ? VW : 1);
#define GDN_F(VEC, NV, GROUP)                                                                                     \
  {                                                                                                                 \
    auto kern = residual_fwd_kernel<T, R, VEC, NV, GROUP>;                                                          \
    kern<<<resident_ctas(kern, s.threads, 0, rows, s.rpb()), s.threads, 0, st>>>(                                   \
        y, ldy, res, pw, gate, gmode, scale, w, rows, D, eps, h, n, rstd);                                          \
  }
  if (wide) {
    GDN_NORM_SHAPE(VW, GDN_F)
  } else {
    GDN_NORM_SHAPE(1, GDN_F)
  }
#undef GDN_F
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

template <typename T, typename R>
gdn_status residual_bwd_t(const T* y, int64_t ldy, const R* res, const float* rstd, const R* dh, const T* dn,
                          const float* pw, const void* gate, int gmode, float scale, const float* w, int rows, int D,
                          T* dy, R* dres, float* dpw, void* dgate, float* dw, float* part, cudaStream_t st) {
  constexpr int VW = 16 / (int)(sizeof(T) < sizeof(R) ? sizeof(T) : sizeof(R));
  const int64_t rt = (int64_t)D * sizeof(T), rr = (int64_t)D * sizeof(R);
  const bool wide = rows16(y, ldy * (int)sizeof(T)) && rows16(res, rr) && rows16(dh, rr) && rows16(dn, rt) &&
                    rows16(pw, 0) && rows16(w, 0) && rows16(gate, gmode == 2 ? rt : 0) && rows16(dy, rt) &&
                    rows16(dres, rr) && rows16(gmode == 2 ? dgate : nullptr, rt) && rt % 16 == 0;
  const Shape s = shape_of(D, wide ? VW : 1);
  const size_t smem = sizeof(float) * s.rpb() * 3 * D;
  int grid = 0;
  bool ok = true;
#define GDN_F(VEC, NV, GROUP)                                                                                       \
  {                                                                                                                 \
    auto kern = residual_bwd_kernel<T, R, VEC, NV, GROUP>;                                                          \
    ok = allow_smem(kern, smem);                                                                                    \
    grid = resident_ctas(kern, s.threads, smem, rows, s.rpb());                                                     \
    if (ok)                                                                                                         \
      kern<<<grid, s.threads, smem, st>>>(y, ldy, res, rstd, dh, dn, pw, gate, gmode, scale, w, rows, D, dy, dres,  \
                                          gmode == 2 ? static_cast<T*>(dgate) : nullptr, part);                     \
  }
  if (wide) {
    GDN_NORM_SHAPE(VW, GDN_F)
  } else {
    GDN_NORM_SHAPE(1, GDN_F)
  }
#undef GDN_F
  if (!ok || cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
  float* dgc = gmode == 1 ? static_cast<float*>(dgate) : nullptr;
  if (!dw && !dpw && !dgc) return GDN_OK;
  columns_kernel<<<(unsigned)ceil_div(3 * (int64_t)D, 8), 256, 0, st>>>(part, grid, D, 3, dw, dpw, dgc);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

// Rows of columns that the largest grid of a backward pass writes.
size_t gated_norm_bwd_workspace_bytes(int V) { return align_up(sizeof(float) * kMostCtas * (size_t)sm_count() * V); }
size_t residual_norm_bwd_workspace_bytes(int D) {
  return align_up(sizeof(float) * kMostCtas * (size_t)sm_count() * 3 * D);
}

gdn_status run_gated_norm_fwd(const void* x, int64_t ldx, const void* z, int64_t ldz, const float* w, int tokens, int H,
                              int V, gdn_dtype dt, float eps, void* y, float* rstd, cudaStream_t s) {
  if (dt == GDN_F32)
    return gated_fwd_t((const float*)x, ldx, (const float*)z, ldz, w, tokens, H, V, eps, (float*)y, rstd, s);
  using T = __nv_bfloat16;
  return gated_fwd_t((const T*)x, ldx, (const T*)z, ldz, w, tokens, H, V, eps, (T*)y, rstd, s);
}

gdn_status run_gated_norm_bwd(const void* x, int64_t ldx, const void* z, int64_t ldz, const float* w, const float* rstd,
                              const void* dy, int tokens, int H, int V, gdn_dtype dt, void* dx, void* dz, float* dw,
                              void* ws, cudaStream_t s) {
  if (dt == GDN_F32)
    return gated_bwd_t((const float*)x, ldx, (const float*)z, ldz, w, rstd, (const float*)dy, tokens, H, V, (float*)dx,
                       (float*)dz, dw, (float*)ws, s);
  using T = __nv_bfloat16;
  return gated_bwd_t((const T*)x, ldx, (const T*)z, ldz, w, rstd, (const T*)dy, tokens, H, V, (T*)dx, (T*)dz, dw,
                     (float*)ws, s);
}

gdn_status run_residual_norm_fwd(const void* y, int64_t ldy, const void* res, const float* pw, const void* gate,
                                 int gmode, float scale, const float* w, int rows, int D, gdn_dtype dt, gdn_dtype rdt,
                                 float eps, void* h, void* n, float* rstd, cudaStream_t s) {
  using T = __nv_bfloat16;
  if (dt == GDN_F32)
    return residual_fwd_t((const float*)y, ldy, (const float*)res, pw, gate, gmode, scale, w, rows, D, eps, (float*)h,
                          (float*)n, rstd, s);
  if (rdt == GDN_F32)
    return residual_fwd_t((const T*)y, ldy, (const float*)res, pw, gate, gmode, scale, w, rows, D, eps, (float*)h,
                          (T*)n, rstd, s);
  return residual_fwd_t((const T*)y, ldy, (const T*)res, pw, gate, gmode, scale, w, rows, D, eps, (T*)h, (T*)n, rstd,
                        s);
}

gdn_status run_residual_norm_bwd(const void* y, int64_t ldy, const void* res, const float* rstd, const void* dh,
                                 const void* dn, const float* pw, const void* gate, int gmode, float scale,
                                 const float* w, int rows, int D, gdn_dtype dt, gdn_dtype rdt, void* dy, void* dres,
                                 float* dpw, void* dgate, float* dw, void* ws, cudaStream_t s) {
  using T = __nv_bfloat16;
  float* part = static_cast<float*>(ws);
  if (dt == GDN_F32)
    return residual_bwd_t((const float*)y, ldy, (const float*)res, rstd, (const float*)dh, (const float*)dn, pw, gate,
                          gmode, scale, w, rows, D, (float*)dy, (float*)dres, dpw, dgate, dw, part, s);
  if (rdt == GDN_F32)
    return residual_bwd_t((const T*)y, ldy, (const float*)res, rstd, (const float*)dh, (const T*)dn, pw, gate, gmode,
                          scale, w, rows, D, (T*)dy, (float*)dres, dpw, dgate, dw, part, s);
  return residual_bwd_t((const T*)y, ldy, (const T*)res, rstd, (const T*)dh, (const T*)dn, pw, gate, gmode, scale, w,
                        rows, D, (T*)dy, (T*)dres, dpw, dgate, dw, part, s);
}

}  // namespace gdn
