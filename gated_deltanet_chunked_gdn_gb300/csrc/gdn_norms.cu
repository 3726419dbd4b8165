// gdn_norms.cu -- norms around a mixer, forward and backward, one pass over the rows:
//
//   gated norm     y = silu(z) * w * xhat,  xhat = x r,  r = 1 / sqrt(mean(x^2) + eps)   (a row: one head of a token)
//   residual norm  u = w_post * y r1 (or y),  h = residual + scale * gate * u,  n = w * h r2 (or none)
//
// Backward of xhat = x r for an upstream gradient a: dx = r (a - xhat mean(a xhat)).  The residual norm's backward
// forms h again from its inputs in fp32 (reading y and the residual costs what reading h would, and h may have been
// rounded to bf16).  Statistics and sums are fp32; every output is rounded once.
//
// All of it is bound by HBM traffic.  A row is held in registers by TPR threads (16 or 32: several rows a CTA, sums by
// shuffles; 128 or 512: a CTA a row), in 16-byte vectors where rows are 16-byte aligned, in single elements otherwise.
// The gradients of the weights are summed by column: every CTA takes rows at a fixed stride, adds each into fp32
// columns of its own (registers or shared memory), and a second launch adds the CTAs' columns in a fixed order.
#include "gdn_internal.h"

namespace gdn {
namespace {

template <typename T, int VEC>
__device__ __forceinline__ void load_vec(const T* p, float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    v[0] = to_f(*p);
  } else if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < VEC; i += 4) {
      const float4 x = *reinterpret_cast<const float4*>(p + i);
      v[i] = x.x, v[i + 1] = x.y, v[i + 2] = x.z, v[i + 3] = x.w;
    }
  } else if constexpr (VEC == 4) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    v[0] = __uint_as_float(x.x << 16), v[1] = __uint_as_float(x.x & 0xffff0000u);
    v[2] = __uint_as_float(x.y << 16), v[3] = __uint_as_float(x.y & 0xffff0000u);
  } else {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[2 * i] = __uint_as_float(w[i] << 16), v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
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
  } else if constexpr (VEC == 4) {
    *reinterpret_cast<uint2*>(p) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
  } else {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
  }
}

// Sum over the TPR threads of a row.  Rows of more than a warp: one barrier, the warps' sums in alternating halves of
// sm[2][32] (a half is written again only after the next sum's barrier, which every reader of it has passed).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* sm, int& phase) {
#pragma unroll
  for (int o = (TPR < 32 ? TPR : 32) / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if constexpr (TPR > 32) {
    float* s = sm + 32 * phase;
    phase ^= 1;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) v += s[i];
  }
  return v;
}

constexpr int kBlock(int TPR) { return TPR <= 32 ? 256 : TPR; }

__device__ __forceinline__ float sigmoid_f(float z) { return 1.f / (1.f + expf(-z)); }

// ------------------------------------------------------------- gated norm
template <typename T, int VEC, int NV, int TPR>
__global__ void __launch_bounds__(kBlock(TPR)) gated_fwd_kernel(const T* __restrict__ x, int64_t ldx,
                                                                const T* __restrict__ z, int64_t ldz,
                                                                const float* __restrict__ w, int rows, int H, int V,
                                                                float eps, T* __restrict__ y,
                                                                float* __restrict__ rstd) {
  __shared__ float sm[64];
  int phase = 0;
  constexpr int RPB = kBlock(TPR) / TPR;
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  const bool live = row < rows;
  const int64_t token = live ? (int)row / H : 0, head = live ? (int)row - token * H : 0;
  const T* xp = x + token * ldx + head * V;
  const T* zp = z ? z + token * ldz + head * V : nullptr;
  float a[NV][VEC], b[NV][VEC], c[NV][VEC];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (i * TPR + t) * VEC;
    const bool in = live && e < V;
    if (in) {
      load_vec<T, VEC>(xp + e, a[i]);
      load_vec<float, VEC>(w + e, c[i]);
      if (zp) load_vec<T, VEC>(zp + e, b[i]);
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) ss += in ? a[i][j] * a[i][j] : 0.f;
  }
  const float r = rsqrtf(row_sum<TPR>(ss, sm, phase) / V + eps);
  if (!live) return;
  if (rstd && t == 0) rstd[row] = r;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (i * TPR + t) * VEC;
    if (e >= V) continue;
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float u = a[i][j] * r * c[i][j];
      a[i][j] = zp ? u * (b[i][j] * sigmoid_f(b[i][j])) : u;
    }
    store_vec<T, VEC>(y + row * V + e, a[i]);
  }
}

template <typename T, int VEC, int NV, int TPR>
__global__ void __launch_bounds__(kBlock(TPR)) gated_bwd_kernel(const T* __restrict__ x, int64_t ldx,
                                                                const T* __restrict__ z, int64_t ldz,
                                                                const float* __restrict__ w,
                                                                const float* __restrict__ rstd,
                                                                const T* __restrict__ dy, int rows, int H, int V,
                                                                T* __restrict__ dx, T* __restrict__ dz,
                                                                float* __restrict__ part) {
  __shared__ float sm[64];
  extern __shared__ float cols[];   // [RPB][V]
  int phase = 0;
  constexpr int RPB = kBlock(TPR) / TPR;
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  float dw[NV][VEC], wv[NV][VEC];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (i * TPR + t) * VEC;
#pragma unroll
    for (int j = 0; j < VEC; ++j) dw[i][j] = 0.f, wv[i][j] = 0.f;
    if (e < V) load_vec<float, VEC>(w + e, wv[i]);
  }
  // whole groups of RPB rows: every thread of a row's warp takes part in its sums
  for (int64_t base = (int64_t)blockIdx.x * RPB; base < rows; base += (int64_t)gridDim.x * RPB) {
    const int64_t row = base + grp;
    const bool live = row < rows;
    const int64_t token = live ? (int)row / H : 0, head = live ? (int)row - token * H : 0;
    const T* xp = x + token * ldx + head * V;
    const T* zp = z ? z + token * ldz + head * V : nullptr;
    const float r = live ? rstd[row] : 0.f;
    float xh[NV][VEC], d[NV][VEC], zz[NV][VEC];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * TPR + t) * VEC;
      if (live && e < V) {
        load_vec<T, VEC>(xp + e, xh[i]);
        load_vec<T, VEC>(dy + row * V + e, d[i]);
        if (zp) load_vec<T, VEC>(zp + e, zz[i]);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) xh[i][j] = 0.f, d[i][j] = 0.f, zz[i][j] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * TPR + t) * VEC;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float h = xh[i][j] * r;
        xh[i][j] = h;
        float du = d[i][j];
        if (zp) {
          const float zv = zz[i][j], sg = sigmoid_f(zv);
          zz[i][j] = du * h * wv[i][j] * (sg * (1.f + zv * (1.f - sg)));
          du *= zv * sg;
        }
        dw[i][j] += du * h;
        d[i][j] = du * wv[i][j];
        s += d[i][j] * h;
      }
      if (zp && live && e < V) store_vec<T, VEC>(dz + row * V + e, zz[i]);
    }
    const float m = row_sum<TPR>(s, sm, phase) / V;
    if (live) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = (i * TPR + t) * VEC;
        if (e >= V) continue;
#pragma unroll
        for (int j = 0; j < VEC; ++j) d[i][j] = r * (d[i][j] - xh[i][j] * m);
        store_vec<T, VEC>(dx + row * V + e, d[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (i * TPR + t) * VEC;
    if (e < V) {
#pragma unroll
      for (int j = 0; j < VEC; ++j) cols[grp * V + e + j] = dw[i][j];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < V; e += kBlock(TPR)) {
    float s = 0.f;
#pragma unroll
    for (int g = 0; g < RPB; ++g) s += cols[g * V + e];
    part[(int64_t)blockIdx.x * V + e] = s;
  }
}

// ---------------------------------------------------------- residual norm
// gate: 0 none, 1 a vector of D fp32, 2 a value of type T for every element
template <typename T, typename R, int VEC, int NV, int TPR>
__global__ void __launch_bounds__(kBlock(TPR)) residual_fwd_kernel(
    const T* __restrict__ y, int64_t ldy, const R* __restrict__ res, const float* __restrict__ pw,
    const void* __restrict__ gate, int gmode, float scale, const float* __restrict__ w, int rows, int D, float eps,
    R* __restrict__ hout, T* __restrict__ nout, float* __restrict__ rstd) {
  __shared__ float sm[64];
  int phase = 0;
  constexpr int RPB = kBlock(TPR) / TPR;
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * RPB + threadIdx.x / TPR;
  const bool live = row < rows;
  float a[NV][VEC], b[NV][VEC];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (i * TPR + t) * VEC;
    const bool in = live && e < D;
    if (in) {
      load_vec<T, VEC>(y + row * ldy + e, a[i]);
      load_vec<R, VEC>(res + row * D + e, b[i]);
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) ss += in ? a[i][j] * a[i][j] : 0.f;
  }
  float r1 = 1.f;
  if (pw) r1 = rsqrtf(row_sum<TPR>(ss, sm, phase) / D + eps);
  ss = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = (i * TPR + t) * VEC;
    if (!live || e >= D) continue;
    float f[VEC];
    if (pw) {
      load_vec<float, VEC>(pw + e, f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) a[i][j] = a[i][j] * r1 * f[j];
    }
    if (gmode == 1) load_vec<float, VEC>(static_cast<const float*>(gate) + e, f);
    if (gmode == 2) load_vec<T, VEC>(static_cast<const T*>(gate) + row * D + e, f);
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const float u = gmode ? a[i][j] * f[j] : a[i][j];
      a[i][j] = fmaf(scale, u, b[i][j]);
      ss += a[i][j] * a[i][j];
    }
    store_vec<R, VEC>(hout + row * D + e, a[i]);
  }
  float r2 = 1.f;
  if (w) {
    r2 = rsqrtf(row_sum<TPR>(ss, sm, phase) / D + eps);
    if (live) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = (i * TPR + t) * VEC;
        if (e >= D) continue;
        float f[VEC];
        load_vec<float, VEC>(w + e, f);
#pragma unroll
        for (int j = 0; j < VEC; ++j) a[i][j] = a[i][j] * r2 * f[j];
        store_vec<T, VEC>(nout + row * D + e, a[i]);
      }
    }
  }
  if (rstd && live && t == 0) rstd[2 * row] = r1, rstd[2 * row + 1] = r2;
}

// cols (shared): [RPB][3][D] sums of dweight, dpost_weight, dgate; a thread adds to columns that no other thread of
// its row touches
template <typename T, typename R, int VEC, int NV, int TPR>
__global__ void __launch_bounds__(kBlock(TPR)) residual_bwd_kernel(
    const T* __restrict__ y, int64_t ldy, const R* __restrict__ res, const float* __restrict__ rstd,
    const R* __restrict__ dh, const T* __restrict__ dn, const float* __restrict__ pw, const void* __restrict__ gate,
    int gmode, float scale, const float* __restrict__ w, int rows, int D, T* __restrict__ dy, R* __restrict__ dres,
    T* __restrict__ dgate, float* __restrict__ part) {
  __shared__ float sm[64];
  extern __shared__ float cols[];
  int phase = 0;
  constexpr int RPB = kBlock(TPR) / TPR;
  const int t = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  float* cw = cols + (int64_t)grp * 3 * D;
  float* cp = cw + D;
  float* cg = cp + D;
  for (int e = threadIdx.x; e < RPB * 3 * D; e += kBlock(TPR)) cols[e] = 0.f;
  __syncthreads();
  for (int64_t base = (int64_t)blockIdx.x * RPB; base < rows; base += (int64_t)gridDim.x * RPB) {
    const int64_t row = base + grp;
    const bool live = row < rows;
    const float r1 = live ? rstd[2 * row] : 0.f, r2 = live ? rstd[2 * row + 1] : 0.f;
    float yh[NV][VEC], d[NV][VEC], hh[NV][VEC], aa[NV][VEC];
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * TPR + t) * VEC;
      if (!live || e >= D) continue;
      load_vec<T, VEC>(y + row * ldy + e, yh[i]);
      if (dh) {
        load_vec<R, VEC>(dh + row * D + e, d[i]);
      } else {
#pragma unroll
        for (int j = 0; j < VEC; ++j) d[i][j] = 0.f;
      }
#pragma unroll
      for (int j = 0; j < VEC; ++j) yh[i][j] *= r1;
      if (w) {
        load_vec<R, VEC>(res + row * D + e, hh[i]);
        load_vec<T, VEC>(dn + row * D + e, aa[i]);
      }
    }
    if (w) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = (i * TPR + t) * VEC;
        if (!live || e >= D) continue;
        float p[VEC], f[VEC], wv[VEC];
        if (pw) load_vec<float, VEC>(pw + e, p);
        if (gmode == 1) load_vec<float, VEC>(static_cast<const float*>(gate) + e, f);
        if (gmode == 2) load_vec<T, VEC>(static_cast<const T*>(gate) + row * D + e, f);
        load_vec<float, VEC>(w + e, wv);
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
          float u = pw ? yh[i][j] * p[j] : yh[i][j];
          if (gmode) u *= f[j];
          const float h = fmaf(scale, u, hh[i][j]) * r2;
          hh[i][j] = h;
          cw[e + j] += aa[i][j] * h;
          aa[i][j] *= wv[j];
          s += aa[i][j] * h;
        }
      }
      const float m = row_sum<TPR>(s, sm, phase) / D;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = (i * TPR + t) * VEC;
        if (!live || e >= D) continue;
#pragma unroll
        for (int j = 0; j < VEC; ++j) d[i][j] += r2 * (aa[i][j] - hh[i][j] * m);
      }
    }
    s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * TPR + t) * VEC;
      if (!live || e >= D) continue;
      store_vec<R, VEC>(dres + row * D + e, d[i]);
      float p[VEC], f[VEC], dg[VEC];
      if (pw) load_vec<float, VEC>(pw + e, p);
      if (gmode == 1) load_vec<float, VEC>(static_cast<const float*>(gate) + e, f);
      if (gmode == 2) load_vec<T, VEC>(static_cast<const T*>(gate) + row * D + e, f);
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        float du = scale * d[i][j];
        dg[j] = du * (pw ? yh[i][j] * p[j] : yh[i][j]);
        if (gmode == 1) cg[e + j] += dg[j];
        if (gmode) du *= f[j];
        if (pw) {
          cp[e + j] += du * yh[i][j];
          du *= p[j];
          s += du * yh[i][j];
        }
        d[i][j] = du;
      }
      if (gmode == 2) store_vec<T, VEC>(dgate + row * D + e, dg);
    }
    float m = 0.f;
    if (pw) m = row_sum<TPR>(s, sm, phase) / D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = (i * TPR + t) * VEC;
      if (!live || e >= D) continue;
      if (pw) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) d[i][j] = r1 * (d[i][j] - yh[i][j] * m);
      }
      store_vec<T, VEC>(dy + row * D + e, d[i]);
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < 3 * D; e += kBlock(TPR)) {
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

// Threads a row and vectors a thread: the fewest threads whose registers hold the row at up to 16 elements a thread
// (32 in the widest rows).
struct Shape {
  int vec, tpr, nv;
};

Shape shape_of(int D, int vec) {
  Shape s{vec, 0, 0};
  const int per = vec == 1 ? 8 : 16;
  s.tpr = D <= 16 * vec && vec > 1 ? 16 : (D <= 32 * per ? 32 : (D <= 128 * per ? 128 : 512));
  const int need = (int)ceil_div(D, (int64_t)s.tpr * vec);
  s.nv = 1;
  while (s.nv < need) s.nv *= 2;
  return s;
}

// CTAs of a backward pass: enough to fill the device, each with its own columns
int bwd_blocks(int64_t rows, int rpb, int64_t smem) {
  const int64_t per = smem > 100 * 1024 ? 1 : (smem > 50 * 1024 ? 2 : 4);
  const int64_t need = ceil_div(rows, rpb), most = per * sm_count();
  return (int)(need < most ? need : most);
}

// Above 48 KB, the kernel's static part counted, shared memory has to be asked for.
template <typename K>
bool allow_smem(K kernel, size_t bytes) {
  return bytes <= 47 * 1024 ||
         cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess;
}

// The shapes that shape_of gives, and no others.
#define GDN_NORM_CASE(VEC, NV, TPR, F)                                                                  \
  case NV:                                                                                              \
    if constexpr ((NV) * (VEC) <= ((TPR) == 512 ? 32 : ((VEC) == 1 ? 8 : 16))) F(VEC, NV, TPR);         \
    break;
#define GDN_NORM_NV(VEC, TPR, F)                                                                        \
  switch (s.nv) {                                                                                       \
    GDN_NORM_CASE(VEC, 1, TPR, F)                                                                       \
    GDN_NORM_CASE(VEC, 2, TPR, F)                                                                       \
    GDN_NORM_CASE(VEC, 4, TPR, F)                                                                       \
    GDN_NORM_CASE(VEC, 8, TPR, F)                                                                       \
    GDN_NORM_CASE(VEC, 16, TPR, F)                                                                      \
    GDN_NORM_CASE(VEC, 32, TPR, F)                                                                      \
  }
#define GDN_NORM_TPR(VEC, F)                                                                            \
  switch (s.tpr) {                                                                                      \
    case 16: if constexpr (VEC > 1) F(VEC, 1, 16); break;                                               \
    case 32: GDN_NORM_NV(VEC, 32, F) break;                                                             \
    case 128: GDN_NORM_NV(VEC, 128, F) break;                                                           \
    case 512: GDN_NORM_NV(VEC, 512, F) break;                                                           \
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
  const int rpb = s.tpr <= 32 ? 256 / s.tpr : 1;
  const unsigned grid = (unsigned)ceil_div(rows, rpb);
#define GDN_F(VEC, NV, TPR)                                                                                          \
  gated_fwd_kernel<T, VEC, NV, TPR><<<grid, kBlock(TPR), 0, st>>>(x, ldx, z, ldz, w, rows, H, V, eps, y, rstd)
  if (wide) {
    GDN_NORM_TPR(VW, GDN_F)
  } else {
    GDN_NORM_TPR(1, GDN_F)
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
  const int rpb = s.tpr <= 32 ? 256 / s.tpr : 1;
  const size_t smem = sizeof(float) * rpb * V;
  const int grid = bwd_blocks(rows, rpb, smem);
  bool ok = true;
#define GDN_F(VEC, NV, TPR)                                                                                         \
  {                                                                                                                 \
    auto kern = gated_bwd_kernel<T, VEC, NV, TPR>;                                                                  \
    ok = allow_smem(kern, smem);                                                                                    \
    if (ok) kern<<<grid, kBlock(TPR), smem, st>>>(x, ldx, z, ldz, w, rstd, dy, rows, H, V, dx, dz, part);           \
  }
  if (wide) {
    GDN_NORM_TPR(VW, GDN_F)
  } else {
    GDN_NORM_TPR(1, GDN_F)
  }
#undef GDN_F
  if (!ok || cudaGetLastError() != cudaSuccess) return GDN_ERR_CUDA;
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
  const int rpb = s.tpr <= 32 ? 256 / s.tpr : 1;
  const unsigned grid = (unsigned)ceil_div(rows, rpb);
#define GDN_F(VEC, NV, TPR)                                                                                    \
  residual_fwd_kernel<T, R, VEC, NV, TPR><<<grid, kBlock(TPR), 0, st>>>(y, ldy, res, pw, gate, gmode, scale, w, rows, \
                                                                        D, eps, h, n, rstd)
  if (wide) {
    GDN_NORM_TPR(VW, GDN_F)
  } else {
    GDN_NORM_TPR(1, GDN_F)
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
  const int rpb = s.tpr <= 32 ? 256 / s.tpr : 1;
  const size_t smem = sizeof(float) * rpb * 3 * D;
  const int grid = bwd_blocks(rows, rpb, smem);
  bool ok = true;
#define GDN_F(VEC, NV, TPR)                                                                                        \
  {                                                                                                                \
    auto kern = residual_bwd_kernel<T, R, VEC, NV, TPR>;                                                           \
    ok = allow_smem(kern, smem);                                                                                   \
    if (ok)                                                                                                        \
      kern<<<grid, kBlock(TPR), smem, st>>>(y, ldy, res, rstd, dh, dn, pw, gate, gmode, scale, w, rows, D, dy,     \
                                            dres, gmode == 2 ? static_cast<T*>(dgate) : nullptr, part);            \
  }
  if (wide) {
    GDN_NORM_TPR(VW, GDN_F)
  } else {
    GDN_NORM_TPR(1, GDN_F)
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
size_t gated_norm_bwd_workspace_bytes(int V) { return align_up(sizeof(float) * 4 * (size_t)sm_count() * V); }
size_t residual_norm_bwd_workspace_bytes(int D) { return align_up(sizeof(float) * 4 * (size_t)sm_count() * 3 * D); }

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
