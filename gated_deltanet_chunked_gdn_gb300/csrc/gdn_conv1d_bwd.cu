// gdn_conv1d_bwd.cu -- backward of the causal depthwise convolution
// (gdn_conv1d.cu).  With ext = [W-1 initial inputs ; x_0 .. x_{L-1}] and, per
// channel,
//     u_p = bias + sum_w weight[w] ext_{p+w},   y_p = act(u_p),
//     final state = ext_L .. ext_{L+W-2},
// the gradients of <dout, y> + <dfinal, final state> are
//     du_p       = dout_p act'(u_p)                     (SiLU: s (1 + u (1 - s)), s = sigmoid(u))
//     dext_j     = sum_w weight[w] du_{j-w} (0 <= j-w < L) + dfinal_{j-L} (j >= L)
//     dx_p       = dext_{p+W-1},   dinitial_j = dext_j (j < W-1)
//     dweight[w] = sum_p du_p ext_{p+w},   dbias = sum_p du_p.
//
// Bound by HBM traffic: x and dout read once, dx written once.  A thread owns
// kVec neighbouring channels over a run of tokens: it walks forward through x and
// dout, recomputes u, and writes dx W-1 tokens behind (the last W-1 values of du
// stay in registers), past the run's end for the W-1 tokens whose du it needs.
// dweight and dbias are fp32 sums in registers, one partial a run in the
// workspace, added up in order by a second launch (results do not depend on the
// run).  A third launch computes dinitial from each sequence's first W-1 tokens.
#include "gdn_internal.h"
#include "gdn_sm100.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kVec = 4;      // channels a thread
constexpr int kRun = 256;    // tokens a run

struct ConvBwdArgs {
  const void *x, *dout, *init, *dfinal;
  const float *weight, *bias;
  const int32_t* cu;
  void *dx, *dinit;
  float *part;   // [runs][D][W + 1]
  float *dweight, *dbias;
  int64_t Ttot, runs;
  int N, Tseq, D;
};

template <typename T>
__device__ __forceinline__ void load_vec(const T* p, float (&f)[kVec]);
template <>
__device__ __forceinline__ void load_vec<float>(const float* p, float (&f)[kVec]) {
  const float4 q = __ldg(reinterpret_cast<const float4*>(p));
  f[0] = q.x, f[1] = q.y, f[2] = q.z, f[3] = q.w;
}
template <>
__device__ __forceinline__ void load_vec<__nv_bfloat16>(const __nv_bfloat16* p, float (&f)[kVec]) {
  const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
  f[0] = __uint_as_float(q.x << 16), f[1] = __uint_as_float(q.x & 0xffff0000u);
  f[2] = __uint_as_float(q.y << 16), f[3] = __uint_as_float(q.y & 0xffff0000u);
}
__device__ __forceinline__ void store_vec(float* p, const float (&f)[kVec]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
}
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&f)[kVec]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(sm100::pack_bf16(f[0], f[1]), sm100::pack_bf16(f[2], f[3]));
}

// Sequence n's token range [s, e); false for malformed cu_seqlens entries.
__device__ __forceinline__ bool bounds(const ConvBwdArgs& a, int n, int64_t& s, int64_t& e) {
  s = a.cu ? a.cu[n] : (int64_t)n * a.Tseq;
  e = a.cu ? a.cu[n + 1] : s + a.Tseq;
  return 0 <= s && s <= e && e <= a.Ttot;
}

__device__ __forceinline__ float rcp_fast(float y) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
  return r;
}

// dout act'(u)
template <bool SILU>
__device__ __forceinline__ float du_of(float u, float g) {
  if (!SILU) return g;
  const float s = rcp_fast(1.f + sm100::ex2_fast(-sm100::kLog2e * u));
  return g * s * fmaf(u, 1.f - s, 1.f);
}

template <typename T, int W, bool SILU>
__global__ void __launch_bounds__(kThreads) conv1d_bwd_kernel(const ConvBwdArgs a) {
  const int c0 = kVec * (blockIdx.y * kThreads + threadIdx.x);
  if (c0 >= a.D) return;
  const int64_t t0 = (int64_t)blockIdx.x * kRun;
  const int64_t t1 = t0 + kRun < a.Ttot ? t0 + kRun : a.Ttot;
  const int64_t D = a.D;
  const T* __restrict__ x = static_cast<const T*>(a.x);
  const T* __restrict__ dy = static_cast<const T*>(a.dout);
  const T* init = static_cast<const T*>(a.init);
  const T* dfin = static_cast<const T*>(a.dfinal);
  T* __restrict__ dx = static_cast<T*>(a.dx);
  float wt[W][kVec], bs[kVec], dw[W][kVec], db[kVec];
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
#pragma unroll
    for (int w = 0; w < W; ++w) wt[w][j] = __ldg(a.weight + (int64_t)(c0 + j) * W + w), dw[w][j] = 0.f;
    bs[j] = a.bias ? __ldg(a.bias + c0 + j) : 0.f;
    db[j] = 0.f;
  }
  int n = 0;
  if (a.cu) {   // the last sequence that starts at or before t0
    int lo = 0, hi = a.N - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.cu[mid] <= t0) lo = mid; else hi = mid - 1;
    }
    n = lo;
  } else {
    n = (int)(t0 / a.Tseq);
  }
  int64_t t = t0;
  while (t < t1 && n < a.N) {
    int64_t s, e;
    if (!bounds(a, n, s, e) || e <= t) {   // malformed, empty or already passed
      ++n;
      continue;
    }
    if (s > t) {   // tokens that no sequence covers
      t = s;
      continue;
    }
    const int64_t b = e < t1 ? e : t1;   // this run's tokens of sequence n: [t, b)
    float ext[W][kVec], du[W][kVec];     // ext_{p} .. ext_{p+W-1}; du of the last W tokens
#pragma unroll
    for (int i = 0; i < W; ++i) {
#pragma unroll
      for (int j = 0; j < kVec; ++j) ext[i][j] = 0.f, du[i][j] = 0.f;
      if (i < W - 1) {
        const int64_t pos = (t - s) - (W - 1) + i;
        if (pos >= 0) load_vec<T>(x + (s + pos) * D + c0, ext[i]);
        else if (init) load_vec<T>(init + ((int64_t)n * (W - 1) + (W - 1) + pos) * D + c0, ext[i]);
      }
    }
    for (int64_t p = t; p < b + W - 1; ++p) {
#pragma unroll
      for (int i = 0; i + 1 < W; ++i)
#pragma unroll
        for (int j = 0; j < kVec; ++j) du[i][j] = du[i + 1][j];
      float g[kVec];
#pragma unroll
      for (int j = 0; j < kVec; ++j) g[j] = 0.f;
      if (p < e) {
        load_vec<T>(x + p * D + c0, ext[W - 1]);
        load_vec<T>(dy + p * D + c0, g);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          float u = bs[j];
#pragma unroll
          for (int w = 0; w < W; ++w) u = fmaf(wt[w][j], ext[w][j], u);
          g[j] = du_of<SILU>(u, g[j]);
        }
        if (p < b) {
#pragma unroll
          for (int j = 0; j < kVec; ++j) {
            db[j] += g[j];
#pragma unroll
            for (int w = 0; w < W; ++w) dw[w][j] = fmaf(g[j], ext[w][j], dw[w][j]);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kVec; ++j) du[W - 1][j] = g[j];
#pragma unroll
      for (int i = 0; i + 1 < W; ++i)
#pragma unroll
        for (int j = 0; j < kVec; ++j) ext[i][j] = ext[i + 1][j];
      const int64_t q = p - (W - 1);   // du[i] is that of token q + i
      if (q >= t) {
        float o[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          o[j] = 0.f;
#pragma unroll
          for (int w = 0; w < W; ++w) o[j] = fmaf(wt[w][j], du[W - 1 - w][j], o[j]);
        }
        const int64_t f = q + (W - 1) - e;   // row of the final state that token q is
        if (dfin && f >= 0) {
          float r[kVec];
          load_vec<T>(dfin + ((int64_t)n * (W - 1) + f) * D + c0, r);
#pragma unroll
          for (int j = 0; j < kVec; ++j) o[j] += r[j];
        }
        store_vec(dx + q * D + c0, o);
      }
    }
    t = b;
  }
  float* part = a.part + ((int64_t)blockIdx.x * D + c0) * (W + 1);
#pragma unroll
  for (int j = 0; j < kVec; ++j) {
#pragma unroll
    for (int w = 0; w < W; ++w) part[j * (W + 1) + w] = dw[w][j];
    part[j * (W + 1) + W] = db[j];
  }
}

// dweight and dbias: the runs' partials in order, a thread per value.
template <int W>
__global__ void __launch_bounds__(256) conv1d_bwd_params_kernel(const ConvBwdArgs a) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, total = (int64_t)a.D * (W + 1);
  if (i >= total) return;
  float s = 0.f;
  for (int64_t r = 0; r < a.runs; ++r) s += a.part[r * total + i];
  const int64_t d = i / (W + 1);
  const int w = (int)(i % (W + 1));
  if (w < W) a.dweight[d * W + w] = s;
  else if (a.dbias) a.dbias[d] = s;
}

// dinitial of sequence n.
template <typename T, int W, bool SILU>
__global__ void __launch_bounds__(kThreads) conv1d_bwd_init_kernel(const ConvBwdArgs a) {
  const int n = blockIdx.x, c0 = kVec * (blockIdx.y * kThreads + threadIdx.x);
  if (c0 >= a.D) return;
  int64_t s, e;
  if (!bounds(a, n, s, e)) return;
  const int64_t L = e - s, D = a.D;
  const T* x = static_cast<const T*>(a.x);
  const T* dy = static_cast<const T*>(a.dout);
  const T* init = static_cast<const T*>(a.init);
  const T* dfin = static_cast<const T*>(a.dfinal);
  T* out = static_cast<T*>(a.dinit) + (int64_t)n * (W - 1) * D + c0;
  float ext[2 * W - 2][kVec], du[W - 1][kVec];
#pragma unroll
  for (int i = 0; i < 2 * W - 2; ++i) {
#pragma unroll
    for (int j = 0; j < kVec; ++j) ext[i][j] = 0.f;
    if (i >= W - 1 ? i - (W - 1) < L : false) load_vec<T>(x + (s + i - (W - 1)) * D + c0, ext[i]);
    else if (i < W - 1 && init) load_vec<T>(init + ((int64_t)n * (W - 1) + i) * D + c0, ext[i]);
  }
#pragma unroll
  for (int p = 0; p < W - 1; ++p) {
#pragma unroll
    for (int j = 0; j < kVec; ++j) du[p][j] = 0.f;
    if (p < L) {
      load_vec<T>(dy + (s + p) * D + c0, du[p]);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        float u = a.bias ? a.bias[c0 + j] : 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) u = fmaf(a.weight[(int64_t)(c0 + j) * W + w], ext[p + w][j], u);
        du[p][j] = du_of<SILU>(u, du[p][j]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    float o[kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
      o[j] = 0.f;
#pragma unroll
      for (int w = 0; w <= i; ++w) o[j] = fmaf(a.weight[(int64_t)(c0 + j) * W + w], du[i - w][j], o[j]);
    }
    if (dfin && i >= L) {
      float r[kVec];
      load_vec<T>(dfin + ((int64_t)n * (W - 1) + i - L) * D + c0, r);
#pragma unroll
      for (int j = 0; j < kVec; ++j) o[j] += r[j];
    }
    store_vec(out + i * D, o);
  }
}

template <typename T, int W, bool SILU>
void launch_conv_bwd(const ConvBwdArgs& a, cudaStream_t s) {
  const unsigned cvb = (unsigned)ceil_div(a.D, kVec * kThreads);
  if (a.runs > 0) conv1d_bwd_kernel<T, W, SILU><<<dim3((unsigned)a.runs, cvb), kThreads, 0, s>>>(a);
  conv1d_bwd_params_kernel<W><<<(unsigned)ceil_div((int64_t)a.D * (W + 1), 256), 256, 0, s>>>(a);
  if constexpr (W > 1) {
    if (a.dinit && a.N > 0) conv1d_bwd_init_kernel<T, W, SILU><<<dim3(a.N, cvb), kThreads, 0, s>>>(a);
  }
}

template <typename T, bool SILU>
void by_width(const ConvBwdArgs& a, int W, cudaStream_t s) {
  switch (W) {
    case 1: launch_conv_bwd<T, 1, SILU>(a, s); break;
    case 2: launch_conv_bwd<T, 2, SILU>(a, s); break;
    case 3: launch_conv_bwd<T, 3, SILU>(a, s); break;
    default: launch_conv_bwd<T, 4, SILU>(a, s); break;
  }
}

}  // namespace

size_t conv1d_bwd_workspace_bytes(int64_t tokens, int D, int W) {
  return align_up(sizeof(float) * (size_t)ceil_div(tokens, kRun) * D * (W + 1)) + kAlign;
}

gdn_status run_causal_conv1d_bwd(const void* x, const float* weight, const float* bias, int W,
                                 const void* initial_state, const int32_t* cu, int N, int B, int T, int D,
                                 gdn_dtype dt, bool silu_act, const void* dout, const void* dfinal_state, void* dx,
                                 float* dweight, float* dbias, void* dinitial_state, void* ws, cudaStream_t s) {
  ConvBwdArgs a;
  a.x = x, a.dout = dout;
  a.init = W > 1 ? initial_state : nullptr;
  a.dfinal = W > 1 ? dfinal_state : nullptr;
  a.dinit = dinitial_state;
  a.weight = weight, a.bias = bias, a.cu = cu;
  a.dx = dx, a.dweight = dweight, a.dbias = dbias;
  a.part = static_cast<float*>(ws);
  a.Ttot = (int64_t)B * T;
  a.runs = ceil_div(a.Ttot, kRun);
  a.N = N, a.Tseq = T, a.D = D;
  if (dt == GDN_F32) silu_act ? by_width<float, true>(a, W, s) : by_width<float, false>(a, W, s);
  else silu_act ? by_width<__nv_bfloat16, true>(a, W, s) : by_width<__nv_bfloat16, false>(a, W, s);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace gdn
