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
// stay in registers), past the run's end for the W-1 tokens whose du it needs.  The
// next four tokens' rows are loaded before the arithmetic of the current ones; four
// CTAs an SM (128 registers) hide the rest best (4 x 8192 tokens, 12288 channels, bf16,
// 2.42 GB: 0.535 ms, 4.5 TB/s; 0.61 with three, 0.96 with five, which spill).
// dweight and dbias are fp32 sums in registers, one partial a run in the
// workspace, added up in order by a second launch (results do not depend on the
// run).  A third launch computes dinitial from each sequence's first W-1 tokens.
#include <type_traits>

#include "gdn_internal.h"
#include "gdn_sm100.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 128;
constexpr int kVec = 4;      // channels a thread, as packed pairs
constexpr int kPairs = kVec / 2;
constexpr int kRun = 256;    // most tokens of a run
constexpr int kU = 4;        // tokens a batch (the next batch loaded ahead)

struct ConvBwdArgs {
  const void *x, *dout, *init, *dfinal;
  const float *weight, *bias;
  const int32_t* cu;
  void *dx, *dinit;
  float *part;   // [runs][D][W + 1]
  float *dweight, *dbias;
  int64_t Ttot, runs;
  int N, Tseq, D, run;   // tokens a run
};

// kVec values of a row, as loaded and as pairs.
template <typename T> using Raw = std::conditional_t<sizeof(T) == 4, float4, uint2>;
__device__ __forceinline__ float4 load_raw(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }
__device__ __forceinline__ uint2 load_raw(const __nv_bfloat16* p) { return __ldg(reinterpret_cast<const uint2*>(p)); }
__device__ __forceinline__ void unpack(float4 q, float2 (&f)[kPairs]) {
  f[0] = make_float2(q.x, q.y), f[1] = make_float2(q.z, q.w);
}
__device__ __forceinline__ void unpack(uint2 q, float2 (&f)[kPairs]) {
  f[0] = make_float2(__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xffff0000u));
  f[1] = make_float2(__uint_as_float(q.y << 16), __uint_as_float(q.y & 0xffff0000u));
}
__device__ __forceinline__ void store_vec(float* p, const float2 (&f)[kPairs]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
}
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float2 (&f)[kPairs]) {
  *reinterpret_cast<uint2*>(p) = make_uint2(sm100::pack_bf16(f[0].x, f[0].y), sm100::pack_bf16(f[1].x, f[1].y));
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

// dout act'(u), a pair
template <bool SILU>
__device__ __forceinline__ float2 du_of(float2 u, float2 g) {
  if constexpr (!SILU) return g;
  const float2 one = make_float2(1.f, 1.f);
  const float2 nl = __fmul2_rn(u, make_float2(-sm100::kLog2e, -sm100::kLog2e));
  const float2 d = __fadd2_rn(make_float2(sm100::ex2_fast(nl.x), sm100::ex2_fast(nl.y)), one);
  const float2 s = make_float2(rcp_fast(d.x), rcp_fast(d.y));
  const float2 r = __fadd2_rn(one, make_float2(-s.x, -s.y));
  return __fmul2_rn(__fmul2_rn(g, s), __ffma2_rn(u, r, one));
}

template <typename T, int W, bool SILU>
__global__ void __launch_bounds__(kThreads, 4) conv1d_bwd_kernel(const ConvBwdArgs a) {
  const int c0 = kVec * (blockIdx.y * kThreads + threadIdx.x);
  if (c0 >= a.D) return;
  const int64_t t0 = (int64_t)blockIdx.x * a.run;
  const int64_t t1 = t0 + a.run < a.Ttot ? t0 + a.run : a.Ttot;
  const int64_t D = a.D;
  const T* __restrict__ x = static_cast<const T*>(a.x);
  const T* __restrict__ dy = static_cast<const T*>(a.dout);
  const T* init = static_cast<const T*>(a.init);
  const T* dfin = static_cast<const T*>(a.dfinal);
  T* __restrict__ dx = static_cast<T*>(a.dx);
  float2 wt[W][kPairs], bs[kPairs], dw[W][kPairs], db[kPairs];
#pragma unroll
  for (int j = 0; j < kPairs; ++j) {
    const int c = c0 + 2 * j;
#pragma unroll
    for (int w = 0; w < W; ++w) {
      wt[w][j] = make_float2(__ldg(a.weight + (int64_t)c * W + w), __ldg(a.weight + (int64_t)(c + 1) * W + w));
      dw[w][j] = make_float2(0.f, 0.f);
    }
    bs[j] = a.bias ? make_float2(__ldg(a.bias + c), __ldg(a.bias + c + 1)) : make_float2(0.f, 0.f);
    db[j] = make_float2(0.f, 0.f);
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
    // ext_{p} .. ext_{p+W-1} of the current token, and du of the last W tokens, channel pairs
    float2 ext[W][kPairs], du[W][kPairs];
#pragma unroll
    for (int i = 0; i < W; ++i) {
#pragma unroll
      for (int j = 0; j < kPairs; ++j) ext[i][j] = du[i][j] = make_float2(0.f, 0.f);
      if (i < W - 1) {
        const int64_t pos = (t - s) - (W - 1) + i;
        if (pos >= 0) unpack(load_raw(x + (s + pos) * D + c0), ext[i]);
        else if (init) unpack(load_raw(init + ((int64_t)n * (W - 1) + (W - 1) + pos) * D + c0), ext[i]);
      }
    }
    // du of the token whose inputs are w0 .. w0[W - 1] (as rows of pairs), and its share of the sums
    auto grad = [&](const float2 (*w0)[kPairs], const float2 (&g)[kPairs], float2 (&o)[kPairs], bool count) {
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        float2 u = bs[j];
#pragma unroll
        for (int w = 0; w < W; ++w) u = __ffma2_rn(wt[w][j], w0[w][j], u);
        o[j] = du_of<SILU>(u, g[j]);
        if (count) {
          db[j] = __fadd2_rn(db[j], o[j]);
#pragma unroll
          for (int w = 0; w < W; ++w) dw[w][j] = __ffma2_rn(o[j], w0[w][j], dw[w][j]);
        }
      }
    };
    auto input = [&](const float2 (*d0)[kPairs], float2 (&o)[kPairs]) {   // dx from du of W tokens
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        o[j] = __fmul2_rn(wt[0][j], d0[W - 1][j]);
#pragma unroll
        for (int w = 1; w < W; ++w) o[j] = __ffma2_rn(wt[w][j], d0[W - 1 - w][j], o[j]);
      }
    };
    int64_t p = t;
    auto step = [&]() {   // one token, anywhere
#pragma unroll
      for (int i = 0; i + 1 < W; ++i)
#pragma unroll
        for (int j = 0; j < kPairs; ++j) du[i][j] = du[i + 1][j];
#pragma unroll
      for (int j = 0; j < kPairs; ++j) du[W - 1][j] = make_float2(0.f, 0.f);
      if (p < e) {
        float2 g[kPairs];
        unpack(load_raw(x + p * D + c0), ext[W - 1]);
        unpack(load_raw(dy + p * D + c0), g);
        grad(ext, g, du[W - 1], p < b);
      }
#pragma unroll
      for (int i = 0; i + 1 < W; ++i)
#pragma unroll
        for (int j = 0; j < kPairs; ++j) ext[i][j] = ext[i + 1][j];
      const int64_t q = p - (W - 1);   // du[i] is that of token q + i
      if (q >= t) {
        float2 o[kPairs];
        input(du, o);
        const int64_t f = q + (W - 1) - e;   // row of the final state that token q is
        if (dfin && f >= 0) {
          float2 r[kPairs];
          unpack(load_raw(dfin + ((int64_t)n * (W - 1) + f) * D + c0), r);
#pragma unroll
          for (int j = 0; j < kPairs; ++j) o[j] = __fadd2_rn(o[j], r[j]);
        }
        store_vec(dx + q * D + c0, o);
      }
      ++p;
    };
    for (; p < b + W - 1 && p < t + W - 1;) step();
    // kU tokens at a time, the next ones' rows on their way
    if (p + kU <= b) {
      Raw<T> rx[kU], ry[kU];
#pragma unroll
      for (int u = 0; u < kU; ++u) rx[u] = load_raw(x + (p + u) * D + c0), ry[u] = load_raw(dy + (p + u) * D + c0);
      for (;;) {
        const bool more = p + 2 * kU <= b;
        // inputs and du of W - 1 tokens before, and of these; ext[0 ..] and du[1 ..] hold the former
        float2 ew[kU + W - 1][kPairs], dv[kU + W - 1][kPairs], g[kU][kPairs];
#pragma unroll
        for (int i = 0; i < W - 1; ++i)
#pragma unroll
          for (int j = 0; j < kPairs; ++j) ew[i][j] = ext[i][j], dv[i][j] = du[i + 1][j];
#pragma unroll
        for (int u = 0; u < kU; ++u) unpack(rx[u], ew[W - 1 + u]), unpack(ry[u], g[u]);
        if (more) {
#pragma unroll
          for (int u = 0; u < kU; ++u)
            rx[u] = load_raw(x + (p + kU + u) * D + c0), ry[u] = load_raw(dy + (p + kU + u) * D + c0);
        }
#pragma unroll
        for (int u = 0; u < kU; ++u) {
          grad(ew + u, g[u], dv[W - 1 + u], true);
          float2 o[kPairs];
          input(dv + u, o);
          store_vec(dx + (p + u - (W - 1)) * D + c0, o);
        }
#pragma unroll
        for (int i = 0; i < W - 1; ++i)
#pragma unroll
          for (int j = 0; j < kPairs; ++j) ext[i][j] = ew[kU + i][j], du[i + 1][j] = dv[kU + i][j];
        p += kU;
        if (!more) break;
      }
    }
    for (; p < b + W - 1;) step();
    t = b;
  }
  float* part = a.part + ((int64_t)blockIdx.x * D + c0) * (W + 1);
#pragma unroll
  for (int j = 0; j < kPairs; ++j) {
#pragma unroll
    for (int w = 0; w < W; ++w) {
      part[2 * j * (W + 1) + w] = dw[w][j].x;
      part[(2 * j + 1) * (W + 1) + w] = dw[w][j].y;
    }
    part[2 * j * (W + 1) + W] = db[j].x;
    part[(2 * j + 1) * (W + 1) + W] = db[j].y;
  }
}

// dweight and dbias: the runs' partials, eight threads to a value (every eighth run
// each, in order), their sums in order.
template <int W>
__global__ void __launch_bounds__(256) conv1d_bwd_params_kernel(const ConvBwdArgs a) {
  __shared__ float sum[8][32];
  const int v = threadIdx.x & 31, k = threadIdx.x >> 5;
  const int64_t i = (int64_t)blockIdx.x * 32 + v, total = (int64_t)a.D * (W + 1);
  float s = 0.f;
  if (i < total) {
#pragma unroll 4
    for (int64_t r = k; r < a.runs; r += 8) s += a.part[r * total + i];
  }
  sum[k][v] = s;
  __syncthreads();
  if (k != 0 || i >= total) return;
#pragma unroll
  for (int j = 1; j < 8; ++j) s += sum[j][v];
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
  float2 ext[2 * W - 2][kPairs], du[W - 1][kPairs], wt[W][kPairs];
#pragma unroll
  for (int j = 0; j < kPairs; ++j)
#pragma unroll
    for (int w = 0; w < W; ++w)
      wt[w][j] = make_float2(a.weight[(int64_t)(c0 + 2 * j) * W + w], a.weight[(int64_t)(c0 + 2 * j + 1) * W + w]);
#pragma unroll
  for (int i = 0; i < 2 * W - 2; ++i) {
#pragma unroll
    for (int j = 0; j < kPairs; ++j) ext[i][j] = make_float2(0.f, 0.f);
    if (i >= W - 1 ? i - (W - 1) < L : false) unpack(load_raw(x + (s + i - (W - 1)) * D + c0), ext[i]);
    else if (i < W - 1 && init) unpack(load_raw(init + ((int64_t)n * (W - 1) + i) * D + c0), ext[i]);
  }
#pragma unroll
  for (int p = 0; p < W - 1; ++p) {
#pragma unroll
    for (int j = 0; j < kPairs; ++j) du[p][j] = make_float2(0.f, 0.f);
    if (p < L) {
      unpack(load_raw(dy + (s + p) * D + c0), du[p]);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) {
        float2 u = a.bias ? make_float2(a.bias[c0 + 2 * j], a.bias[c0 + 2 * j + 1]) : make_float2(0.f, 0.f);
#pragma unroll
        for (int w = 0; w < W; ++w) u = __ffma2_rn(wt[w][j], ext[p + w][j], u);
        du[p][j] = du_of<SILU>(u, du[p][j]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    float2 o[kPairs];
#pragma unroll
    for (int j = 0; j < kPairs; ++j) {
      o[j] = make_float2(0.f, 0.f);
#pragma unroll
      for (int w = 0; w <= i; ++w) o[j] = __ffma2_rn(wt[w][j], du[i - w][j], o[j]);
    }
    if (dfin && i >= L) {
      float2 r[kPairs];
      unpack(load_raw(dfin + ((int64_t)n * (W - 1) + i - L) * D + c0), r);
#pragma unroll
      for (int j = 0; j < kPairs; ++j) o[j] = __fadd2_rn(o[j], r[j]);
    }
    store_vec(out + i * D, o);
  }
}

template <typename T, int W, bool SILU>
void launch_conv_bwd(const ConvBwdArgs& a, cudaStream_t s) {
  const unsigned cvb = (unsigned)ceil_div(a.D, kVec * kThreads);
  if (a.runs > 0) conv1d_bwd_kernel<T, W, SILU><<<dim3((unsigned)a.runs, cvb), kThreads, 0, s>>>(a);
  conv1d_bwd_params_kernel<W><<<(unsigned)ceil_div((int64_t)a.D * (W + 1), 32), 256, 0, s>>>(a);
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

namespace {
// Long runs spread their start and the W-1 tokens behind them over more tokens;
// shorter ones (down to 32) while fewer than eight CTAs an SM would run.
int run_length(int64_t tokens, int D) {
  int run = kRun;
  while (run > 32 && ceil_div(tokens, run) * ceil_div(D, kVec * kThreads) < 8 * sm_count()) run /= 2;
  return run;
}
}  // namespace

size_t conv1d_bwd_workspace_bytes(int64_t tokens, int D, int W) {
  return align_up(sizeof(float) * (size_t)ceil_div(tokens, run_length(tokens, D)) * D * (W + 1)) + kAlign;
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
  a.run = run_length(a.Ttot, D);
  a.runs = ceil_div(a.Ttot, a.run);
  a.N = N, a.Tseq = T, a.D = D;
  if (dt == GDN_F32) silu_act ? by_width<float, true>(a, W, s) : by_width<float, false>(a, W, s);
  else silu_act ? by_width<__nv_bfloat16, true>(a, W, s) : by_width<__nv_bfloat16, false>(a, W, s);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace gdn
