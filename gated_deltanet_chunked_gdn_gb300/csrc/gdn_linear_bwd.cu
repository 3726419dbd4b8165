// gdn_linear_bwd.cu -- backward of decayed linear attention, in fp32 arithmetic for every type and head dim.
//
// With S0 the state before a chunk, G the adjoint of the state behind it, M_ij = e^{b_i - b_j} (j <= i), w_j =
// e^{b_last - b_j}:
//
//   P = scale M * (q k^T),  W = scale M * (do v^T),  A = W * (q k^T)       (elementwise)
//   dq = W k + scale e^{b} (do S0^T)      dk = W^T q + w (v G^T)      dv = P^T do + w (k G)
//   G before the chunk = e^{b_last} G + scale sum_i e^{b_i} q_i do_i^T
//
// dg_s is the sum over the pairs of tokens j < s <= i that the decay at s lies between: within the chunk the suffix sums
// of (row - column sums of A), from outside into the chunk those of q_i . (scale e^{b_i} S0 do_i), out of it the prefix
// sums of k_j . (w_j G v_j), past it e^{b_last} <G, S0>.  Every chunk forms its own, so that no rounding is carried from
// chunk to chunk.  Heads that share q and k write their dq and dk to the workspace in fp32; a launch behind adds them
// in order.
#include "gdn_linear_simt.cuh"

namespace gdn {
namespace lin {
namespace {

// Sum over the 16 threads of a row of the 16 x 16 grid (half a warp).
__device__ __forceinline__ float row16(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Gradients of one chunk of one value head.
template <typename T, typename TG>
__global__ void __launch_bounds__(kThreads) grads_kernel(
    const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, const T* __restrict__ dout, Shape d,
    const float* __restrict__ g, Pieces pc, float scale, const float* __restrict__ S0, const float* __restrict__ G,
    TG* __restrict__ dq, TG* __restrict__ dk, T* __restrict__ dv, float* __restrict__ dg) {
  extern __shared__ __align__(16) float sm[];
  float* As = sm;                      // operands of the running product
  float* Bs = As + kC * kLd;
  float* Pn = Bs + kC * kLd;           // P [i][j]
  float* Wn = Pn + kC * kLd;           // W [i][j]
  float* Wt = Wn + kC * kLd;           // W [j][i]
  float* hi = Wt + kC * kLd;
  float* lo = hi + kC;
  float* up = lo + kC;                 // scale e^{b_i}
  float* down = up + kC;               // e^{b_last - b_j}
  float* row = down + kC;              // row sums of A, then with what comes into the chunk
  float* out = row + kC;               // what leaves the chunk
  float* colp = out + kC;              // [16][64] column sums of A, by row group
  float* red = colp + 16 * kC;         // [8] warps' parts of <G, S0>
  const int c = blockIdx.x / d.Hv, h = blockIdx.x % d.Hv, hq = h / (d.Hv / d.Hqk);
  const Piece p = piece_of(pc, c);
  if (!p.ok) return;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  if (tid < 32) chunk_sums(g + (d.g_per_head ? h : p.tok0 * d.Hv + h), d.g_per_head ? 0 : d.Hv, p.len, tid, hi, lo);
  __syncthreads();
  if (tid < kC) {
    up[tid] = scale * expf(hi[tid] + lo[tid]);
    down[tid] = expf((hi[kC - 1] - hi[tid]) + (lo[kC - 1] - lo[tid]));
  }
  const T* qp = q + p.tok0 * d.ldq + (int64_t)hq * d.K;
  const T* kp = k + p.tok0 * d.ldk + (int64_t)hq * d.K;
  const T* vp = v + p.tok0 * d.ldv + (int64_t)h * d.V;
  const int64_t ldo = (int64_t)d.Hv * d.V;
  const T* op = dout + p.tok0 * ldo + (int64_t)h * d.V;
  float acc[4][4], qk[4][4];
  zero(qk);
  for (int d0 = 0; d0 < d.K; d0 += kC) {
    __syncthreads();
    load_t(As, qp + d0, d.ldq, p.len, nullptr);
    load_t(Bs, kp + d0, d.ldk, p.len, nullptr);
    __syncthreads();
    fma_tile(qk, As, Bs, ty, tx);
  }
  zero(acc);
  for (int e0 = 0; e0 < d.V; e0 += kC) {
    __syncthreads();
    load_t(As, op + e0, ldo, p.len, nullptr);
    load_t(Bs, vp + e0, d.ldv, p.len, nullptr);
    __syncthreads();
    fma_tile(acc, As, Bs, ty, tx);
  }
  {
    float rs[4] = {0.f, 0.f, 0.f, 0.f}, cs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = 4 * ty + r, j = 4 * tx + u;
        const float m = j <= i ? scale * expf((hi[i] - hi[j]) + (lo[i] - lo[j])) : 0.f;
        const float pv = j <= i ? m * qk[r][u] : 0.f, wv = j <= i ? m * acc[r][u] : 0.f;
        const float a = j < i ? wv * qk[r][u] : 0.f;   // a token with itself has no decay between
        Pn[i * kLd + j] = pv;
        Wn[i * kLd + j] = wv;
        Wt[j * kLd + i] = wv;
        rs[r] += a;
        cs[u] += a;
      }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      rs[r] = row16(rs[r]);
      if (tx == 0) row[4 * ty + r] = rs[r], out[4 * ty + r] = 0.f;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) colp[ty * kC + 4 * tx + u] = cs[u];
  }
  const float* S = S0 + ((int64_t)c * d.Hv + h) * d.K * d.V;
  const float* A = G + ((int64_t)c * d.Hv + h) * d.K * d.V;
  // dv = P^T do + w (k G)
  for (int e0 = 0; e0 < d.V; e0 += kC) {
    zero(acc);
    __syncthreads();
    load_n(Bs, op + e0, ldo, p.len, nullptr);
    __syncthreads();
    fma_tile(acc, Pn, Bs, ty, tx);
    for (int d0 = 0; d0 < d.K; d0 += kC) {
      __syncthreads();
      load_t(As, kp + d0, d.ldk, p.len, down);
      load_n(Bs, A + (int64_t)d0 * d.V + e0, d.V, kC, nullptr);
      __syncthreads();
      fma_tile(acc, As, Bs, ty, tx);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int j = 4 * ty + r;
      if (j < p.len) store4(dv + (p.tok0 + j) * ldo + (int64_t)h * d.V + e0 + 4 * tx, acc[r]);
    }
  }
  // dq = W k + scale e^b (do S0^T),  dk = W^T q + w (v G^T); TG rows: value heads, or the q/k heads themselves
  const int64_t ldg = (int64_t)d.Hv * d.K;
  float gs = 0.f;   // <G, S0>
  for (int d0 = 0; d0 < d.K; d0 += kC) {
    zero(acc);
    for (int e0 = 0; e0 < d.V; e0 += kC) {
      __syncthreads();
      load_t(As, op + e0, ldo, p.len, up);
      load_t(Bs, S + (int64_t)d0 * d.V + e0, d.V, kC, nullptr);
      __syncthreads();
      fma_tile(acc, As, Bs, ty, tx);
#pragma unroll
      for (int r = ty; r < kC; r += 16) {   // Bs is [e][d]
        const float4 s4 = *reinterpret_cast<const float4*>(Bs + r * kLd + 4 * tx);
        const float sv[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
        for (int u = 0; u < 4; ++u) gs = fmaf(sv[u], A[(int64_t)(d0 + 4 * tx + u) * d.V + e0 + r], gs);
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = 4 * ty + r;
      float s = 0.f;
      if (i < p.len) {
        const float4 x = load4(qp + i * d.ldq + d0 + 4 * tx);
        s = x.x * acc[r][0] + x.y * acc[r][1] + x.z * acc[r][2] + x.w * acc[r][3];
      }
      s = row16(s);
      if (tx == 0) row[i] += s;
    }
    __syncthreads();
    load_n(Bs, kp + d0, d.ldk, p.len, nullptr);
    __syncthreads();
    fma_tile(acc, Wt, Bs, ty, tx);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int i = 4 * ty + r;
      if (i < p.len) store4(dq + (p.tok0 + i) * ldg + (int64_t)h * d.K + d0 + 4 * tx, acc[r]);
    }
    zero(acc);
    for (int e0 = 0; e0 < d.V; e0 += kC) {
      __syncthreads();
      load_t(As, vp + e0, d.ldv, p.len, down);
      load_t(Bs, A + (int64_t)d0 * d.V + e0, d.V, kC, nullptr);
      __syncthreads();
      fma_tile(acc, As, Bs, ty, tx);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int j = 4 * ty + r;
      float s = 0.f;
      if (j < p.len) {
        const float4 x = load4(kp + j * d.ldk + d0 + 4 * tx);
        s = x.x * acc[r][0] + x.y * acc[r][1] + x.z * acc[r][2] + x.w * acc[r][3];
      }
      s = row16(s);
      if (tx == 0) out[j] += s;
    }
    __syncthreads();
    load_n(Bs, qp + d0, d.ldq, p.len, nullptr);
    __syncthreads();
    fma_tile(acc, Wn, Bs, ty, tx);
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int j = 4 * ty + r;
      if (j < p.len) store4(dk + (p.tok0 + j) * ldg + (int64_t)h * d.K + d0 + 4 * tx, acc[r]);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) gs += __shfl_xor_sync(0xffffffffu, gs, o);
  if ((tid & 31) == 0) red[tid >> 5] = gs;
  __syncthreads();
  if (tid < kC) {
    float s = 0.f;
#pragma unroll
    for (int r = 0; r < 16; ++r) s += colp[r * kC + tid];
    row[tid] -= s;
  }
  __syncthreads();
  if (tid < 32) {
    // dg_s = sum_{i >= s} row_i + sum_{j < s} out_j + e^{b_last} <G, S0>
    double past = 0.0;
#pragma unroll
    for (int w = 0; w < 8; ++w) past += red[w];
    past *= (double)expf(hi[kC - 1] + lo[kC - 1]);
    const int r = 2 * tid;
    const double ra = row[r], rb = row[r + 1], oa = out[r], ob = out[r + 1];
    double suf = ra + rb, pre = oa + ob;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double a = __shfl_down_sync(0xffffffffu, suf, o), b = __shfl_up_sync(0xffffffffu, pre, o);
      if (tid + o < 32) suf += a;
      if (tid >= o) pre += b;
    }
    pre -= oa + ob;
    const double x0 = suf + pre + past, x1 = suf - ra + pre + oa + past;
    if (d.g_per_head) {
      double s = (r < p.len ? x0 : 0.0) + (r + 1 < p.len ? x1 : 0.0);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (tid == 0) dg[(int64_t)c * d.Hv + h] = (float)s;
    } else {
      float* gp = dg + p.tok0 * d.Hv + h;
      if (r < p.len) gp[(int64_t)r * d.Hv] = (float)x0;
      if (r + 1 < p.len) gp[(int64_t)(r + 1) * d.Hv] = (float)x1;
    }
  }
}

// dg of fixed decays: the chunks' sums of one head, in a fixed order
__global__ void __launch_bounds__(256) head_decays_kernel(const float* __restrict__ part, int Hv, int most,
                                                          const int32_t* __restrict__ nc, float* __restrict__ dg) {
  __shared__ double sm[256];
  const int h = blockIdx.x, n = nc ? *nc : most;
  if (n < 0) return;
  double s = 0.0;
  for (int c = threadIdx.x; c < n; c += 256) s += part[(int64_t)c * Hv + h];
  sm[threadIdx.x] = s;
  __syncthreads();
  for (int o = 128; o > 0; o >>= 1) {
    if (threadIdx.x < o) sm[threadIdx.x] += sm[threadIdx.x + o];
    __syncthreads();
  }
  if (threadIdx.x == 0) dg[h] = (float)sm[0];
}

constexpr size_t kGradSmem = sizeof(float) * (5 * kC * kLd + 6 * kC + 16 * kC + 8);

struct Layout {
  size_t tables, total, part, states, adjoints, dq, dk, end;
};

Layout layout_of(const gdn_linear_problem& p) {
  const size_t cells = (size_t)pieces_max(p, kC) * p.Hv;
  Layout L;
  L.tables = kAlign;
  L.total = L.tables + pieces_bytes(p, kC);
  L.part = L.total + align_up(4 * cells);
  L.states = L.part + (p.g_per_head ? align_up(4 * cells) : 0);
  L.adjoints = L.states + 4 * cells * p.K * p.V;
  L.dq = L.adjoints + 4 * cells * p.K * p.V;
  const size_t own = p.Hv == p.Hqk ? 0 : align_up(4 * (size_t)p.B * p.T * p.Hv * p.K);
  L.dk = L.dq + own;
  L.end = L.dk + own;
  return L;
}

template <typename T>
gdn_status bwd_t(const gdn_linear_problem& p, const T* q, const T* k, const T* v, const float* g, float scale,
                 const float* h0, const T* dout, const float* dht, T* dq, T* dk, T* dv, float* dg, float* dh0,
                 const Pieces& pc, const Layout& L, uint8_t* ws, cudaStream_t s) {
  const Shape d = shape_of(p);
  const int most = pieces_max(p, kC);
  int32_t* status = reinterpret_cast<int32_t*>(ws);
  float* total = reinterpret_cast<float*>(ws + L.total);
  float* S = reinterpret_cast<float*>(ws + L.states);
  float* G = reinterpret_cast<float*>(ws + L.adjoints);
  gdn_status st = launch_states<T, false>(d, k, p.ld_k, v, p.ld_v, g, pc, most, 1.f, S, total, status, s);
  if (st == GDN_OK) st = launch_sums<false>(d, pc, p.N, total, h0, S, nullptr, nullptr, 0, s);
  if (st == GDN_OK)
    st = launch_states<T, true>(d, q, p.ld_q, dout, (int64_t)p.Hv * p.V, g, pc, most, scale, G, total, status, s);
  if (st == GDN_OK) st = launch_sums<true>(d, pc, p.N, total, dht, G, dh0, nullptr, 0, s);
  if (st != GDN_OK) return st;
  float* part = reinterpret_cast<float*>(ws + L.part);
  const bool shared = p.Hv != p.Hqk;
  if (most > 0) {
    const unsigned grid = (unsigned)((int64_t)most * p.Hv);
    float* dgp = p.g_per_head ? part : dg;
    auto run = [&](auto kern, auto* a, auto* b) {
      if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kGradSmem) != cudaSuccess)
        return GDN_ERR_CUDA;
      kern<<<grid, kThreads, kGradSmem, s>>>(q, k, v, dout, d, g, pc, scale, S, G, a, b, dv, dgp);
      return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
    };
    if (shared)
      st = run(grads_kernel<T, float>, reinterpret_cast<float*>(ws + L.dq), reinterpret_cast<float*>(ws + L.dk));
    else
      st = run(grads_kernel<T, T>, dq, dk);
    if (st != GDN_OK) return st;
  }
  if (shared && most > 0) {
    st = launch_heads<T>(p, reinterpret_cast<const float*>(ws + L.dq), pc.nc, dq, s);
    if (st == GDN_OK) st = launch_heads<T>(p, reinterpret_cast<const float*>(ws + L.dk), pc.nc, dk, s);
    if (st != GDN_OK) return st;
  }
  return p.g_per_head ? launch_head_decays(p, part, pc.nc, dg, s) : GDN_OK;
}

}  // namespace

gdn_status launch_head_decays(const gdn_linear_problem& p, const float* part, const int32_t* nc, float* dg,
                              cudaStream_t s) {
  head_decays_kernel<<<p.Hv, 256, 0, s>>>(part, p.Hv, pieces_max(p, kC), nc, dg);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

size_t simt_bwd_bytes(const gdn_linear_problem& p) { return layout_of(p).end; }

gdn_status simt_bwd(const gdn_linear_problem& p, const void* q, const void* k, const void* v, const float* g,
                    float scale, const float* h0, const int32_t* cu, const void* dout, const float* dht, void* dq,
                    void* dk, void* dv, float* dg, float* dh0, void* ws, cudaStream_t s) {
  uint8_t* at = static_cast<uint8_t*>(ws);
  int32_t* status = reinterpret_cast<int32_t*>(at);
  if (cudaMemsetAsync(status, 0, sizeof(int32_t), s) != cudaSuccess) return GDN_ERR_CUDA;
  const Layout L = layout_of(p);
  if (launch_pieces(p, kC, cu, at + L.tables, status, s) != cudaSuccess) return GDN_ERR_CUDA;
  const Pieces pc = pieces_at(p, kC, at + L.tables);
  if (p.dt == GDN_F32)
    return bwd_t<float>(p, (const float*)q, (const float*)k, (const float*)v, g, scale, h0, (const float*)dout, dht,
                        (float*)dq, (float*)dk, (float*)dv, dg, dh0, pc, L, at, s);
  using T = __nv_bfloat16;
  return bwd_t<T>(p, (const T*)q, (const T*)k, (const T*)v, g, scale, h0, (const T*)dout, dht, (T*)dq, (T*)dk, (T*)dv,
                  dg, dh0, pc, L, at, s);
}

}  // namespace lin

size_t linear_bwd_workspace_bytes(const gdn_linear_problem& p) {
  return lin::tc_bwd_supported(p) ? lin::tc_bwd_bytes(p) : lin::simt_bwd_bytes(p);
}

gdn_status run_linear_bwd(const gdn_linear_problem& p, const void* q, const void* k, const void* v, const float* g,
                          float scale, const float* h0, const int32_t* cu, const void* dout, const float* dht,
                          void* dq, void* dk, void* dv, float* dg, float* dh0, void* ws, cudaStream_t s) {
  return (lin::tc_bwd_supported(p) ? lin::tc_bwd : lin::simt_bwd)(p, q, k, v, g, scale, h0, cu, dout, dht, dq, dk, dv, dg, dh0, ws, s);
}

}  // namespace gdn
