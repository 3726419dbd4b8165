// gdn_scan_bwd.cu -- gradients of the selective state space scan (gdn_scan.cu;
// layout and scalar functions in gdn_scan.cuh).
//
// With a_t = e^{dt_t A}, dy_t = dout_t silu(z_t) and the adjoint of the state
//     q_t = C_t dy_t + a_{t+1} q_{t+1}      (a q past the last token: dht)
// the gradients are, for channel d and summed over what is not an index,
//     dC_t  = dy_t h_t                 dB_t     = dt_t x_t q_t
//     dx_t  = dt_t q_t.B_t + D dy_t    ddt_t    = x_t q_t.B_t + sum_n A a_t q_t h_{t-1}
//     dA    = dt_t a_t q_t h_{t-1}     ddelta_t = ddt_t sigmoid(delta_t + dt_bias)
//     dz_t  = dout_t (C_t.h_t + D x_t) silu'(z_t),   dD = dy_t x_t,   ddt_bias = ddelta_t
//     dh0   = a_1 q_1.
//
// A warp owns channels as in the forward.  It runs its segment of a sequence
// forward once, keeping the state before every tile, then walks back: a tile's
// states are recomputed four tokens at a time into registers (with the states
// before each four in shared memory), and the adjoint passes over them.  Sums
// over the state lanes (q.B, the A term, y) and over the channel lanes (dB, dC)
// are reduce-scattered four tokens at a time; the warps of a CTA add their dB and
// dC through shared memory and write one partial a CTA, which a second launch
// adds up in order, as it does the per-CTA partials of dA, dD and ddt_bias: no
// atomics, so results do not depend on the run.
//
// Few chains are cut into segments as in the forward; the adjoints at the
// segments' ends come from the same chaining backwards in time.
//
// What bounds it (one GB300): as the forward, issue and latency at 8 warps an SM.
// 230 instructions a token and warp of 256 updates, IPC 2.0 of 4, LSU wavefronts
// 38 %, DRAM 8 % (by ncu, 237 registers).  4 x 4096 tokens, 4096 channels, 16
// states, bf16, gated: 1.82 ms, one hundredth of it for the compensated sums of dD
// and ddt_bias and for infinite ones.
#include "gdn_scan.cuh"

namespace gdn {
namespace scan {
namespace {

struct BwdArgs {
  Args a;
  const void* dout;
  const float* dht;
  bool vg, vo;           // dout, and the outputs like x, in pairs
  float* qseg;           // [segments][D][S]: local adjoints, then the adjoints at the segments' ends
  float* qdt;            // [segments][D]
  float4* ck;            // [CTAs][tiles of a segment][warps][2][32]: states before the tiles
  int64_t units;         // bound on the segments
  int slots, tiles;      // CTAs that share the segments of a channel block, tiles of a segment
  float* pbc;            // [channel blocks of a group][tokens][G][2][S]
  float *pA, *pD, *pbias;   // [slots][D][S], [slots][D], [slots][D]
  void *dx, *ddelta, *dz, *dB, *dC;
  float *dA, *dD, *dbias, *dh0;
  int cgrp;              // CTA channel blocks a group
  int64_t Ttot;
};

// dout silu(z)
template <typename T>
__device__ __forceinline__ float2 gated(float2 g, float2 z, bool has) {
  return has ? make_float2(g.x * z.x * sigmoid(z.x), g.y * z.y * sigmoid(z.y)) : g;
}

// ---------------------------------------------- adjoints across segments
// Each segment but a sequence's first, run backwards from a zero adjoint:
// a q at its start, and the sum of its steps.
template <typename T, int RL>
__global__ void __launch_bounds__(128) scan_rev_kernel(const BwdArgs b) {
  using L = Lanes<RL>;
  const Args& a = b.a;
  __shared__ __align__(16) float sC[4][L::TT][L::SP];
  __shared__ __align__(16) float4 sdt[4][L::TT][L::CL];   // dt, dy of a channel pair
  const L ln;
  const int w = threadIdx.x >> 5;
  const int cb = blockIdx.y * 4 + w, g = cb / a.cbg;
  if (g >= a.G) return;
  Unit u;
  if (!unit_of(a, blockIdx.x, u) || u.first) return;
  const int d = g * a.Dg + (cb - g * a.cbg) * L::CPW + 2 * ln.chl, dend = (g + 1) * a.Dg;
  const bool ok0 = d < dend, ok1 = d + 1 < dend;
  const int n0 = 4 * ln.sl, nn = a.S - n0;
  const bool v4 = a.S % 4 == 0;
  float2 A2[2][2], q[2][2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    float r[4] = {0.f, 0.f, 0.f, 0.f};
    if (c ? ok1 : ok0) load4(a.A + (int64_t)(d + c) * a.S + n0, nn, v4, r);
    A2[c][0] = make_float2(rate2(r[0]), rate2(r[1]));
    A2[c][1] = make_float2(rate2(r[2]), rate2(r[3]));
    q[c][0] = q[c][1] = make_float2(0.f, 0.f);
  }
  const float2 bias = make_float2(a.bias && ok0 ? a.bias[d] : 0.f, a.bias && ok1 ? a.bias[d + 1] : 0.f);
  const T* pd = reinterpret_cast<const T*>(static_cast<const char*>(a.dl) + u.tok0 * a.bd) + d;
  const T* pz = a.z ? reinterpret_cast<const T*>(static_cast<const char*>(a.z) + u.tok0 * a.bz) + d : nullptr;
  const T* pg = static_cast<const T*>(b.dout) + u.tok0 * a.D + d;
  const T* pC = reinterpret_cast<const T*>(static_cast<const char*>(a.C) + u.tok0 * a.bc) + g * a.S;
  constexpr int VE = RowVec<T, RL>::VE, NV = RowVec<T, RL>::NV, NPV = (NV + 31) / 32;
  Raw2<T> rd[4], rz[4], rg[4];
  uint4 rC[NPV];
  auto load_tile = [&](int t0) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int t = t0 + ln.token(k);
      rd[k].zero(), rz[k].zero(), rg[k].zero();
      if (t < u.len && ok0) {
        rd[k].load(row(pd, t, a.bd), a.vin, ok0, ok1);
        rg[k].load(pg + (int64_t)t * a.D, b.vg, ok0, ok1);
        if (pz) rz[k].load(row(pz, t, a.bz), a.vin, ok0, ok1);
      }
    }
#pragma unroll
    for (int i = 0; i < NPV; ++i) {
      const int p = (ln.lane + 32 * i) * VE, t = t0 + p / L::SP, n = p % L::SP;
      rC[i] = make_uint4(0u, 0u, 0u, 0u);
      if ((NV % 32 == 0 || ln.lane + 32 * i < NV) && t < u.len) rC[i] = load_row16<T, VE>(row(pC, t, a.bc), n, a.S, a.vbc);
    }
  };
  float2 dts = make_float2(0.f, 0.f);
  int t0 = (u.len - 1) / L::TT * L::TT;
  load_tile(t0);
  for (; t0 >= 0; t0 -= L::TT) {
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float2 dt = rd[k].f();
      dt.x += bias.x, dt.y += bias.y;
      if (a.softplus) {
        float2 e;
        dt = softplus2(dt, e);
      }
      if (t0 + ln.token(k) >= u.len) dt = make_float2(0.f, 0.f);
      dts.x += dt.x, dts.y += dt.y;
      const float2 dy = gated<T>(rg[k].f(), rz[k].f(), pz != nullptr);
      if (!ln.dup) sdt[w][ln.token(k)][ln.chl] = make_float4(dt.x, dy.x, dt.y, dy.y);
    }
#pragma unroll
    for (int i = 0; i < NPV; ++i)
      if (NV % 32 == 0 || ln.lane + 32 * i < NV) put_row16<T, VE>(&sC[w][0][0] + (ln.lane + 32 * i) * VE, rC[i]);
    __syncwarp();
    if (t0 > 0) load_tile(t0 - L::TT);
#pragma unroll 4
    for (int t = L::TT - 1; t >= 0; --t) {
      const float4 s = sdt[w][t][ln.chl];
      const float4 cc = *reinterpret_cast<const float4*>(&sC[w][t][n0]);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float dt = c ? s.z : s.x, dy = c ? s.w : s.y;
        const float2 dt2 = make_float2(dt, dt), dy2 = make_float2(dy, dy);
        q[c][0] = __fmul2_rn(decay2(dt2, A2[c][0]), __ffma2_rn(dy2, make_float2(cc.x, cc.y), q[c][0]));
        q[c][1] = __fmul2_rn(decay2(dt2, A2[c][1]), __ffma2_rn(dy2, make_float2(cc.z, cc.w), q[c][1]));
      }
    }
  }
  if (ln.dup) dts = make_float2(0.f, 0.f);
#pragma unroll
  for (int m = 16; m >= L::CL && RL > 1; m >>= 1) {
    dts.x += __shfl_xor_sync(~0u, dts.x, m);
    dts.y += __shfl_xor_sync(~0u, dts.y, m);
  }
  if (ln.sl == 0) {
    if (ok0) b.qdt[(int64_t)blockIdx.x * a.D + d] = dts.x;
    if (ok1) b.qdt[(int64_t)blockIdx.x * a.D + d + 1] = dts.y;
  }
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const float s[4] = {q[c][0].x, q[c][0].y, q[c][1].x, q[c][1].y};
    if (c ? ok1 : ok0) store4(b.qseg + ((int64_t)blockIdx.x * a.D + d + c) * a.S + n0, nn, v4, s);
  }
}

// qseg: local adjoints -> the a q that enters each segment at its end.
__global__ void __launch_bounds__(256) rev_chain_kernel(const BwdArgs b) {
  const Args& a = b.a;
  const int64_t DS = (int64_t)a.D * a.S;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int k = blockIdx.y + gridDim.y * blockIdx.z;
  if (i >= DS || k >= (a.cu ? a.seg0[a.N + 1] : a.N)) return;
  const int n = a.cu ? a.seg0[a.N + 2 + k] : k;
  const int d = (int)(i / a.S);
  const int64_t u0 = a.cu ? a.seg0[n] : (int64_t)n * a.nseg;
  const int64_t u1 = a.cu ? a.seg0[n + 1] : u0 + a.nseg;
  const float r = rate2(a.A[i]);
  float q = b.dht ? b.dht[n * DS + i] : 0.f;
  for (int64_t u = u1 - 1; u > u0; u -= 8) {   // eight segments' loads at a time
    float loc[8], dt[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const bool in = u - k > u0;
      loc[k] = in ? b.qseg[(u - k) * DS + i] : 0.f;
      dt[k] = in ? b.qdt[(u - k) * a.D + d] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (u - k <= u0) break;
      b.qseg[(u - k) * DS + i] = q;
      q = fmaf(sm100::ex2_fast(r * dt[k]), q, loc[k]);
    }
  }
  b.qseg[u0 * DS + i] = q;
}

// ------------------------------------------------------------ the gradients

__device__ __forceinline__ float2 sub2(float2 a, float2 b) { return __fadd2_rn(a, make_float2(-b.x, -b.y)); }

// sum += v; what the addition drops is kept in `lost` and put back into the next one.
// (Nothing is kept of a sum that is not finite: its difference to itself would make an
// infinity a NaN.)
__device__ __forceinline__ void add_kept(float2& sum, float2& lost, float2 v) {
  const float2 y = sub2(v, lost), s = __fadd2_rn(sum, y), l = sub2(sub2(s, sum), y);
  lost.x = fabsf(l.x) <= FLT_MAX ? l.x : 0.f;
  lost.y = fabsf(l.y) <= FLT_MAX ? l.y : 0.f;
  sum = s;
}

// Warps of a CTA (one group's channels), and its shared memory.
constexpr int kBwdRing = 3;   // tiles as loaded: one in use, two on their way
constexpr int bwd_warps(int RL) { return RL >= 8 ? 4 : 8; }

template <typename T, int RL>
struct Smem {
  using L = Lanes<RL>;
  static constexpr int W = bwd_warps(RL);
  static constexpr int NS = L::NG > 1 ? L::NG - 1 : 1;
  // rows as loaded: x, delta, dout and z of the warps' channels, B and C
  alignas(16) T rx[kBwdRing][4][W][L::TT][L::CPW];
  alignas(16) T rbc[kBwdRing][2][L::TT][L::SP];
  float B[L::TT][L::SP], C[L::TT][L::SP];
  float4 dt[W][L::TT][L::CL];     // dt of a channel pair, dt x
  float2 dy[W][L::TT][L::CL];
  float4 sub[W][NS][2][32];       // states before the tile's second, third, .. four tokens
  float red[W][L::TT][2][L::SP];  // dB and dC of a warp's channels
};

// Sums over the channel lanes of v[tok][2][4] (four tokens' dB and dC): lane chl
// ends with the 32 / CL sums from index chl * (32 / CL) on, in v[0 ..].
template <int CL>
__device__ __forceinline__ void reduce_channels(float (&v)[32], int lane) {
  int n = 16;
#pragma unroll
  for (int m = CL / 2; m >= 1; m >>= 1) {
    const bool up = lane & m;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (i < n) {
        const float send = up ? v[i] : v[i + n];
        const float keep = up ? v[i + n] : v[i];
        v[i] = keep + __shfl_xor_sync(~0u, send, m);
      }
    n >>= 1;
  }
}

template <typename T, int RL, int ROWS>
__global__ void __launch_bounds__(32 * bwd_warps(RL)) scan_bwd_kernel(const BwdArgs b) {
  using L = Lanes<RL>;
  using SM = Smem<T, RL>;
  constexpr bool ASYNC = ROWS != kRegs;
  constexpr int W = SM::W, NT = 32 * W;
  extern __shared__ __align__(16) char raw_smem[];
  SM& sm = *reinterpret_cast<SM*>(raw_smem);
  const Args& a = b.a;
  const L ln;
  const int w = threadIdx.x >> 5;
  const int g = blockIdx.y / b.cgrp, jb = blockIdx.y - g * b.cgrp;
  const int wb = jb * W + w;   // warp block of the group; past the group's end: nothing to do but the barriers
  const int dw = g * a.Dg + wb * L::CPW, d = dw + 2 * ln.chl, dend = (g + 1) * a.Dg;
  const bool ok0 = d < dend, ok1 = d + 1 < dend;
  const int n0 = 4 * ln.sl, nn = a.S - n0;
  const bool v4 = a.S % 4 == 0;
  const bool gate = a.z != nullptr;
  constexpr float kLn2 = 0.6931471805599453f;

  float2 A2[2][2], dA[2][2], lost[2][2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    lost[c][0] = lost[c][1] = make_float2(0.f, 0.f);
    float r[4] = {0.f, 0.f, 0.f, 0.f};
    if (c ? ok1 : ok0) load4(a.A + (int64_t)(d + c) * a.S + n0, nn, v4, r);
    A2[c][0] = make_float2(rate2(r[0]), rate2(r[1]));
    A2[c][1] = make_float2(rate2(r[2]), rate2(r[3]));
    dA[c][0] = dA[c][1] = make_float2(0.f, 0.f);
  }
  const float2 bias = make_float2(a.bias && ok0 ? a.bias[d] : 0.f, a.bias && ok1 ? a.bias[d + 1] : 0.f);
  const float2 skip = make_float2(a.Dp && ok0 ? a.Dp[d] : 0.f, a.Dp && ok1 ? a.Dp[d + 1] : 0.f);
  float2 dD = make_float2(0.f, 0.f), dbias = dD, lostD = dD, lostb = dD;
  float4* ck = b.ck + ((int64_t)(blockIdx.y * b.slots + blockIdx.x) * b.tiles) * (W * 64) + w * 64 + ln.lane;

  Unit u;
  for (int64_t un = blockIdx.x; un < b.units && unit_of(a, un, u); un += b.slots) {
    const T* px = reinterpret_cast<const T*>(static_cast<const char*>(a.x) + u.tok0 * a.bx) + d;
    const T* pd = reinterpret_cast<const T*>(static_cast<const char*>(a.dl) + u.tok0 * a.bd) + d;
    const T* pz = gate ? reinterpret_cast<const T*>(static_cast<const char*>(a.z) + u.tok0 * a.bz) + d : nullptr;
    const T* pg = static_cast<const T*>(b.dout) + u.tok0 * a.D + d;
    const T* pB = reinterpret_cast<const T*>(static_cast<const char*>(a.B) + u.tok0 * a.bb) + g * a.S;
    const T* pC = reinterpret_cast<const T*>(static_cast<const char*>(a.C) + u.tok0 * a.bc) + g * a.S;

    float2 h[2][2], q[2][2];   // state; a q from the right
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float s[4] = {0.f, 0.f, 0.f, 0.f}, r[4] = {0.f, 0.f, 0.f, 0.f};
      if (c ? ok1 : ok0) {
        // (a cut sequence's first and last too: dh0, which its first one writes, may be h0 or dht)
        const bool cut = !u.first || !u.last;
        const float* from = cut    ? a.hseg + (un * a.D + d + c) * a.S
                            : a.h0 ? a.h0 + ((int64_t)u.n * a.D + d + c) * a.S : nullptr;
        if (from) load4(from + n0, nn, v4, s);
        const float* end = cut     ? b.qseg + (un * a.D + d + c) * a.S
                           : b.dht ? b.dht + ((int64_t)u.n * a.D + d + c) * a.S : nullptr;
        if (end) load4(end + n0, nn, v4, r);
      }
      h[c][0] = make_float2(s[0], s[1]), h[c][1] = make_float2(s[2], s[3]);
      q[c][0] = make_float2(r[0], r[1]), q[c][1] = make_float2(r[2], r[3]);
    }

    // tile i's rows into ring slot r (those that the walk back needs too)
    auto fetch = [&](int i, int r, bool back) {
      if constexpr (ASYNC) {
        constexpr int XROW = L::CPW * sizeof(T), SROW = L::SP * sizeof(T);
        constexpr int CX = chunk<ROWS, XROW>(), CB = chunk<ROWS, SROW>();
        if (i >= 0) {
          const int t0 = i * L::TT, vx = (dend - dw) * (int)sizeof(T), vs = a.S * (int)sizeof(T);
          auto rows = [&](int k, const T* p, int stride) {
            copy_rows<L::TT, XROW, CX>((char*)&sm.rx[r][k][w][0][0], (const char*)(p - 2 * ln.chl), stride, t0, u.len, vx,
                                       ln.lane);
          };
          rows(0, px, a.bx);
          rows(1, pd, a.bd);
          if (back) {
            rows(2, pg, a.D * (int)sizeof(T));
            if (gate) rows(3, pz, a.bz);
          }
          if (w == 0)
            copy_rows<L::TT, SROW, CB>((char*)&sm.rbc[r][0][0][0], (const char*)pB, a.bb, t0, u.len, vs, ln.lane);
          if (w == 1 && back)
            copy_rows<L::TT, SROW, CB>((char*)&sm.rbc[r][1][0][0], (const char*)pC, a.bc, t0, u.len, vs, ln.lane);
        }
        copies_commit();
      }
    };
    // a pair of this lane's channels of row kind k (x, delta, dout, z) at token tk of slot r's tile
    auto pair = [&](int k, int r, int tk, int t, const T* p, int stride, bool vec) {
      Raw2<T> v;
      v.zero();
      if constexpr (ASYNC) v.load_shared(&sm.rx[r][k][w][tk][2 * ln.chl]);
      else if (t < u.len && ok0) v.load(row(p, t, stride), vec, ok0, ok1);
      return v.f();
    };
    // a tile's steps and inputs into shared memory; x and softplus' stay
    float2 xs[4], sp[4];
    auto stage = [&](int t0, int r, bool back) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int tk = ln.token(k), t = t0 + tk;
        const float2 x = pair(0, r, tk, t, px, a.bx, a.vin);
        float2 dt = __fadd2_rn(pair(1, r, tk, t, pd, a.bd, a.vin), bias);
        if (a.softplus) {
          float2 e;
          const float2 v = dt;
          dt = softplus2(dt, e);
          // sigmoid(v), from e^{-|v|}
          if (back) sp[k] = make_float2((v.x >= 0.f ? 1.f : e.x) * rcp_approx(1.f + e.x),
                                        (v.y >= 0.f ? 1.f : e.y) * rcp_approx(1.f + e.y));
        } else if (back) {
          sp[k] = make_float2(1.f, 1.f);
        }
        if (t >= u.len) dt = make_float2(0.f, 0.f);
        xs[k] = x;
        const float2 dx = __fmul2_rn(dt, x);   // x is zero past the end
        float2 dy;
        if (back) {
          dy = pair(2, r, tk, t, pg, a.D * (int)sizeof(T), b.vg);
          if (gate) dy = gated<T>(dy, pair(3, r, tk, t, pz, a.bz, a.vin), true);
        }
        if (!ln.dup) {
          sm.dt[w][tk][ln.chl] = make_float4(dt.x, dt.y, dx.x, dx.y);
          if (back) sm.dy[w][tk][ln.chl] = dy;
        }
      }
      // B (and C) of the CTA's group
      constexpr int VE = RowVec<T, RL>::VE, NV = RowVec<T, RL>::NV;
      for (int i = threadIdx.x; i < NV; i += NT) {
        const int p = i * VE, t = t0 + p / L::SP, n = p % L::SP;
        uint4 rb = make_uint4(0u, 0u, 0u, 0u), rc = rb;
        if constexpr (ASYNC) {
          rb = get_vec<VE * sizeof(T)>(&sm.rbc[r][0][0][0] + p);
          if (back) rc = get_vec<VE * sizeof(T)>(&sm.rbc[r][1][0][0] + p);
        } else if (t < u.len) {
          rb = load_row16<T, VE>(row(pB, t, a.bb), n, a.S, a.vbc);
          if (back) rc = load_row16<T, VE>(row(pC, t, a.bc), n, a.S, a.vbc);
        }
        put_row16<T, VE>(&sm.B[0][0] + p, rb);
        if (back) put_row16<T, VE>(&sm.C[0][0] + p, rc);
      }
    };
    // one token of the recurrence
    auto advance = [&](int t, float2 (&hh)[2][2], float2 (&aa)[2][2]) {
      const float4 s = sm.dt[w][t][ln.chl];
      const float4 bb = *reinterpret_cast<const float4*>(&sm.B[t][n0]);
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float dt = c ? s.y : s.x, ux = c ? s.w : s.z;
        const float2 dt2 = make_float2(dt, dt), ux2 = make_float2(ux, ux);
        aa[c][0] = decay2(dt2, A2[c][0]);
        aa[c][1] = decay2(dt2, A2[c][1]);
        hh[c][0] = __ffma2_rn(aa[c][0], hh[c][0], __fmul2_rn(ux2, make_float2(bb.x, bb.y)));
        hh[c][1] = __ffma2_rn(aa[c][1], hh[c][1], __fmul2_rn(ux2, make_float2(bb.z, bb.w)));
      }
    };

    // forward: the state before every tile
    const int ntile = (u.len + L::TT - 1) / L::TT;
#pragma unroll
    for (int k = 0; k < kBwdRing - 1; ++k) fetch(k < ntile - 1 ? k : -1, k, false);
    for (int i = 0, r = 0; i < ntile; ++i) {
      if (i + 1 == ntile) break;   // the last tile's is in h
      float4* o = ck + (int64_t)i * (W * 64);
      o[0] = make_float4(h[0][0].x, h[0][0].y, h[0][1].x, h[0][1].y);
      o[32] = make_float4(h[1][0].x, h[1][0].y, h[1][1].x, h[1][1].y);
      if (ASYNC) copies_wait<kBwdRing - 2>();
      __syncthreads();   // copies are here; the tile before has been used
      fetch(i + kBwdRing - 1 < ntile - 1 ? i + kBwdRing - 1 : -1, r == 0 ? kBwdRing - 1 : r - 1, false);
      stage(i * L::TT, r, false);
      __syncthreads();
      float2 aa[2][2];
#pragma unroll 4
      for (int t = 0; t < L::TT; ++t) advance(t, h, aa);
      r = r + 1 == kBwdRing ? 0 : r + 1;
    }

    // backward, the state before the next tile loaded ahead
    float4 c0, c1;
    if (ASYNC) copies_wait<0>();
#pragma unroll
    for (int k = 0; k < kBwdRing - 1; ++k) fetch(ntile - 1 - k, k, true);
    for (int i = ntile - 1, r = 0; i >= 0; --i) {
      const int t0 = i * L::TT;
      if (i + 1 < ntile) {
        h[0][0] = make_float2(c0.x, c0.y), h[0][1] = make_float2(c0.z, c0.w);
        h[1][0] = make_float2(c1.x, c1.y), h[1][1] = make_float2(c1.z, c1.w);
      }
      if (ASYNC) copies_wait<kBwdRing - 2>();
      __syncthreads();
      if (i > 0) c0 = ck[(int64_t)(i - 1) * (W * 64)], c1 = ck[(int64_t)(i - 1) * (W * 64) + 32];
      fetch(i - (kBwdRing - 1), r == 0 ? kBwdRing - 1 : r - 1, true);
      stage(t0, r, true);
      __syncthreads();
      // states before each four tokens
      if (L::NG > 1) {
        const float2 k00 = h[0][0], k01 = h[0][1], k10 = h[1][0], k11 = h[1][1];
#pragma unroll 1
        for (int gr = 0; gr < L::NG - 1; ++gr) {
          float2 aa[2][2];
#pragma unroll
          for (int j = 0; j < 4; ++j) advance(4 * gr + j, h, aa);
#pragma unroll
          for (int c = 0; c < 2; ++c)
            sm.sub[w][gr][c][ln.lane] = make_float4(h[c][0].x, h[c][0].y, h[c][1].x, h[c][1].y);
        }
        h[0][0] = k00, h[0][1] = k01, h[1][0] = k10, h[1][1] = k11;
      }
      const float2 first00 = h[0][0], first01 = h[0][1], first10 = h[1][0], first11 = h[1][1];
      // dA, dD and ddt_bias of the tile first: a sum over all tokens in one place would lose small terms
      float2 tA[2][2], tD = make_float2(0.f, 0.f), tb = tD;
#pragma unroll
      for (int c = 0; c < 2; ++c) tA[c][0] = tA[c][1] = make_float2(0.f, 0.f);
#pragma unroll
      for (int gr = L::NG - 1; gr >= 0; --gr) {
        float2 hs[2][2];   // state before the four tokens
        if (gr > 0) {
          const float4 s0 = sm.sub[w][gr - 1][0][ln.lane], s1 = sm.sub[w][gr - 1][1][ln.lane];
          hs[0][0] = make_float2(s0.x, s0.y), hs[0][1] = make_float2(s0.z, s0.w);
          hs[1][0] = make_float2(s1.x, s1.y), hs[1][1] = make_float2(s1.z, s1.w);
        } else {
          hs[0][0] = first00, hs[0][1] = first01, hs[1][0] = first10, hs[1][1] = first11;
        }
        float2 hh[4][2][2], aa[4][2][2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int e = 0; e < 2; ++e) hh[j][c][e] = j ? hh[j - 1][c][e] : hs[c][e];
          advance(4 * gr + j, hh[j], aa[j]);
        }
        float v[24], cs[32];
#pragma unroll
        for (int j = 3; j >= 0; --j) {
          const int t = 4 * gr + j;
          const float4 s = sm.dt[w][t][ln.chl];
          const float2 dy = sm.dy[w][t][ln.chl];
          const float4 bb = *reinterpret_cast<const float4*>(&sm.B[t][n0]);
          const float4 cc = *reinterpret_cast<const float4*>(&sm.C[t][n0]);
          const float2 B2[2] = {make_float2(bb.x, bb.y), make_float2(bb.z, bb.w)};
          const float2 C2[2] = {make_float2(cc.x, cc.y), make_float2(cc.z, cc.w)};
          float2 dB2[2], dC2[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float dt = c ? s.y : s.x, ux = c ? s.w : s.z, gy = c ? dy.y : dy.x;
            const float2 dt2 = make_float2(dt, dt), ux2 = make_float2(ux, ux), gy2 = make_float2(gy, gy);
            float2 gB = make_float2(0.f, 0.f), wA = gB, y2 = gB;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float2 qq = __ffma2_rn(gy2, C2[e], q[c][e]);
              dC2[e] = c ? __ffma2_rn(gy2, hh[j][c][e], dC2[e]) : __fmul2_rn(gy2, hh[j][c][e]);
              dB2[e] = c ? __ffma2_rn(ux2, qq, dB2[e]) : __fmul2_rn(ux2, qq);
              gB = __ffma2_rn(qq, B2[e], gB);
              y2 = __ffma2_rn(hh[j][c][e], C2[e], y2);
              const float2 aq = __fmul2_rn(aa[j][c][e], qq);
              const float2 wq = __fmul2_rn(aq, j ? hh[j - 1][c][e] : hs[c][e]);
              tA[c][e] = __ffma2_rn(wq, dt2, tA[c][e]);
              wA = __ffma2_rn(wq, A2[c][e], wA);
              q[c][e] = aq;
            }
            v[6 * j + c] = gB.x + gB.y;
            v[6 * j + 2 + c] = wA.x + wA.y;
            v[6 * j + 4 + c] = y2.x + y2.y;
          }
          cs[8 * j + 0] = dB2[0].x, cs[8 * j + 1] = dB2[0].y, cs[8 * j + 2] = dB2[1].x, cs[8 * j + 3] = dB2[1].y;
          cs[8 * j + 4] = dC2[0].x, cs[8 * j + 5] = dC2[0].y, cs[8 * j + 6] = dC2[1].x, cs[8 * j + 7] = dC2[1].y;
        }
        reduce_states<RL, 6>(v, ln.lane);
        reduce_channels<L::CL>(cs, ln.lane);
        constexpr int NV = 32 / L::CL;
#pragma unroll
        for (int i2 = 0; i2 < NV; ++i2) {
          const int idx = ln.chl * NV + i2;
          sm.red[w][4 * gr + idx / 8][(idx / 4) % 2][n0 + idx % 4] = cs[i2];
        }
        // this lane's tokens
#pragma unroll
        for (int j = 0; j < L::TPL; ++j) {
          const int k = gr * L::TPL + j, tk = ln.token(k), t = t0 + tk;
          const float4 s = sm.dt[w][tk][ln.chl];
          const float2 dy = sm.dy[w][tk][ln.chl], x = xs[k];
          const float2 gB = make_float2(v[6 * j], v[6 * j + 1]);
          const float2 wA = make_float2(v[6 * j + 2], v[6 * j + 3]);
          const float2 dx = make_float2(fmaf(gB.x, s.x, skip.x * dy.x), fmaf(gB.y, s.y, skip.y * dy.y));
          const float2 dd = make_float2(fmaf(gB.x, x.x, wA.x * kLn2) * sp[k].x, fmaf(gB.y, x.y, wA.y * kLn2) * sp[k].y);
          if (t < u.len && ok0 && !ln.dup) {
            const int64_t o = (u.tok0 + t) * a.D + d;
            store2(static_cast<T*>(b.dx) + o, dx, b.vo, ok0, ok1);
            store2(static_cast<T*>(b.ddelta) + o, dd, b.vo, ok0, ok1);
            tD = __ffma2_rn(dy, x, tD);
            tb = __fadd2_rn(tb, dd);
            if (gate) {
              const float2 z = pair(3, r, tk, t, pz, a.bz, a.vin);
              const float2 gr2 = pair(2, r, tk, t, pg, a.D * (int)sizeof(T), b.vg);
              const float s0 = sigmoid(z.x), s1 = sigmoid(z.y);
              const float2 dz = make_float2(
                  gr2.x * fmaf(skip.x, x.x, v[6 * j + 4]) * (s0 * fmaf(z.x, 1.f - s0, 1.f)),
                  gr2.y * fmaf(skip.y, x.y, v[6 * j + 5]) * (s1 * fmaf(z.y, 1.f - s1, 1.f)));
              store2(static_cast<T*>(b.dz) + o, dz, b.vo, ok0, ok1);
            }
          }
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) add_kept(dA[c][e], lost[c][e], tA[c][e]);
      add_kept(dD, lostD, tD);
      add_kept(dbias, lostb, tb);
      // dB and dC of the CTA's channels
      __syncthreads();
      for (int p = threadIdx.x; p < L::TT * 2 * L::SP; p += NT) {
        const int tk = p / (2 * L::SP), m = p % (2 * L::SP), n = m % L::SP, t = t0 + tk;
        if (n >= a.S || t >= u.len) continue;
        float sum = 0.f;
#pragma unroll
        for (int ww = 0; ww < W; ++ww) sum += sm.red[ww][tk][m / L::SP][n];
        b.pbc[((((int64_t)jb * b.Ttot + u.tok0 + t) * a.G + g) * 2 + m / L::SP) * a.S + n] = sum;
      }
      r = r + 1 == kBwdRing ? 0 : r + 1;
    }
    if (ASYNC) copies_wait<0>();
    if (b.dh0 && u.first) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const float s[4] = {q[c][0].x, q[c][0].y, q[c][1].x, q[c][1].y};
        if (c ? ok1 : ok0) store4(b.dh0 + ((int64_t)u.n * a.D + d + c) * a.S + n0, nn, v4, s);
      }
    }
  }

  // this CTA's parameter gradients
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    const float s[4] = {dA[c][0].x, dA[c][0].y, dA[c][1].x, dA[c][1].y};
    if (c ? ok1 : ok0) store4(b.pA + ((int64_t)blockIdx.x * a.D + d + c) * a.S + n0, nn, v4, s);
  }
#pragma unroll
  for (int m = 16; m >= L::CL && RL > 1; m >>= 1) {
    dD.x += __shfl_xor_sync(~0u, dD.x, m), dD.y += __shfl_xor_sync(~0u, dD.y, m);
    dbias.x += __shfl_xor_sync(~0u, dbias.x, m), dbias.y += __shfl_xor_sync(~0u, dbias.y, m);
  }
  if (ln.sl == 0) {
    const int64_t o = (int64_t)blockIdx.x * a.D + d;
    if (ok0) b.pD[o] = dD.x, b.pbias[o] = dbias.x;
    if (ok1) b.pD[o + 1] = dD.y, b.pbias[o + 1] = dbias.y;
  }
}

// dB and dC: the channel blocks' partials in order, a thread per (token, group, state).
template <typename T>
__global__ void __launch_bounds__(256) scan_bwd_bc_kernel(const BwdArgs b) {
  const Args& a = b.a;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int64_t row = (int64_t)a.G * 2 * a.S, all = b.Ttot * row;
  if (i >= all || (a.cu && a.seg0[a.N] < 0)) return;
  float s = 0.f;
  for (int j = 0; j < b.cgrp; ++j) s += b.pbc[j * all + i];
  const int n = (int)(i % a.S), which = (int)(i / a.S % 2);
  const int64_t tg = i / (2 * a.S);
  static_cast<T*>(which ? b.dC : b.dB)[tg * a.S + n] = from_f<T>(s);
}

// dA, dD and ddt_bias: the slots' partials in order.
__global__ void __launch_bounds__(256) scan_bwd_params_kernel(const BwdArgs b) {
  const Args& a = b.a;
  const int64_t DS = (int64_t)a.D * a.S;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= DS + 2 * a.D || (a.cu && a.seg0[a.N] < 0)) return;
  const float* p;
  float* o;
  int64_t n;
  if (i < DS) p = b.pA + i, o = b.dA + i, n = DS;
  else if (i < DS + a.D) p = b.pD + (i - DS), o = b.dD ? b.dD + (i - DS) : nullptr, n = a.D;
  else p = b.pbias + (i - DS - a.D), o = b.dbias ? b.dbias + (i - DS - a.D) : nullptr, n = a.D;
  if (!o) return;
  float s = 0.f;
  for (int k = 0; k < b.slots; ++k) s += p[k * n];
  *o = s;
}

struct BwdLayout {
  size_t status, seg0, hseg, dtsum, qseg, qdt, ck, pbc, pA, pD, pbias, total;
  int cgrp, slots, tiles, warps;
};

constexpr int kMaxSeg = 8192;   // tokens a segment: bounds the states kept before the tiles

// CTAs that the device holds at once (eight warps an SM, by their registers), and a
// problem's channel blocks.
int64_t bwd_capacity(const Plan& pl) { return (int64_t)sm_count() * (8 / bwd_warps(pl.RL)); }
int64_t bwd_blocks(const gdn_scan_problem& p, const Plan& pl) { return p.G * ceil_div(pl.cbg, bwd_warps(pl.RL)); }

// A CTA holds its place for a whole segment, so segments are made for one round of
// CTAs: equal lengths are cut when that lets twice as many run, packed sequences into
// halves of a CTA's share of the tokens (at least 64).
Plan bwd_plan(const gdn_scan_problem& p) {
  Plan pl = make_plan(p);
  const int64_t cap = bwd_capacity(pl), cbs = bwd_blocks(p, pl);
  int64_t len;
  if (p.varlen) {
    len = (int64_t)align_up((size_t)(p.T * cbs / (2 * cap)), kTileMax);
    if (len < 64) len = 64;
    if (len > kMaxSeg) len = kMaxSeg;
    pl.seglen = (int)len;
    pl.max_units = p.T / len + p.N;
    pl.cut = p.T > len;
  } else {
    int64_t n = 2 * p.B * cbs <= cap ? cap / (p.B * cbs) : 1;
    if (n > p.T / 64) n = p.T / 64 > 1 ? p.T / 64 : 1;
    len = (int64_t)align_up((size_t)ceil_div(p.T, n), kTileMax);
    if (len > kMaxSeg) len = kMaxSeg;
    pl.seglen = (int)len;
    pl.nseg = (int)ceil_div(p.T, len);
    pl.max_units = (int64_t)p.B * pl.nseg;
    pl.cut = pl.nseg > 1;
  }
  return pl;
}

BwdLayout bwd_layout(const gdn_scan_problem& p, const Plan& pl) {
  BwdLayout l;
  l.warps = bwd_warps(pl.RL);
  l.cgrp = (int)ceil_div(pl.cbg, l.warps);
  const int tt = pl.RL >= 4 ? 16 : 4 * pl.RL;
  const int64_t most = p.T < pl.seglen ? p.T : pl.seglen;
  l.tiles = (int)ceil_div(most > 0 ? most : 1, tt);
  const int64_t cbs = bwd_blocks(p, pl), cap = bwd_capacity(pl), want = cap / cbs > 1 ? cap / cbs : 1;
  l.slots = (int)(pl.max_units < want ? pl.max_units : want);
  const size_t DS = (size_t)p.D * p.S, f = sizeof(float);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align_up(bytes);
    return at;
  };
  l.status = take(kAlign);
  l.seg0 = take(p.varlen ? seg0_bytes(p.N, p.T, pl.seglen) : 0);
  l.hseg = take(pl.cut ? f * pl.max_units * DS : 0);
  l.dtsum = take(pl.cut ? f * pl.max_units * p.D : 0);
  l.qseg = take(pl.cut ? f * pl.max_units * DS : 0);
  l.qdt = take(pl.cut ? f * pl.max_units * p.D : 0);
  l.ck = take((size_t)cbs * l.slots * l.tiles * l.warps * 64 * sizeof(float4));
  l.pbc = take(f * l.cgrp * (size_t)p.B * p.T * p.G * 2 * p.S);
  l.pA = take(f * l.slots * DS);
  l.pD = take(f * l.slots * p.D);
  l.pbias = take(f * l.slots * p.D);
  l.total = o;
  return l;
}

template <typename T, int RL>
cudaError_t launch_bwd(const BwdArgs& b, const Plan& pl, cudaStream_t s) {
  const Args& a = b.a;
  if (pl.cut) {
    scan_rev_kernel<T, RL><<<dim3((unsigned)pl.max_units, (unsigned)ceil_div((int64_t)a.G * a.cbg, 4)), 128, 0, s>>>(b);
    const int64_t ncut = a.cu ? max_cut(a.N, a.T, a.seglen) : a.N, ny = ncut < 32768 ? ncut : 32768;
    rev_chain_kernel<<<dim3((unsigned)ceil_div((int64_t)a.D * a.S, 256), (unsigned)ny, (unsigned)ceil_div(ncut, ny)),
                       256, 0, s>>>(b);
  }
  constexpr size_t bytes = sizeof(Smem<T, RL>);
  const int64_t es = sizeof(T);
  RowsOf r = {Lanes<RL>::CPW * (int)es, 4 * RL * (int)es, a.G > 1, a.Dg * es, a.S * es};
  r.x(a.x, a.bx), r.x(a.dl, a.bd), r.x(a.z, a.bz), r.x(b.dout, a.D * es), r.s(a.B, a.bb), r.s(a.C, a.bc);
  auto* k = r.rows == kWide ? scan_bwd_kernel<T, RL, kWide> : r.rows == kNarrow ? scan_bwd_kernel<T, RL, kNarrow> : scan_bwd_kernel<T, RL, kRegs>;
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e != cudaSuccess) return e;
  k<<<dim3(b.slots, a.G * b.cgrp), 32 * bwd_warps(RL), bytes, s>>>(b);
  if (b.Ttot > 0)
    scan_bwd_bc_kernel<T><<<(unsigned)ceil_div(b.Ttot * a.G * 2 * a.S, 256), 256, 0, s>>>(b);
  scan_bwd_params_kernel<<<(unsigned)ceil_div((int64_t)a.D * a.S + 2 * a.D, 256), 256, 0, s>>>(b);
  return cudaGetLastError();
}

template <typename T>
cudaError_t dispatch_bwd(const BwdArgs& b, const Plan& pl, cudaStream_t s) {
  switch (pl.RL) {
    case 1: return launch_bwd<T, 1>(b, pl, s);
    case 2: return launch_bwd<T, 2>(b, pl, s);
    case 4: return launch_bwd<T, 4>(b, pl, s);
    case 8: return launch_bwd<T, 8>(b, pl, s);
    default: return launch_bwd<T, 16>(b, pl, s);
  }
}

bool even_pairs(const void* p, size_t es, int64_t ld, bool even) {
  return even && ld % 2 == 0 && reinterpret_cast<uintptr_t>(p) % (2 * es) == 0;
}

}  // namespace
}  // namespace scan

using namespace scan;

size_t scan_bwd_workspace_bytes(const gdn_scan_problem& p) { return bwd_layout(p, bwd_plan(p)).total; }

gdn_status run_scan_bwd(const gdn_scan_problem& p, const void* x, const void* delta, const float* A, const void* B,
                        const void* C, const float* Dp, const void* z, const float* dt_bias, const float* h0,
                        const int32_t* cu, const void* dout, const float* dht, void* dx, void* ddelta, float* dA,
                        void* dB, void* dC, float* dD, void* dz, float* ddt_bias, float* dh0, void* ws,
                        cudaStream_t s) {
  const Plan pl = bwd_plan(p);
  const BwdLayout l = bwd_layout(p, pl);
  BwdArgs b = {};
  b.a = base_args(p, pl, x, delta, A, B, C, Dp, z, dt_bias, h0, cu);
  Args& a = b.a;
  char* w = static_cast<char*>(ws);
  auto at = [&](size_t o) { return reinterpret_cast<float*>(w + o); };
  const size_t es = p.dt == GDN_F32 ? 4 : 2;
  const bool even = a.Dg % 2 == 0;
  b.dout = dout, b.dht = dht;
  b.vg = even_pairs(dout, es, p.D, even);
  b.vo = even_pairs(dx, es, p.D, even) && even_pairs(ddelta, es, p.D, even) && (!dz || even_pairs(dz, es, p.D, even));
  b.units = pl.max_units, b.slots = l.slots, b.tiles = l.tiles, b.cgrp = l.cgrp;
  b.ck = reinterpret_cast<float4*>(w + l.ck);
  b.pbc = at(l.pbc), b.pA = at(l.pA), b.pD = at(l.pD), b.pbias = at(l.pbias);
  b.dx = dx, b.ddelta = ddelta, b.dz = dz, b.dB = dB, b.dC = dC;
  b.dA = dA, b.dD = dD, b.dbias = ddt_bias, b.dh0 = dh0;
  b.Ttot = (int64_t)p.B * p.T;
  if (p.varlen) {
    int32_t* seg0 = reinterpret_cast<int32_t*>(w + l.seg0);
    a.seg0 = seg0;
    if (launch_prepare_segments(cu, p.N, p.T, pl.seglen, seg0, reinterpret_cast<int32_t*>(w + l.status), s) !=
        cudaSuccess)
      return GDN_ERR_CUDA;
  }
  if (pl.cut) {
    a.hseg = at(l.hseg), a.dtsum = at(l.dtsum);
    b.qseg = at(l.qseg), b.qdt = at(l.qdt);
    if (launch_segment_states(a, pl, p.dt, s) != cudaSuccess) return GDN_ERR_CUDA;
  }
  const cudaError_t e =
      p.dt == GDN_F32 ? dispatch_bwd<float>(b, pl, s) : dispatch_bwd<__nv_bfloat16>(b, pl, s);
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace gdn
