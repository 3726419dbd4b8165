// gdn_scan.cu -- the selective state space scan: prompts and training
// sequences (gdn_selective_scan_fwd) and single tokens on a state pool
// (gdn_selective_scan_step).  The recurrence, the layout of a warp and the
// scalar functions are in gdn_scan.cuh.
//
// Forward.  Each warp runs its channels through a segment of a sequence on its
// own (no block barrier): tiles of 16 tokens, whose x, delta, z, B and C are
// loaded one tile ahead into registers; the tile's steps (softplus), dt x, B and
// C go through a few KB of shared memory as fp32, and every token is then
//     a = 2^{dt A log2 e}, h = a h + (dt x) B, y = sum_n C h
// on 2 x 4 states a lane, the products on packed fp32 pairs.  The sums over the
// state lanes are reduce-scattered four tokens at a time, so that a lane ends
// with the token whose x and z it loaded.  Per state: one ex2 and four FMA-pipe
// operations, which both units (32 and 128 lanes a cycle) pass in the same time.
//
// Few chains.  When the channels of all sequences do not fill the SMs, sequences
// are cut into segments: a states-only pass runs every segment but a sequence's
// last from zero, a small kernel chains the segments' end states through their
// decays 2^{A log2 e sum dt}, and the full pass starts each segment from its
// state.  The states-only pass repeats the ex2 of the full pass, so nothing is
// cut when the chains are enough.
#include "gdn_scan.cuh"

namespace gdn {
namespace scan {
namespace {

constexpr int kWarps = 4;   // warps a CTA

template <typename T, int RL, bool STATES>
__global__ void __launch_bounds__(32 * kWarps) scan_kernel(const Args a) {
  using L = Lanes<RL>;
  __shared__ __align__(16) float sB[kWarps][L::TT][L::SP];
  __shared__ __align__(16) float sC[STATES ? 1 : kWarps][STATES ? 1 : L::TT][STATES ? 4 : L::SP];
  __shared__ __align__(16) float4 sdt[kWarps][L::TT][L::CL];
  const L ln;
  const int w = threadIdx.x >> 5;
  const int cb = blockIdx.y * kWarps + w;
  const int g = cb / a.cbg;
  if (g >= a.G) return;
  Unit u;
  if (!unit_of(a, blockIdx.x, u)) return;
  if (STATES && u.last) return;   // nobody starts from its end

  const int d = g * a.Dg + (cb - g * a.cbg) * L::CPW + 2 * ln.chl;   // this lane's channel pair
  const int dend = (g + 1) * a.Dg;
  const bool ok0 = d < dend, ok1 = d + 1 < dend;
  const int n0 = 4 * ln.sl, nn = a.S - n0;   // this lane's states
  const bool v4 = a.S % 4 == 0;

  // decay rates (base 2) and states, as packed pairs of states
  float2 A2[2][2], h[2][2];
#pragma unroll
  for (int c = 0; c < 2; ++c) {
    float r[4] = {0.f, 0.f, 0.f, 0.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
    if (c ? ok1 : ok0) {
      load4(a.A + (int64_t)(d + c) * a.S + n0, nn, v4, r);
      if (!STATES) {
        const float* from = nullptr;
        if (!u.first) from = a.hseg + ((int64_t)blockIdx.x * a.D + d + c) * a.S;
        else if (a.h0) from = a.h0 + ((int64_t)u.n * a.D + d + c) * a.S;
        if (from) load4(from + n0, nn, v4, s);
      }
    }
    A2[c][0] = make_float2(r[0] * sm100::kLog2e, r[1] * sm100::kLog2e);
    A2[c][1] = make_float2(r[2] * sm100::kLog2e, r[3] * sm100::kLog2e);
    h[c][0] = make_float2(s[0], s[1]);
    h[c][1] = make_float2(s[2], s[3]);
  }
  const float2 bias = make_float2(a.bias && ok0 ? a.bias[d] : 0.f, a.bias && ok1 ? a.bias[d + 1] : 0.f);
  const float2 skip = make_float2(a.Dp && ok0 ? a.Dp[d] : 0.f, a.Dp && ok1 ? a.Dp[d + 1] : 0.f);

  const T* px = static_cast<const T*>(a.x) + u.tok0 * a.ldx + d;
  const T* pd = static_cast<const T*>(a.dl) + u.tok0 * a.ldd + d;
  const T* pz = a.z ? static_cast<const T*>(a.z) + u.tok0 * a.ldz + d : nullptr;
  const T* pB = static_cast<const T*>(a.B) + u.tok0 * a.ldb + g * a.S;
  const T* pC = static_cast<const T*>(a.C) + u.tok0 * a.ldc + g * a.S;

  Raw2<T> rx[4], rd[4], rz[4], rB[L::NPB], rC[L::NPB];
  auto load_tile = [&](int t0) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int t = t0 + ln.token(k);
      rx[k].zero(), rd[k].zero(), rz[k].zero();
      if (t < u.len && ok0) {
        rx[k].load(px + t * a.ldx, a.vx, ok0, ok1);
        rd[k].load(pd + t * a.ldd, a.vd, ok0, ok1);
        if (!STATES && pz) rz[k].load(pz + t * a.ldz, a.vz, ok0, ok1);
      }
    }
#pragma unroll
    for (int i = 0; i < L::NPB; ++i) {
      const int p = ln.lane + 32 * i, t = t0 + p / (L::SP / 2), n = 2 * (p % (L::SP / 2));
      rB[i].zero(), rC[i].zero();
      if (p < L::TT * L::SP / 2 && t < u.len && n < a.S) {
        rB[i].load(pB + t * a.ldb + n, a.vb, true, n + 1 < a.S);
        if (!STATES) rC[i].load(pC + t * a.ldc + n, a.vc, true, n + 1 < a.S);
      }
    }
  };

  float2 dts = make_float2(0.f, 0.f);   // STATES: sum of this lane's steps
  load_tile(0);
  for (int t0 = 0; t0 < u.len; t0 += L::TT) {
    // this tile to shared memory, the next one's loads behind it
    float2 xs[4], zs[4];
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 x = rx[k].f();
      float2 dt = rd[k].f();
      dt.x += bias.x, dt.y += bias.y;
      if (a.softplus) {
        float e;
        dt.x = softplus(dt.x, e), dt.y = softplus(dt.y, e);
      }
      if (t0 + ln.token(k) >= u.len) dt = make_float2(0.f, 0.f);   // past the end: the state stays
      xs[k] = x;
      if (!STATES) zs[k] = rz[k].f();
      if (STATES) dts.x += dt.x, dts.y += dt.y;
      if (!ln.dup) sdt[w][ln.token(k)][ln.chl] = make_float4(dt.x, dt.x * x.x, dt.y, dt.y * x.y);
    }
#pragma unroll
    for (int i = 0; i < L::NPB; ++i) {
      const int p = ln.lane + 32 * i, t = p / (L::SP / 2), n = 2 * (p % (L::SP / 2));
      if (p < L::TT * L::SP / 2) {
        *reinterpret_cast<float2*>(&sB[w][t][n]) = rB[i].f();
        if constexpr (!STATES) *reinterpret_cast<float2*>(&sC[w][t][n]) = rC[i].f();
      }
    }
    __syncwarp();
    if (t0 + L::TT < u.len) load_tile(t0 + L::TT);

#pragma unroll
    for (int gr = 0; gr < L::NG; ++gr) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int t = 4 * gr + j;
        const float4 q = sdt[w][t][ln.chl];
        const float4 b = *reinterpret_cast<const float4*>(&sB[w][t][n0]);
        float4 cc;
        if constexpr (!STATES) cc = *reinterpret_cast<const float4*>(&sC[w][t][n0]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float dt = c ? q.z : q.x, ux = c ? q.w : q.y;
          const float2 dt2 = make_float2(dt, dt), ux2 = make_float2(ux, ux);
          const float2 e0 = __fmul2_rn(dt2, A2[c][0]), e1 = __fmul2_rn(dt2, A2[c][1]);
          const float2 a0 = make_float2(sm100::ex2_fast(e0.x), sm100::ex2_fast(e0.y));
          const float2 a1 = make_float2(sm100::ex2_fast(e1.x), sm100::ex2_fast(e1.y));
          h[c][0] = __ffma2_rn(a0, h[c][0], __fmul2_rn(ux2, make_float2(b.x, b.y)));
          h[c][1] = __ffma2_rn(a1, h[c][1], __fmul2_rn(ux2, make_float2(b.z, b.w)));
          if constexpr (!STATES) {
            float2 y2 = __fmul2_rn(h[c][0], make_float2(cc.x, cc.y));
            y2 = __ffma2_rn(h[c][1], make_float2(cc.z, cc.w), y2);
            v[2 * j + c] = y2.x + y2.y;
          }
        }
      }
      if constexpr (!STATES) {
        reduce_states<RL, 2>(v, ln.lane);
#pragma unroll
        for (int j = 0; j < L::TPL; ++j) {
          const int k = gr * L::TPL + j, t = t0 + ln.token(k);
          float2 o = make_float2(fmaf(skip.x, xs[k].x, v[2 * j]), fmaf(skip.y, xs[k].y, v[2 * j + 1]));
          if (pz) o.x *= zs[k].x * sigmoid(zs[k].x), o.y *= zs[k].y * sigmoid(zs[k].y);
          if (t < u.len && ok0 && !ln.dup)
            store2(static_cast<T*>(a.y) + (u.tok0 + t) * a.D + d, o, a.vy, ok0, ok1);
        }
      }
    }
  }

  // end states
  if constexpr (STATES) {
    if (ln.dup) dts = make_float2(0.f, 0.f);
#pragma unroll
    for (int m = 16; m >= L::CL && RL > 1; m >>= 1) {
      dts.x += __shfl_xor_sync(~0u, dts.x, m);
      dts.y += __shfl_xor_sync(~0u, dts.y, m);
    }
    if (ln.sl == 0) {
      if (ok0) a.dtsum[(int64_t)blockIdx.x * a.D + d] = dts.x;
      if (ok1) a.dtsum[(int64_t)blockIdx.x * a.D + d + 1] = dts.y;
    }
  }
  float* to = nullptr;
  if (STATES) to = a.hseg + (int64_t)blockIdx.x * a.D * a.S;
  else if (a.ht && u.last) to = a.ht + (int64_t)u.n * a.D * a.S;
  if (to) {
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const float s[4] = {h[c][0].x, h[c][0].y, h[c][1].x, h[c][1].y};
      if (c ? ok1 : ok0) store4(to + (int64_t)(d + c) * a.S + n0, nn, v4, s);
    }
  }
}

// hseg: local end states -> start states, a thread per (cut sequence, channel,
// state).
__global__ void __launch_bounds__(256) chain_kernel(const Args a) {
  const int64_t DS = (int64_t)a.D * a.S;
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int q = blockIdx.y + gridDim.y * blockIdx.z;
  if (i >= DS || q >= (a.cu ? a.seg0[a.N + 1] : a.N)) return;
  const int n = a.cu ? a.seg0[a.N + 2 + q] : q;
  const int d = (int)(i / a.S);
  const int64_t u0 = a.cu ? a.seg0[n] : (int64_t)n * a.nseg;
  const int64_t u1 = a.cu ? a.seg0[n + 1] : u0 + a.nseg;
  const float r = a.A[i] * sm100::kLog2e;
  float h = a.h0 ? a.h0[n * DS + i] : 0.f;
  for (int64_t u = u0; u + 1 < u1; ++u) {
    const float end = a.hseg[u * DS + i], dt = a.dtsum[u * a.D + d];
    if (u > u0) a.hseg[u * DS + i] = h;
    h = fmaf(sm100::ex2_fast(r * dt), h, end);
  }
  if (u1 > u0 + 1) a.hseg[(u1 - 1) * DS + i] = h;
}

// One CTA: checks cu_seqlens, writes every sequence's first segment and lists
// the sequences that have several (see Args::seg0).
__global__ void __launch_bounds__(1024) prepare_segments_kernel(const int32_t* __restrict__ cu, int N, int64_t T,
                                                                int seglen, int32_t* __restrict__ seg0,
                                                                int32_t* __restrict__ status) {
  __shared__ int64_t wsum[32];
  __shared__ int64_t carry;
  __shared__ int bad;
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  if (tid == 0) {
    bad = cu[0] != 0 || cu[N] != T;
    carry = 0;
  }
  __syncthreads();
  for (int64_t b = 0; b < N; b += 1024) {
    const int64_t n = b + tid;
    int64_t cnt = 0;   // segments, and 2^40 when there are several
    if (n < N) {
      const int64_t len = (int64_t)cu[n + 1] - cu[n];
      if (len < 0 || cu[n] < 0 || cu[n + 1] > T) bad = 1;
      else if (len <= seglen) cnt = 1;
      else cnt = (len + seglen - 1) / seglen + (1ll << 40);
    }
    int64_t s = cnt;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int64_t o = __shfl_up_sync(~0u, s, m);
      if (lane >= m) s += o;
    }
    if (lane == 31) wsum[w] = s;
    __syncthreads();
    if (w == 0) {
      int64_t t = wsum[lane];
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const int64_t o = __shfl_up_sync(~0u, t, m);
        if (lane >= m) t += o;
      }
      wsum[lane] = t;
    }
    __syncthreads();
    const int64_t before = carry + (w ? wsum[w - 1] : 0) + s - cnt;
    if (n < N && !bad) {   // a malformed batch may count more segments than there is room for
      seg0[n] = (int32_t)(before & ((1ll << 40) - 1));
      if (cnt >> 40) seg0[N + 2 + (before >> 40)] = (int32_t)n;
    }
    __syncthreads();
    if (tid == 1023) carry = before + cnt;
    __syncthreads();
  }
  if (tid == 0) {
    seg0[N] = bad ? -1 : (int32_t)(carry & ((1ll << 40) - 1));
    seg0[N + 1] = bad ? 0 : (int32_t)(carry >> 40);
    *status = bad ? GDN_DEV_BAD_CU_SEQLENS : GDN_DEV_OK;
  }
}

// ------------------------------------------------------------- single tokens

struct StepArgs {
  Args a;
  float* state;
  const int32_t* idx;
  int slots;
  int64_t Ttot;
};

// RL neighbouring lanes hold a channel's states, four each, so that a warp reads
// and writes 512 consecutive bytes of the pool.  Bound by the state's bytes (read
// and written once a call, with the evict-first hint: a pool is touched once a
// step).  Tokens of a sequence follow one another in registers.
template <typename T, int RL>
__global__ void __launch_bounds__(256) scan_step_kernel(const StepArgs p) {
  const Args& a = p.a;
  constexpr int CPB = 256 / RL;   // channels a CTA
  const int n = blockIdx.x;
  const int sl = threadIdx.x % RL, d = blockIdx.y * CPB + threadIdx.x / RL;
  const int64_t s0 = a.cu ? a.cu[n] : (int64_t)n * a.T;
  const int64_t len = a.cu ? (int64_t)a.cu[n + 1] - s0 : a.T;
  if (len <= 0 || s0 < 0 || s0 + len > p.Ttot) return;   // empty or malformed: touch nothing
  const bool ok = d < a.D;
  const int dd = ok ? d : a.D - 1;   // lanes past the end repeat the last channel and write nothing
  const int g = dd / a.Dg;
  const int slot = p.idx ? p.idx[n] : n;
  T* y = static_cast<T*>(a.y);
  if (slot < 0 || slot >= p.slots) {   // no state: zero outputs
    if (ok && sl == 0)
      for (int64_t t = 0; t < len; ++t) y[(s0 + t) * a.D + d] = from_f<T>(0.f);
    return;
  }
  const int n0 = 4 * sl, nn = a.S - n0;
  const bool v4 = a.S % 4 == 0;
  float* S = p.state + ((int64_t)slot * a.D + dd) * a.S + n0;
  float h[4], A2[4];
  if (v4 && nn >= 4) {
    const float4 q = __ldcs(reinterpret_cast<const float4*>(S));
    h[0] = q.x, h[1] = q.y, h[2] = q.z, h[3] = q.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = i < nn ? S[i] : 0.f;
  }
  load4(a.A + (int64_t)dd * a.S + n0, nn, v4, A2);
#pragma unroll
  for (int i = 0; i < 4; ++i) A2[i] *= sm100::kLog2e;
  const float bias = a.bias ? a.bias[dd] : 0.f, skip = a.Dp ? a.Dp[dd] : 0.f;
  const T* px = static_cast<const T*>(a.x) + s0 * a.ldx + dd;
  const T* pd = static_cast<const T*>(a.dl) + s0 * a.ldd + dd;
  const T* pz = a.z ? static_cast<const T*>(a.z) + s0 * a.ldz + dd : nullptr;
  const T* pB = static_cast<const T*>(a.B) + s0 * a.ldb + g * a.S + n0;
  const T* pC = static_cast<const T*>(a.C) + s0 * a.ldc + g * a.S + n0;
  for (int64_t t = 0; t < len; ++t) {
    const float x = to_f(px[t * a.ldx]);
    float dt = to_f(pd[t * a.ldd]) + bias;
    const float z = pz ? to_f(pz[t * a.ldz]) : 0.f;
    float b[4], c[4];
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      Raw2<T> rb, rc;
      rb.zero(), rc.zero();
      if (i < nn) {
        rb.load(pB + t * a.ldb + i, a.vb, true, i + 1 < nn);
        rc.load(pC + t * a.ldc + i, a.vc, true, i + 1 < nn);
      }
      const float2 fb = rb.f(), fc = rc.f();
      b[i] = fb.x, b[i + 1] = fb.y, c[i] = fc.x, c[i + 1] = fc.y;
    }
    if (a.softplus) {
      float e;
      dt = softplus(dt, e);
    }
    const float ux = dt * x;
    float o = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = fmaf(sm100::ex2_fast(dt * A2[i]), h[i], ux * b[i]);
      o = fmaf(c[i], h[i], o);
    }
#pragma unroll
    for (int m = 1; m < RL; m <<= 1) o += __shfl_xor_sync(~0u, o, m);
    o = fmaf(skip, x, o);
    if (pz) o *= z * sigmoid(z);
    if (ok && sl == 0) y[(s0 + t) * a.D + d] = from_f<T>(o);
  }
  if (!ok) return;
  if (v4 && nn >= 4) {
    __stcs(reinterpret_cast<float4*>(S), make_float4(h[0], h[1], h[2], h[3]));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < nn) S[i] = h[i];
  }
}

template <typename F>
void by_lanes(int RL, F&& f) {
  switch (RL) {
    case 1: f(std::integral_constant<int, 1>()); break;
    case 2: f(std::integral_constant<int, 2>()); break;
    case 4: f(std::integral_constant<int, 4>()); break;
    case 8: f(std::integral_constant<int, 8>()); break;
    default: f(std::integral_constant<int, 16>()); break;
  }
}

template <typename T, bool STATES>
void launch_scan(const Args& a, const Plan& pl, cudaStream_t s) {
  const dim3 grid((unsigned)pl.max_units, (unsigned)ceil_div((int64_t)a.G * a.cbg, kWarps));
  by_lanes(pl.RL, [&](auto rl) { scan_kernel<T, decltype(rl)::value, STATES><<<grid, 32 * kWarps, 0, s>>>(a); });
}

bool pairs(const void* p, size_t es, int64_t ld, bool rows_even) {
  return rows_even && ld % 2 == 0 && reinterpret_cast<uintptr_t>(p) % (2 * es) == 0;
}

struct Layout {
  size_t status, seg0, hseg, dtsum, total;
};

Layout layout_of(const gdn_scan_problem& p, const Plan& pl) {
  Layout l;
  size_t o = 0;
  l.status = o, o += kAlign;
  l.seg0 = o, o += p.varlen ? align_up(seg0_bytes(p.N, p.T, pl.seglen)) : 0;
  l.hseg = o, o += pl.cut ? align_up(sizeof(float) * (size_t)pl.max_units * p.D * p.S) : 0;
  l.dtsum = o, o += pl.cut ? align_up(sizeof(float) * (size_t)pl.max_units * p.D) : 0;
  l.total = o;
  return l;
}

}  // namespace

Plan make_plan(const gdn_scan_problem& p) {
  Plan pl;
  pl.RL = lanes_for(p.S);
  pl.cpw = 64 / pl.RL;
  pl.cbg = (int)ceil_div(p.D / p.G, pl.cpw);
  const int64_t cw = (int64_t)p.G * pl.cbg;         // warps a line of tokens
  const int64_t slots = (int64_t)sm_count() * 8;    // warps that fill the SMs
  if (p.varlen) {
    int64_t len = align_up((size_t)(p.T * cw / slots), kTileMax);
    if (len < 128) len = 128;
    pl.seglen = (int)len;
    pl.nseg = 1;
    pl.max_units = p.T / len + p.N;
    pl.cut = p.T > len;
  } else {
    int64_t n = 1;
    if (p.B * cw < slots) n = ceil_div(slots, p.B * cw);
    if (n > p.T / 128) n = p.T / 128 > 1 ? p.T / 128 : 1;
    pl.seglen = (int)align_up((size_t)ceil_div(p.T, n), kTileMax);
    pl.nseg = (int)ceil_div(p.T, pl.seglen);
    pl.max_units = (int64_t)p.B * pl.nseg;
    pl.cut = pl.nseg > 1;
  }
  return pl;
}

Args base_args(const gdn_scan_problem& p, const Plan& pl, const void* x, const void* delta, const float* A,
               const void* B, const void* C, const float* Dp, const void* z, const float* dt_bias, const float* h0,
               const int32_t* cu) {
  Args a = {};
  const size_t es = p.dt == GDN_F32 ? 4 : 2;
  a.x = x, a.dl = delta, a.z = z, a.B = B, a.C = C;
  a.A = A, a.Dp = Dp, a.bias = dt_bias, a.h0 = h0;
  a.cu = p.varlen ? cu : nullptr;
  a.D = p.D, a.S = p.S, a.G = p.G, a.Dg = p.D / p.G;
  const int64_t gs = (int64_t)p.G * p.S;
  a.ldx = p.ld_x ? p.ld_x : p.D;
  a.ldd = p.ld_delta ? p.ld_delta : p.D;
  a.ldz = p.ld_z ? p.ld_z : p.D;
  a.ldb = p.ld_b ? p.ld_b : gs;
  a.ldc = p.ld_c ? p.ld_c : gs;
  a.T = p.T, a.N = p.N;
  a.cbg = pl.cbg, a.nseg = pl.nseg, a.seglen = pl.seglen;
  a.softplus = p.softplus;
  const bool even = a.Dg % 2 == 0;
  a.vx = pairs(x, es, a.ldx, even);
  a.vd = pairs(delta, es, a.ldd, even);
  a.vz = pairs(z, es, a.ldz, even);
  a.vb = pairs(B, es, a.ldb, a.S % 2 == 0);
  a.vc = pairs(C, es, a.ldc, a.S % 2 == 0);
  return a;
}

cudaError_t launch_prepare_segments(const int32_t* cu, int N, int64_t T, int seglen, int32_t* seg0, int32_t* status,
                                    cudaStream_t s) {
  prepare_segments_kernel<<<1, 1024, 0, s>>>(cu, N, T, seglen, seg0, status);
  return cudaGetLastError();
}

cudaError_t launch_segment_states(const Args& a, const Plan& pl, gdn_dtype dt, cudaStream_t s) {
  if (dt == GDN_F32) launch_scan<float, true>(a, pl, s);
  else launch_scan<__nv_bfloat16, true>(a, pl, s);
  const int64_t ncut = a.cu ? max_cut(a.N, a.T, a.seglen) : a.N;   // sequences that may have several segments
  const int64_t ny = ncut < 32768 ? ncut : 32768;
  const dim3 grid((unsigned)ceil_div((int64_t)a.D * a.S, 256), (unsigned)ny, (unsigned)ceil_div(ncut, ny));
  chain_kernel<<<grid, 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace scan

using namespace scan;

size_t scan_fwd_workspace_bytes(const gdn_scan_problem& p) { return layout_of(p, make_plan(p)).total; }

gdn_status run_scan_fwd(const gdn_scan_problem& p, const void* x, const void* delta, const float* A, const void* B,
                        const void* C, const float* Dp, const void* z, const float* dt_bias, const float* h0,
                        const int32_t* cu, void* y, float* ht, void* ws, cudaStream_t s) {
  const Plan pl = make_plan(p);
  const Layout l = layout_of(p, pl);
  Args a = base_args(p, pl, x, delta, A, B, C, Dp, z, dt_bias, h0, cu);
  char* w = static_cast<char*>(ws);
  a.y = y, a.ht = ht;
  a.vy = pairs(y, p.dt == GDN_F32 ? 4 : 2, p.D, a.Dg % 2 == 0);
  if (p.varlen) {
    a.seg0 = reinterpret_cast<int32_t*>(w + l.seg0);
    if (launch_prepare_segments(cu, p.N, p.T, pl.seglen, reinterpret_cast<int32_t*>(w + l.seg0),
                                reinterpret_cast<int32_t*>(w + l.status), s) != cudaSuccess)
      return GDN_ERR_CUDA;
  }
  if (pl.cut) {
    a.hseg = reinterpret_cast<float*>(w + l.hseg);
    a.dtsum = reinterpret_cast<float*>(w + l.dtsum);
    if (launch_segment_states(a, pl, p.dt, s) != cudaSuccess) return GDN_ERR_CUDA;
  }
  if (p.dt == GDN_F32) launch_scan<float, false>(a, pl, s);
  else launch_scan<__nv_bfloat16, false>(a, pl, s);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status run_scan_step(const gdn_scan_problem& p, const void* x, const void* delta, const float* A, const void* B,
                         const void* C, const float* Dp, const void* z, const float* dt_bias, float* state,
                         const int32_t* state_indices, int state_slots, const int32_t* cu, void* y, cudaStream_t s) {
  const Plan pl = make_plan(p);
  StepArgs sa;
  sa.a = base_args(p, pl, x, delta, A, B, C, Dp, z, dt_bias, nullptr, cu);
  sa.a.y = y;
  sa.state = state, sa.idx = state_indices, sa.slots = state_slots;
  sa.Ttot = (int64_t)p.B * p.T;
  by_lanes(pl.RL, [&](auto rl) {
    constexpr int R = decltype(rl)::value;
    const dim3 grid(p.N, (unsigned)ceil_div(p.D, 256 / R));
    if (p.dt == GDN_F32) scan_step_kernel<float, R><<<grid, 256, 0, s>>>(sa);
    else scan_step_kernel<__nv_bfloat16, R><<<grid, 256, 0, s>>>(sa);
  });
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace gdn
