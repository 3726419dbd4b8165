// gdn_scan.cu -- the selective state space scan: prompts and training
// sequences (gdn_selective_scan_fwd) and single tokens on a state pool
// (gdn_selective_scan_step).  The recurrence, the layout of a warp and the
// scalar functions are in gdn_scan.cuh.
//
// Forward.  Each warp runs its channels through a segment of a sequence on its
// own (no block barrier): tiles of 16 tokens, whose x, delta, z, B and C come by
// asynchronous copies two tiles ahead (rows that are not aligned: through
// registers); the tile's steps (softplus), dt x, B and
// C go through a few KB of shared memory as fp32, and every token is then
//     a = 2^{dt A log2 e}, h = a h + (dt x) B, y = sum_n C h
// on 2 x 4 states a lane, the products on packed fp32 pairs.  The sums over the
// state lanes are reduce-scattered four tokens at a time, so that a lane ends
// with the token whose x and z it loaded.  Per state: one ex2 and four FMA-pipe
// operations, which both units (32 and 128 lanes a cycle) pass in the same time.
//
// What bounds it (one GB300): neither unit nor HBM, but issue and latency at the
// few warps that the chains make.  57 instructions a token and warp (256 updates),
// IPC 2.0 of 4, where a packed pair takes two issue slots; ex2 34 %, LSU wavefronts
// 49 %, DRAM 14 % (by ncu).  4096 channels, 16 states, bf16, gated: 4 x 8192 tokens
// 0.81 ms, 1 x 4096 tokens 0.148 ms in seven segments (states 56 us, chain 4,
// outputs 86).
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

// Warps a CTA (they share nothing; the widest layout's tiles need the room).
constexpr int warps_of(int RL) { return RL == 16 ? 2 : 4; }
constexpr int kRing = 3;   // tiles as loaded: one in use, two on their way

// Shared memory of a warp: the tile being run as fp32, and tiles as loaded.
template <typename T, int RL, bool STATES>
struct Tiles {
  using L = Lanes<RL>;
  static constexpr int NZ = STATES ? 1 : L::TT;
  float4 dt[L::TT][L::CL];   // dt, dt x of a channel pair
  float B[L::TT][L::SP], C[NZ][L::SP];
  alignas(16) T rx[kRing][L::TT][L::CPW];
  alignas(16) T rd[kRing][L::TT][L::CPW];
  alignas(16) T rz[STATES ? 1 : kRing][NZ][L::CPW];
  alignas(16) T rB[kRing][L::TT][L::SP];
  alignas(16) T rC[STATES ? 1 : kRing][NZ][L::SP];
};

template <typename T, int RL, bool STATES, bool GATE, int ROWS>
__global__ void __launch_bounds__(32 * warps_of(RL), 3) scan_kernel(const Args a) {
  using L = Lanes<RL>;
  constexpr bool ASYNC = ROWS != kRegs;
  constexpr int XROW = L::CPW * sizeof(T), SROW = L::SP * sizeof(T), CX = chunk<ROWS, XROW>(), CB = chunk<ROWS, SROW>();
  constexpr int W = warps_of(RL);
  constexpr int VE = RowVec<T, RL>::VE, NV = RowVec<T, RL>::NV, NPV = (NV + 31) / 32;
  extern __shared__ __align__(16) char raw_smem[];
  const L ln;
  const int w = threadIdx.x >> 5;
  Tiles<T, RL, STATES>& sm = reinterpret_cast<Tiles<T, RL, STATES>*>(raw_smem)[w];
  const int cb = blockIdx.y * W + w;
  const int g = cb / a.cbg;
  if (g >= a.G) return;
  Unit u;
  // (the states pass leaves out every sequence's last segment, from whose end nobody
  // starts; equal lengths do not even launch it, or the CTAs that do run would share
  // half of the SMs)
  const int64_t un = STATES && !a.cu ? blockIdx.x / (a.nseg - 1) * a.nseg + blockIdx.x % (a.nseg - 1) : blockIdx.x;
  if (!unit_of(a, un, u)) return;
  if (STATES && u.last) return;

  const int dw = g * a.Dg + (cb - g * a.cbg) * L::CPW, d = dw + 2 * ln.chl;   // the warp's and this lane's channels
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
        // (a cut sequence's first segment too: ht, which its last one writes, may be h0)
        if (!u.first || !u.last) from = a.hseg + (un * a.D + d + c) * a.S;
        else if (a.h0) from = a.h0 + ((int64_t)u.n * a.D + d + c) * a.S;
        if (from) load4(from + n0, nn, v4, s);
      }
    }
    A2[c][0] = make_float2(rate2(r[0]), rate2(r[1]));
    A2[c][1] = make_float2(rate2(r[2]), rate2(r[3]));
    h[c][0] = make_float2(s[0], s[1]);
    h[c][1] = make_float2(s[2], s[3]);
  }
  const float2 bias = make_float2(a.bias && ok0 ? a.bias[d] : 0.f, a.bias && ok1 ? a.bias[d + 1] : 0.f);
  const float2 skip = make_float2(a.Dp && ok0 ? a.Dp[d] : 0.f, a.Dp && ok1 ? a.Dp[d + 1] : 0.f);

  // the warp's first row of every tensor
  const char* px = static_cast<const char*>(a.x) + u.tok0 * a.bx + dw * (int64_t)sizeof(T);
  const char* pd = static_cast<const char*>(a.dl) + u.tok0 * a.bd + dw * (int64_t)sizeof(T);
  const char* pz = static_cast<const char*>(a.z) + u.tok0 * a.bz + dw * (int64_t)sizeof(T);
  const char* pB = static_cast<const char*>(a.B) + u.tok0 * a.bb + g * a.S * (int64_t)sizeof(T);
  const char* pC = static_cast<const char*>(a.C) + u.tok0 * a.bc + g * a.S * (int64_t)sizeof(T);
  T* py = static_cast<T*>(a.y) + u.tok0 * a.D + d;

  // A tile's rows into ring slot r: by copies, or in two steps through registers.
  Raw2<T> gx[4], gd[4], gz[4];
  uint4 gB[NPV], gC[NPV];
  auto fetch = [&](int t0, int r) {
    if constexpr (ASYNC) {
      const int vx = (dend - dw) * (int)sizeof(T), vs = a.S * (int)sizeof(T);
      copy_rows<L::TT, XROW, CX>((char*)&sm.rx[r][0][0], px, a.bx, t0, u.len, vx, ln.lane);
      copy_rows<L::TT, XROW, CX>((char*)&sm.rd[r][0][0], pd, a.bd, t0, u.len, vx, ln.lane);
      copy_rows<L::TT, SROW, CB>((char*)&sm.rB[r][0][0], pB, a.bb, t0, u.len, vs, ln.lane);
      if constexpr (!STATES) {
        copy_rows<L::TT, SROW, CB>((char*)&sm.rC[r][0][0], pC, a.bc, t0, u.len, vs, ln.lane);
        if (GATE) copy_rows<L::TT, XROW, CX>((char*)&sm.rz[r][0][0], pz, a.bz, t0, u.len, vx, ln.lane);
      }
      copies_commit();
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int t = t0 + ln.token(k);
        gx[k].zero(), gd[k].zero(), gz[k].zero();
        if (t < u.len && ok0) {
          gx[k].load(row((const T*)px, t, a.bx) + 2 * ln.chl, a.vin, ok0, ok1);
          gd[k].load(row((const T*)pd, t, a.bd) + 2 * ln.chl, a.vin, ok0, ok1);
          if (!STATES && GATE) gz[k].load(row((const T*)pz, t, a.bz) + 2 * ln.chl, a.vin, ok0, ok1);
        }
      }
#pragma unroll
      for (int i = 0; i < NPV; ++i) {
        const int p = (ln.lane + 32 * i) * VE, t = t0 + p / L::SP, n = p % L::SP;
        gB[i] = gC[i] = make_uint4(0u, 0u, 0u, 0u);
        if ((NV % 32 == 0 || ln.lane + 32 * i < NV) && t < u.len) {
          gB[i] = load_row16<T, VE>(row((const T*)pB, t, a.bb), n, a.S, a.vbc);
          if (!STATES) gC[i] = load_row16<T, VE>(row((const T*)pC, t, a.bc), n, a.S, a.vbc);
        }
      }
    }
  };
  auto fetched = [&](int r) {   // the registers' tile into slot r
    if constexpr (!ASYNC) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int t = ln.token(k), c = 2 * ln.chl;
        gx[k].store(&sm.rx[r][t][c]), gd[k].store(&sm.rd[r][t][c]);
        if constexpr (!STATES && GATE) gz[k].store(&sm.rz[r][t][c]);
      }
#pragma unroll
      for (int i = 0; i < NPV; ++i) {
        if (NV % 32 == 0 || ln.lane + 32 * i < NV) {
          const int p = (ln.lane + 32 * i) * VE;
          copy_vec<VE * sizeof(T)>(&sm.rB[r][0][0] + p, gB[i]);
          if constexpr (!STATES) copy_vec<VE * sizeof(T)>(&sm.rC[r][0][0] + p, gC[i]);
        }
      }
    }
  };

  float2 xs[4], zs[4];                  // x and z of this lane's tokens of the tile being run
  float2 dts = make_float2(0.f, 0.f);   // STATES: sum of this lane's steps
  // One of this lane's tokens of ring slot r's tile (first token t0) as fp32; past the sequence's end steps and inputs are zero: the state stays.
  auto stage = [&](int k, int t0, int r) {
    const int t = ln.token(k), c = 2 * ln.chl;
    Raw2<T> x, e;
    x.load_shared(&sm.rx[r][t][c]), e.load_shared(&sm.rd[r][t][c]);
    float2 dt = __fadd2_rn(e.f(), bias);
    if (a.softplus) {
      float2 ex;
      dt = softplus2(dt, ex);
    }
    xs[k] = x.f();
    if constexpr (!STATES && GATE) {
      Raw2<T> z;
      z.load_shared(&sm.rz[r][t][c]);
      zs[k] = z.f();
    }
    const float2 dx = __fmul2_rn(dt, xs[k]);   // x is zero past the end
    if (t0 + t >= u.len) dt = make_float2(0.f, 0.f);
    if (STATES) dts = __fadd2_rn(dts, dt);
    if (!ln.dup) sm.dt[t][ln.chl] = make_float4(dt.x, dt.y, dx.x, dx.y);
  };
  auto stage_rows = [&](int r) {
#pragma unroll
    for (int i = 0; i < NPV; ++i) {
      if (NV % 32 == 0 || ln.lane + 32 * i < NV) {
        const int p = (ln.lane + 32 * i) * VE;
        put_row16<T, VE>(&sm.B[0][0] + p, get_vec<VE * sizeof(T)>(&sm.rB[r][0][0] + p));
        if constexpr (!STATES) put_row16<T, VE>(&sm.C[0][0] + p, get_vec<VE * sizeof(T)>(&sm.rC[r][0][0] + p));
      }
    }
  };

  const int ntile = (u.len + L::TT - 1) / L::TT;
  if (ntile > 0) {
#pragma unroll
    for (int i = 0; i < kRing - 1; ++i) fetch(i * L::TT, i), fetched(i);
  }
  for (int i = 0, r = 0; i < ntile; ++i) {
    const int t0 = i * L::TT;
    const int rn = r == 0 ? kRing - 1 : r - 1;   // the slot that tile i - 1 has left
    if (ASYNC) copies_wait<kRing - 2>();
    __syncwarp();
    fetch(t0 + (kRing - 1) * L::TT, rn);
#pragma unroll
    for (int k = 0; k < 4; ++k) stage(k, t0, r);
    stage_rows(r);
    __syncwarp();
#pragma unroll
    for (int gr = 0; gr < L::NG; ++gr) {
      // four tokens' decays and inputs, then the recurrence over them
      float v[8];
      float2 aa[4][2][2], uu[4][2][2];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float4 q = sm.dt[4 * gr + j][ln.chl];
        const float4 bb = *reinterpret_cast<const float4*>(&sm.B[4 * gr + j][n0]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float dc = c ? q.y : q.x, ux = c ? q.w : q.z;
          const float2 dt2 = make_float2(dc, dc), ux2 = make_float2(ux, ux);
          aa[j][c][0] = decay2(dt2, A2[c][0]);
          aa[j][c][1] = decay2(dt2, A2[c][1]);
          uu[j][c][0] = __fmul2_rn(ux2, make_float2(bb.x, bb.y));
          uu[j][c][1] = __fmul2_rn(ux2, make_float2(bb.z, bb.w));
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float4 cc;
        if constexpr (!STATES) cc = *reinterpret_cast<const float4*>(&sm.C[4 * gr + j][n0]);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          h[c][0] = __ffma2_rn(aa[j][c][0], h[c][0], uu[j][c][0]);
          h[c][1] = __ffma2_rn(aa[j][c][1], h[c][1], uu[j][c][1]);
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
          float2 o = __ffma2_rn(skip, xs[k], make_float2(v[2 * j], v[2 * j + 1]));
          if constexpr (GATE) {
            const float2 nl = __fmul2_rn(zs[k], make_float2(-sm100::kLog2e, -sm100::kLog2e));
            const float2 den = __fadd2_rn(make_float2(sm100::ex2_fast(nl.x), sm100::ex2_fast(nl.y)), make_float2(1.f, 1.f));
            o = __fmul2_rn(__fmul2_rn(o, zs[k]), make_float2(rcp_approx(den.x), rcp_approx(den.y)));
          }
          if constexpr (ASYNC) {   // the rows are even: both channels or none
            if (t < u.len && ok1 && !ln.dup) store2(py + (int64_t)t * a.D, o);
          } else if (t < u.len && ok0 && !ln.dup) {
            store2(py + (int64_t)t * a.D, o, a.vy, ok0, ok1);
          }
        }
      }
    }
    if (!ASYNC) fetched(rn);
    r = r + 1 == kRing ? 0 : r + 1;
  }
  if (ASYNC) copies_wait<0>();

  // end states
  if constexpr (STATES) {
    if (ln.dup) dts = make_float2(0.f, 0.f);
#pragma unroll
    for (int m = 16; m >= L::CL && RL > 1; m >>= 1) {
      dts.x += __shfl_xor_sync(~0u, dts.x, m);
      dts.y += __shfl_xor_sync(~0u, dts.y, m);
    }
    if (ln.sl == 0) {
      if (ok0) a.dtsum[un * a.D + d] = dts.x;
      if (ok1) a.dtsum[un * a.D + d + 1] = dts.y;
    }
  }
  float* to = nullptr;
  if (STATES) to = a.hseg + un * a.D * a.S;
  else if (a.ht && u.last) {
    const int r = a.slot ? a.slot[u.n] : u.n;
    if (!a.slot || (r >= 0 && r < a.slots)) to = a.ht + (int64_t)r * a.D * a.S;
  }
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
  const float r = rate2(a.A[i]);
  float h = a.h0 ? a.h0[n * DS + i] : 0.f;
  // eight segments' loads at a time
  for (int64_t u = u0; u + 1 < u1; u += 8) {
    float end[8], dt[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const bool in = u + k + 1 < u1;
      end[k] = in ? a.hseg[(u + k) * DS + i] : 0.f;
      dt[k] = in ? a.dtsum[(u + k) * a.D + d] : 0.f;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (u + k + 1 >= u1) break;
      a.hseg[(u + k) * DS + i] = h;
      h = fmaf(sm100::ex2_fast(r * dt[k]), h, end[k]);
    }
  }
  a.hseg[(u1 - 1) * DS + i] = h;
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
  for (int i = 0; i < 4; ++i) A2[i] = rate2(A2[i]);
  const float bias = a.bias ? a.bias[dd] : 0.f, skip = a.Dp ? a.Dp[dd] : 0.f;
  const T* px = reinterpret_cast<const T*>(static_cast<const char*>(a.x) + s0 * a.bx) + dd;
  const T* pd = reinterpret_cast<const T*>(static_cast<const char*>(a.dl) + s0 * a.bd) + dd;
  const T* pz = reinterpret_cast<const T*>(static_cast<const char*>(a.z) + s0 * a.bz) + dd;
  const T* pB = reinterpret_cast<const T*>(static_cast<const char*>(a.B) + s0 * a.bb) + g * a.S + n0;
  const T* pC = reinterpret_cast<const T*>(static_cast<const char*>(a.C) + s0 * a.bc) + g * a.S + n0;
  for (int t = 0; t < len; ++t) {
    const float x = to_f(*row(px, t, a.bx));
    float dt = to_f(*row(pd, t, a.bd)) + bias;
    const float z = a.z ? to_f(*row(pz, t, a.bz)) : 0.f;
    float b[4], c[4];
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      Raw2<T> rb, rc;
      rb.zero(), rc.zero();
      if (i < nn) {
        rb.load(row(pB, t, a.bb) + i, a.vbc, true, i + 1 < nn);
        rc.load(row(pC, t, a.bc) + i, a.vbc, true, i + 1 < nn);
      }
      const float2 fb = rb.f(), fc = rc.f();
      b[i] = fb.x, b[i + 1] = fb.y, c[i] = fc.x, c[i + 1] = fc.y;
    }
    if (a.softplus) dt = softplus(dt);
    const float ux = dt * x;
    float o = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      h[i] = fmaf(decay(dt, A2[i]), h[i], ux * b[i]);
      o = fmaf(c[i], h[i], o);
    }
#pragma unroll
    for (int m = 1; m < RL; m <<= 1) o += __shfl_xor_sync(~0u, o, m);
    o = fmaf(skip, x, o);
    if (a.z) o *= z * sigmoid(z);
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

// One token a sequence: a thread takes a channel's states (or two quarters of them,
// 4 RL apart, so that neighbouring lanes stay on neighbouring 16 bytes) of NSEQ
// sequences, whose loads are all on their way before the first is used; decay rates
// and the rest of a channel's parameters are read once.  512 sequences, 4096 channels,
// 16 states, bf16 (286 MB): 60 us, 4.8 TB/s, with two sequences and four CTAs an SM;
// 66 with four sequences and two CTAs; 100 with one sequence and a quarter a thread.
template <typename T, int RL, int NQ, int NSEQ>
__global__ void __launch_bounds__(256, 4) scan_token_kernel(const StepArgs p) {
  const Args& a = p.a;
  constexpr int CPB = 256 / RL;   // channels a CTA
  const int nfirst = blockIdx.x * NSEQ;
  const int sl = threadIdx.x % RL, d = blockIdx.y * CPB + threadIdx.x / RL;
  const bool ok = d < a.D;
  const int dd = ok ? d : a.D - 1;   // lanes past the end repeat the last channel and write nothing
  const int g = dd / a.Dg;
  const bool v4 = a.S % 4 == 0;
  int slot[NSEQ];
#pragma unroll
  for (int i = 0; i < NSEQ; ++i) {
    const int n = nfirst + i;
    slot[i] = -2;   // no sequence
    if (n < a.N) {
      const int k = p.idx ? p.idx[n] : n;
      slot[i] = k >= 0 && k < p.slots ? k : -1;   // -1: no state, zero output
    }
  }
  float h[NSEQ][NQ][4];
  Raw4<T> rB[NSEQ][NQ], rC[NSEQ][NQ];
  T rx[NSEQ], rd[NSEQ], rz[NSEQ];
#pragma unroll
  for (int i = 0; i < NSEQ; ++i) {
    const int n = nfirst + i;
    if (slot[i] < 0) continue;
    const float* S = p.state + ((int64_t)slot[i] * a.D + dd) * a.S;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int n0 = 4 * (sl + RL * q), nn = a.S - n0;
      if (v4 && nn >= 4) {
        const float4 v = __ldcs(reinterpret_cast<const float4*>(S + n0));
        h[i][q][0] = v.x, h[i][q][1] = v.y, h[i][q][2] = v.z, h[i][q][3] = v.w;
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) h[i][q][j] = j < nn ? S[n0 + j] : 0.f;
      }
      rB[i][q].load(row(static_cast<const T*>(a.B), n, a.bb) + g * a.S + n0, nn, a.vbc);
      rC[i][q].load(row(static_cast<const T*>(a.C), n, a.bc) + g * a.S + n0, nn, a.vbc);
    }
    rx[i] = row(static_cast<const T*>(a.x), n, a.bx)[dd];
    rd[i] = row(static_cast<const T*>(a.dl), n, a.bd)[dd];
    rz[i] = a.z ? row(static_cast<const T*>(a.z), n, a.bz)[dd] : from_f<T>(0.f);
  }
  float A2[NQ][4];
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    load4(a.A + (int64_t)dd * a.S + 4 * (sl + RL * q), a.S - 4 * (sl + RL * q), v4, A2[q]);
#pragma unroll
    for (int j = 0; j < 4; ++j) A2[q][j] = rate2(A2[q][j]);
  }
  const float bias = a.bias ? a.bias[dd] : 0.f, skip = a.Dp ? a.Dp[dd] : 0.f;
  T* y = static_cast<T*>(a.y);
#pragma unroll
  for (int i = 0; i < NSEQ; ++i) {
    const int n = nfirst + i;
    if (slot[i] == -2) break;
    if (slot[i] == -1) {   // (the same for the whole CTA)
      if (ok && sl == 0) y[(int64_t)n * a.D + d] = from_f<T>(0.f);
      continue;
    }
    const float x = to_f(rx[i]);
    float dt = to_f(rd[i]) + bias;
    if (a.softplus) dt = softplus(dt);
    const float ux = dt * x;
    const float2 dt2 = make_float2(dt, dt), ux2 = make_float2(ux, ux);
    float2 o2 = make_float2(0.f, 0.f);
    float* S = p.state + ((int64_t)slot[i] * a.D + dd) * a.S;
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float2 hn = __ffma2_rn(decay2(dt2, make_float2(A2[q][2 * j], A2[q][2 * j + 1])),
                                     make_float2(h[i][q][2 * j], h[i][q][2 * j + 1]), __fmul2_rn(ux2, j ? rB[i][q].hi() : rB[i][q].lo()));
        h[i][q][2 * j] = hn.x, h[i][q][2 * j + 1] = hn.y;
        o2 = __ffma2_rn(j ? rC[i][q].hi() : rC[i][q].lo(), hn, o2);
      }
      const int n0 = 4 * (sl + RL * q), nn = a.S - n0;
      if (ok) {
        if (v4 && nn >= 4) {
          __stcs(reinterpret_cast<float4*>(S + n0), make_float4(h[i][q][0], h[i][q][1], h[i][q][2], h[i][q][3]));
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (j < nn) S[n0 + j] = h[i][q][j];
        }
      }
    }
    float o = o2.x + o2.y;
#pragma unroll
    for (int m = 1; m < RL; m <<= 1) o += __shfl_xor_sync(~0u, o, m);
    o = fmaf(skip, x, o);
    if (a.z) {
      const float z = to_f(rz[i]);
      o *= z * sigmoid(z);
    }
    if (ok && sl == 0) y[(int64_t)n * a.D + d] = from_f<T>(o);
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
  by_lanes(pl.RL, [&](auto rl) {
    constexpr int R = decltype(rl)::value, W = warps_of(R);
    const int64_t units = STATES && !a.cu ? pl.max_units - a.N : pl.max_units;
    const dim3 grid((unsigned)units, (unsigned)ceil_div((int64_t)a.G * a.cbg, W));
    const size_t bytes = W * sizeof(Tiles<T, R, STATES>);
    auto go = [&](auto gate) {
      constexpr bool Z = decltype(gate)::value;
      auto* k = a.rows == kWide     ? scan_kernel<T, R, STATES, Z, kWide>
                : a.rows == kNarrow ? scan_kernel<T, R, STATES, Z, kNarrow>
                                    : scan_kernel<T, R, STATES, Z, kRegs>;
      if (bytes > 48 * 1024) cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
      k<<<grid, 32 * W, bytes, s>>>(a);
    };
    if constexpr (STATES) go(std::false_type());
    else if (a.z) go(std::true_type());
    else go(std::false_type());
  });
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
  const int64_t cw = (int64_t)p.G * pl.cbg;              // warps a line of tokens
  // Warps that the SMs hold in most layouts: three CTAs of four each.  (By their tiles'
  // shared memory fp32 with 9 to 32 states holds 8, more than 32 states 10 in bf16 and 6
  // in fp32; the rules below were measured in bf16 with 16 states, and cut those prompts
  // into more segments than run at once.)
  const int64_t fill = (int64_t)sm_count() * 12;
  // A cut costs a second run over all tokens but the last segments'.  Equal lengths
  // are cut when fewer than three warps an SM would run, into as many segments as run
  // at once (one GB300, 4096 channels, 16 states: 1 x 4096 tokens, 256 warps, 291 us
  // uncut, 185 / 170 / 150 / 161 / 179 in 4 / 6 / 7 / 8 / 9 segments; 4 x 8192 tokens,
  // 1024 warps, 811 us uncut, 1051 in two).  Packed sequences, whose lengths the host does not know, are
  // cut so that the longest ones do not outlast the rest (64 sequences of up to 2048
  // tokens, 2048 channels: 160 / 181 / 206 / 300 us with segments of 128 / 256 / 512 /
  // 1024 tokens).
  if (p.varlen) {
    int64_t len = (int64_t)align_up((size_t)(p.T * cw / (4 * fill)), kTileMax);
    if (len < 128) len = 128;
    pl.seglen = (int)len;
    pl.nseg = 1;
    pl.max_units = p.T / len + p.N;
    pl.cut = p.T > len;
  } else {
    int64_t n = p.B * cw < 3 * sm_count() ? fill / (p.B * cw) : 1;
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
  a.bx = (int)((p.ld_x ? p.ld_x : p.D) * es);
  a.bd = (int)((p.ld_delta ? p.ld_delta : p.D) * es);
  a.bz = (int)((p.ld_z ? p.ld_z : p.D) * es);
  a.bb = (int)((p.ld_b ? p.ld_b : gs) * es);
  a.bc = (int)((p.ld_c ? p.ld_c : gs) * es);
  a.T = p.T, a.N = p.N;
  a.cbg = pl.cbg, a.nseg = pl.nseg, a.seglen = pl.seglen;
  a.softplus = p.softplus;
  a.vin = a.Dg % 2 == 0 && aligned_rows(x, a.bx, 2 * es) && aligned_rows(delta, a.bd, 2 * es) &&
          (!z || aligned_rows(z, a.bz, 2 * es));
  const int ve = 16 / (int)es < 4 * pl.RL ? 16 / (int)es : 4 * pl.RL;   // RowVec::VE
  a.vbc = ve * es == 16 && a.S == 4 * pl.RL && aligned_rows(B, a.bb, 16) && aligned_rows(C, a.bc, 16);
  RowsOf r = {64 / pl.RL * (int)es, 4 * pl.RL * (int)es, a.G > 1, a.Dg * (int64_t)es, a.S * (int64_t)es};
  r.x(x, a.bx), r.x(delta, a.bd), r.x(z, a.bz), r.s(B, a.bb), r.s(C, a.bc);
  a.rows = a.Dg % 2 == 0 ? r.rows : kRegs;
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
                        const int32_t* cu, void* y, float* ht, const int32_t* state_indices, int state_slots,
                        void* ws, cudaStream_t s) {
  const Plan pl = make_plan(p);
  const Layout l = layout_of(p, pl);
  Args a = base_args(p, pl, x, delta, A, B, C, Dp, z, dt_bias, h0, cu);
  char* w = static_cast<char*>(ws);
  a.y = y, a.ht = ht, a.slot = state_indices, a.slots = state_slots;
  const int es = p.dt == GDN_F32 ? 4 : 2;
  a.vy = a.Dg % 2 == 0 && aligned_rows(y, p.D * es, 2 * es);
  if (!a.vy) a.rows = kRegs;
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
  Plan pl = {};   // (no segments here)
  pl.RL = lanes_for(p.S);
  pl.nseg = 1;
  StepArgs sa;
  sa.a = base_args(p, pl, x, delta, A, B, C, Dp, z, dt_bias, nullptr, cu);
  sa.a.y = y;
  sa.state = state, sa.idx = state_indices, sa.slots = state_slots;
  sa.Ttot = (int64_t)p.B * p.T;
  // One token a sequence: by the sequence for a few (latency), two at a time for many.
  const bool token = !sa.a.cu && p.T == 1;
  by_lanes(pl.RL, [&](auto rl) {
    constexpr int R = decltype(rl)::value, Q = R > 1 ? 2 : 1, L = R / Q;
    auto go = [&](auto* t) {
      using T = std::remove_pointer_t<decltype(t)>;
      if (token && p.N >= 64) {
        scan_token_kernel<T, L, Q, 2><<<dim3((unsigned)ceil_div(p.N, 2), (unsigned)ceil_div(p.D, 256 / L)), 256, 0, s>>>(sa);
      } else if (token) {
        scan_token_kernel<T, R, 1, 1><<<dim3(p.N, (unsigned)ceil_div(p.D, 256 / R)), 256, 0, s>>>(sa);
      } else {
        scan_step_kernel<T, R><<<dim3(p.N, (unsigned)ceil_div(p.D, 256 / R)), 256, 0, s>>>(sa);
      }
    };
    if (p.dt == GDN_F32) go(static_cast<float*>(nullptr));
    else go(static_cast<__nv_bfloat16*>(nullptr));
  });
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace gdn
