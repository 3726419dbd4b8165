// gdn_linear.cu -- decayed linear attention: the forward pass's dispatch (bf16: the walk of gdn_linear_tc.cu; fp32:
// three launches over 64-token chunks, the chunks' own states, the sums along each sequence, the outputs, with the
// kernels of gdn_linear_tc32.cu), the tables of packed batches, and the step on a state pool.
#include "gdn_linear_sums.cuh"

namespace gdn {
namespace lin {

// ------------------------------------------------- pieces of packed batches
namespace {

// One CTA: first piece of every sequence (a running sum over tiles of 1024 sequences), then every piece by a search
// for its sequence.
__global__ void __launch_bounds__(1024) pieces_kernel(const int32_t* __restrict__ cu, int N, int T, int size, int most,
                                                      int32_t* __restrict__ seq, int32_t* __restrict__ tok0,
                                                      int32_t* __restrict__ len, int32_t* __restrict__ first,
                                                      int32_t* __restrict__ nc, int32_t* __restrict__ status,
                                                      bool begin) {
  __shared__ int warp_sum[32];
  __shared__ int carry, bad;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (tid == 0) carry = 0, bad = cu[0] != 0 || cu[N] != T;
  __syncthreads();
  for (int base = 0; base < N; base += 1024) {
    const int n = base + tid;
    int64_t L = 0;
    if (n < N) {
      const int64_t a = cu[n], b = cu[n + 1];
      L = b - a;
      if (L < 0 || a < 0 || b > T) bad = 1, L = 0;
    }
    const int mine = (int)((L + size - 1) / size);
    int s = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += t;
    }
    if (lane == 31) warp_sum[warp] = s;
    __syncthreads();
    if (warp == 0) {
      int w = warp_sum[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += t;
      }
      warp_sum[lane] = w;
    }
    __syncthreads();
    const int before = carry + (warp ? warp_sum[warp - 1] : 0) + s - mine;
    if (n < N) first[n] = before;
    __syncthreads();
    if (tid == 1023) carry = before + mine;
    __syncthreads();
  }
  const int total = carry;
  if (tid == 0) {
    if (total > most) bad = 1;
    first[N] = total;
    *nc = bad ? -1 : total;
    if (bad || begin) *status = bad ? GDN_DEV_BAD_CU_SEQLENS : 0;
  }
  __syncthreads();
  if (bad) return;
  for (int c = tid; c < total; c += 1024) {
    int lo = 0, hi = N - 1;   // the last sequence with first <= c and pieces of its own
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= c) lo = mid;
      else hi = mid - 1;
    }
    const int at = (c - first[lo]) * size, L = cu[lo + 1] - cu[lo];
    seq[c] = lo;
    tok0[c] = cu[lo] + at;
    len[c] = L - at < size ? L - at : size;
  }
}

}  // namespace

int pieces_max(const gdn_linear_problem& p, int size) {
  return (int)(p.varlen ? p.T / size + (int64_t)p.N : p.B * ceil_div(p.T, size));
}

size_t pieces_bytes(const gdn_linear_problem& p, int size) {
  return p.varlen ? align_up(sizeof(int32_t) * (3 * (size_t)pieces_max(p, size) + p.N + 2)) : 0;
}

Pieces pieces_at(const gdn_linear_problem& p, int size, void* tables) {
  Pieces t;
  memset(&t, 0, sizeof(t));
  t.T = p.T;
  t.size = size;
  t.per = (int)ceil_div(p.T, size);
  if (p.varlen) {
    const int most = pieces_max(p, size);
    int32_t* at = static_cast<int32_t*>(tables);
    t.seq = at;
    t.tok0 = at + most;
    t.len = at + 2 * (int64_t)most;
    t.first = at + 3 * (int64_t)most;
    t.nc = t.first + p.N + 1;
  }
  return t;
}

cudaError_t launch_pieces(const gdn_linear_problem& p, int size, const int32_t* cu, void* tables, int32_t* status,
                          bool begin, cudaStream_t s) {
  if (!p.varlen) return begin ? cudaMemsetAsync(status, 0, sizeof(int32_t), s) : cudaSuccess;
  const Pieces t = pieces_at(p, size, tables);
  pieces_kernel<<<1, 1024, 0, s>>>(cu, p.N, p.T, size, pieces_max(p, size), const_cast<int32_t*>(t.seq),
                                   const_cast<int32_t*>(t.tok0), const_cast<int32_t*>(t.len),
                                   const_cast<int32_t*>(t.first), const_cast<int32_t*>(t.nc), status, begin);
  return cudaGetLastError();
}

// ------------------------------------------------------ sums along sequences
namespace {

// Along every sequence, in place: S_c (what chunk c adds) becomes the state before chunk c (rev: the adjoint of the
// state behind it); four elements of a state a thread.  2 x 4096 tokens of 16 heads of 128 (64 chunks a sequence):
// 48 us, 5.7 TB/s; with loads only after the sums before, 132.  Four CTAs an SM: with the 76 registers that the decays in
// two floats would take, three, 37 packed sequences of up to 24 chunks take 21 us instead of 17.  blockIdx.y: the first or the second of two sums.
__global__ void __launch_bounds__(256, 4) sums_kernel(Shape d, Pieces pc, const Two* __restrict__ total, Sum first,
                                                   Sum second) {
  const Sum m = blockIdx.y ? second : first;
  const float* __restrict__ init = m.init;
  float* __restrict__ S = m.S;
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
  Two a[2][AHEAD];
  auto chunk = [&](int i) { return m.rev ? c1 - 1 - i : c0 + i; };
  auto fetch = [&](float4 (&y)[AHEAD], Two (&f)[AHEAD], int base) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (base + i < c1 - c0) {
        y[i] = __ldcs(reinterpret_cast<const float4*>(S + ((int64_t)chunk(base + i) * d.Hv + h) * kv + at));
        f[i] = total[(int64_t)chunk(base + i) * d.Hv + h];
      }
  };
  auto add = [&](const float4 (&y)[AHEAD], const Two (&f)[AHEAD], int base) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
      if (base + i < c1 - c0) {
        *reinterpret_cast<float4*>(S + ((int64_t)chunk(base + i) * d.Hv + h) * kv + at) = run;
        const float h = f[i].h, l = f[i].l;
        run.x = fmaf(h, run.x, fmaf(l, run.x, y[i].x)), run.y = fmaf(h, run.y, fmaf(l, run.y, y[i].y));
        run.z = fmaf(h, run.z, fmaf(l, run.z, y[i].z)), run.w = fmaf(h, run.w, fmaf(l, run.w, y[i].w));
      }
  };
  fetch(x[0], a[0], 0);
  for (int base = 0; base < c1 - c0; base += 2 * AHEAD) {
    fetch(x[1], a[1], base + AHEAD);
    add(x[0], a[0], base);
    fetch(x[0], a[0], base + 2 * AHEAD);
    add(x[1], a[1], base + AHEAD);
  }
  if (m.fin) {
    int64_t row = n;
    if (m.idx) {
      row = m.idx[n];
      if (row < 0 || row >= m.slots) return;
    }
    *reinterpret_cast<float4*>(m.fin + (row * d.Hv + h) * kv + at) = run;
  }
}

}  // namespace

gdn_status launch_sums(const Shape& d, const Pieces& pc, int N, const Two* total, const Sum& first, const Sum& second,
                       int sides, cudaStream_t s) {
  const int64_t grid = (int64_t)N * d.Hv * ((int64_t)d.K * d.V / 1024);
  sums_kernel<<<dim3((unsigned)grid, sides), 256, 0, s>>>(d, pc, total, first, second);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

// -------------------------------------------------------------- the step
namespace {

// One CTA per (sequence, value head, COLS columns of V): the state's slice lives in registers for all of the
// sequence's tokens (COLS / 4 column groups of float4, the other threads' groups along K) and is read and written
// once.  Bound by the state's traffic, 8 K V bytes a head; streaming hints, since a pool larger than L2 is touched
// once a step.  512 sequences of 32 heads of 128 x 128: 314 us, 6.8 TB/s of their states (309 with the decay in one float);
// one sequence: 2.7 us.
template <typename T, int K, int COLS>
__global__ void __launch_bounds__(256) lin_step_kernel(const T* __restrict__ q, const T* __restrict__ k,
                                                       const T* __restrict__ v, int64_t ldq, int64_t ldk, int64_t ldv,
                                                       const float* __restrict__ g, int g_per_head, float scale,
                                                       float* __restrict__ state,
                                                       const int32_t* __restrict__ state_indices, int slots,
                                                       const int32_t* __restrict__ cu, int Tseq, int64_t Ttot, int Hqk,
                                                       int Hv, int V, T* __restrict__ o) {
  constexpr int CG = COLS / 4, RG = 256 / CG, RPG = K / RG;
  static_assert(RPG >= 1 && RPG * RG == K, "every thread holds rows");
  __shared__ float ks[K], qs[K];
  __shared__ __align__(16) float part[8][COLS];   // written as float4
  const int e0 = COLS * blockIdx.x, h = blockIdx.y % Hv;
  const int n = blockIdx.y / Hv;
  const int tid = threadIdx.x, cg = tid % CG, rg = tid / CG, lane = tid & 31, warp = tid >> 5;
  const int hq = h / (Hv / Hqk);
  const int64_t tok0 = cu ? cu[n] : (int64_t)n * Tseq;
  const int64_t L = cu ? (int64_t)cu[n + 1] - cu[n] : Tseq;
  if (L <= 0 || tok0 < 0 || tok0 + L > Ttot) return;   // malformed offsets: touch nothing
  const int slot = state_indices ? state_indices[n] : n;
  if (slot < 0 || slot >= slots) {
    for (int64_t t = 0; t < L; ++t)
      if (tid < COLS) o[((tok0 + t) * Hv + h) * (int64_t)V + e0 + tid] = from_f<T>(0.f);
    return;
  }
  float* S = state + (((int64_t)slot * Hv + h) * K) * (int64_t)V + e0 + 4 * cg;
  float gt = g[g_per_head ? h : tok0 * Hv + h];
  float s[RPG][4];
#pragma unroll
  for (int r = 0; r < RPG; ++r) {
    const float4 x = __ldcs(reinterpret_cast<const float4*>(S + (int64_t)(rg * RPG + r) * V));
    s[r][0] = x.x, s[r][1] = x.y, s[r][2] = x.z, s[r][3] = x.w;
  }
  for (int64_t t = 0; t < L; ++t) {
    const int64_t tok = tok0 + t;
    if (tid < K) {
      ks[tid] = to_f(k[tok * ldk + hq * K + tid]);
      qs[tid] = to_f(q[tok * ldq + hq * K + tid]);
    }
    const Two a = exp_two({gt, 0.f});
    if (t + 1 < L && !g_per_head) gt = g[(tok + 1) * Hv + h];
    const float4 v4 = load4(v + tok * ldv + (int64_t)h * V + e0 + 4 * cg);
    const float vv[4] = {v4.x, v4.y, v4.z, v4.w};
    __syncthreads();
    float p[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int r = 0; r < RPG; ++r) {
      const float kd = ks[rg * RPG + r], qd = qs[rg * RPG + r];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[r][j] = fmaf(a.h, s[r][j], fmaf(a.l, s[r][j], kd * vv[j]));
        p[j] = fmaf(qd, s[r][j], p[j]);
      }
    }
    // over the row groups of a warp by shuffles, over the warps through shared memory
#pragma unroll
    for (int off = CG; off < 32; off <<= 1)
#pragma unroll
      for (int j = 0; j < 4; ++j) p[j] += __shfl_xor_sync(0xffffffffu, p[j], off);
    if (lane < CG) *reinterpret_cast<float4*>(&part[warp][4 * cg]) = make_float4(p[0], p[1], p[2], p[3]);
    __syncthreads();
    if (tid < COLS) {
      float acc = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) acc += part[w][tid];
      o[(tok * Hv + h) * (int64_t)V + e0 + tid] = from_f<T>(scale * acc);
    }
    // part is written again only after the next token's first barrier, which the readers above pass after reading
  }
#pragma unroll
  for (int r = 0; r < RPG; ++r)
    __stcs(reinterpret_cast<float4*>(S + (int64_t)(rg * RPG + r) * V), make_float4(s[r][0], s[r][1], s[r][2], s[r][3]));
}

template <typename T, int COLS>
gdn_status launch_step(const gdn_linear_problem& p, const T* q, const T* k, const T* v, const float* g, float scale,
                       float* state, const int32_t* idx, int slots, const int32_t* cu, T* o, cudaStream_t s) {
  const int64_t y = (int64_t)p.N * p.Hv;
  if (y > 65535) {   // sequences in several launches: the grid's second dimension ends there
    const int per = 65535 / p.Hv;
    for (int n = 0; n < p.N; n += per) {
      gdn_linear_problem c = p;
      c.N = p.N - n < per ? p.N - n : per;
      const int64_t t = p.varlen ? 0 : (int64_t)n * p.T;
      const gdn_status st = launch_step<T, COLS>(c, q + t * p.ld_q, k + t * p.ld_k, v + t * p.ld_v,
                                                 p.g_per_head ? g : g + t * p.Hv, scale, idx ? state : state + (int64_t)n * p.Hv * p.K * p.V,
                                                 idx ? idx + n : nullptr, idx ? slots : slots - n, p.varlen ? cu + n : nullptr,
                                                 o + t * p.Hv * p.V, s);
      if (st != GDN_OK) return st;
    }
    return GDN_OK;
  }
  const dim3 grid(p.V / COLS, (unsigned)y);
  const int64_t Ttot = (int64_t)p.B * p.T;
#define GDN_STEP(K)                                                                                                   \
  lin_step_kernel<T, K, COLS><<<grid, 256, 0, s>>>(q, k, v, p.ld_q, p.ld_k, p.ld_v, g, p.g_per_head, scale, state,    \
                                                   idx, slots, p.varlen ? cu : nullptr, p.T, Ttot, p.Hqk, p.Hv, p.V, o)
  if (p.K == 64) GDN_STEP(64);
  else if (p.K == 128) GDN_STEP(128);
  else GDN_STEP(256);
#undef GDN_STEP
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

template <typename T>
gdn_status step_t(const gdn_linear_problem& p, const void* q, const void* k, const void* v, const float* g,
                  float scale, float* state, const int32_t* idx, int slots, const int32_t* cu, void* o,
                  cudaStream_t s) {
  // few heads: narrower slices, so that every SM has some (32 heads of 128, slices of 16 and of 64 columns: 1 sequence
  // 2.57 and 2.70 us, 4 sequences 4.87 and 3.61, before the decay took two floats, which adds 0.1 to each)
  if (2 * (int64_t)p.N * p.Hv * (p.V / 64) < sm_count())
    return launch_step<T, 16>(p, (const T*)q, (const T*)k, (const T*)v, g, scale, state, idx, slots, cu, (T*)o, s);
  return launch_step<T, 64>(p, (const T*)q, (const T*)k, (const T*)v, g, scale, state, idx, slots, cu, (T*)o, s);
}

}  // namespace
}  // namespace lin

gdn_status run_linear_step(const gdn_linear_problem& p, const void* q, const void* k, const void* v, const float* g,
                           float scale, float* state, const int32_t* idx, int slots, const int32_t* cu, void* o,
                           cudaStream_t s) {
  if ((int64_t)p.B * p.T == 0) return GDN_OK;
  if (p.dt == GDN_F32) return lin::step_t<float>(p, q, k, v, g, scale, state, idx, slots, cu, o, s);
  return lin::step_t<__nv_bfloat16>(p, q, k, v, g, scale, state, idx, slots, cu, o, s);
}

// ------------------------------------------------------------- forward, fp32
namespace lin {
namespace {

// [status][tables][total: chunks x Hv, in two floats][states: chunks x Hv x K x V]
size_t fwd32_bytes(const gdn_linear_problem& p) {
  const size_t cells = (size_t)pieces_max(p, kC) * p.Hv;
  return kAlign + pieces_bytes(p, kC) + align_up(sizeof(Two) * cells) + 4 * cells * p.K * p.V;
}

gdn_status fwd32(const gdn_linear_problem& p, const float* q, const float* k, const float* v, const float* g,
                 float scale, const float* h0, const int32_t* cu, float* o, float* ht, const int32_t* idx, int slots,
                 void* ws, cudaStream_t s) {
  uint8_t* at = static_cast<uint8_t*>(ws);
  int32_t* status = reinterpret_cast<int32_t*>(at);
  void* tables = at + kAlign;
  if (launch_pieces(p, kC, cu, tables, status, true, s) != cudaSuccess) return GDN_ERR_CUDA;
  const Pieces pc = pieces_at(p, kC, tables);
  const Shape d = shape_of(p);
  const int most = pieces_max(p, kC);
  Two* total = reinterpret_cast<Two*>(at + kAlign + pieces_bytes(p, kC));
  float* states = reinterpret_cast<float*>(total) + align_up(sizeof(Two) * (size_t)most * p.Hv) / 4;
  const Side<float> side{k, v, p.ld_k, p.ld_v, 1.f, states, false};
  gdn_status st = launch_states(d, side, side, 1, g, pc, most, total, status, s);
  if (st == GDN_OK) st = launch_sums(d, pc, p.N, total, Sum{h0, states, ht, idx, slots, false}, s);
  return st == GDN_OK ? launch_outputs(d, q, k, v, g, pc, most, scale, states, o, status, s) : st;
}

}  // namespace
}  // namespace lin

size_t linear_fwd_workspace_bytes(const gdn_linear_problem& p) {
  return p.dt == GDN_BF16 ? lin::tc_fwd_bytes(p) : lin::fwd32_bytes(p);
}

gdn_status run_linear_fwd(const gdn_linear_problem& p, const void* q, const void* k, const void* v, const float* g,
                          float scale, const float* h0, const int32_t* cu, void* o, float* ht, const int32_t* idx,
                          int slots, void* ws, cudaStream_t s) {
  if (p.dt == GDN_BF16) return lin::tc_fwd(p, q, k, v, g, scale, h0, cu, o, ht, idx, slots, ws, s);
  return lin::fwd32(p, (const float*)q, (const float*)k, (const float*)v, g, scale, h0, cu, (float*)o, ht, idx, slots,
                    ws, s);
}

}  // namespace gdn
