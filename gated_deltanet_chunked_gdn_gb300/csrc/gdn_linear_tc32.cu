// gdn_linear_tc32.cu -- the chunks' own states and the outputs of decayed linear attention for fp32 and K, V in
// {64, 128} on the tensor cores.
//
// An fp32 value is the sum of three bf16 values to its last bit or so (8 bits each); a product of two such sums keeps
// the six of its nine terms that reach 2^-24 of it, each exact in the fp32 accumulators.  Six bf16 products cost a
// sixth of 1.89 PFLOP/s, against 74 TFLOP/s of fp32 FMAs.
//
//   states:   D[e][d] = V^T (w K)                                (w_j = e^{b_last - b_j}; the adjoint's: q, do)
//   outputs:  P = scale M (Q K^T),   o^T[e][i] = scale e^{b_i} (S0^T Q^T) + V^T P^T
//
// Lanes of the tensor memory are the value columns, so that a warp writes 32 neighbours of a row of S or o.  Tiles of
// 64 rows or columns are read as 128 where they stand in A; the lanes behind them are ignored.
#include "gdn_linear_tc.cuh"

namespace gdn {
namespace lin {
namespace {

// Threads of a CTA: four quads of a 64-row tile each, whatever K.
template <int KD>
constexpr int kThreads32 = KD == 64 ? 256 : 512;

// Rows of `cols` fp32 -> three tiles `tile` bytes apart of 64-column atom columns, row r times w[r]; zeros past `rows`.
template <int ROWS, int COLS, int N>
__device__ __forceinline__ void fetch(float4 (&x)[ROWS * COLS / 4 / N], const float* src, int64_t ld, int rows) {
#pragma unroll
  for (int u = 0; u < ROWS * COLS / 4 / N; ++u) {
    const int quad = threadIdx.x + u * N, r = quad / (COLS / 4), c = quad % (COLS / 4) * 4;
    x[u] = r < rows ? *reinterpret_cast<const float4*>(src + r * ld + c) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
}
template <int ROWS, int COLS, int N>
__device__ __forceinline__ void place(uint8_t* sm, const float4 (&x)[ROWS * COLS / 4 / N], const float* w) {
  constexpr uint32_t tile = ROWS * COLS * 2;
#pragma unroll
  for (int u = 0; u < ROWS * COLS / 4 / N; ++u) {
    const int quad = threadIdx.x + u * N, r = quad / (COLS / 4), c = quad % (COLS / 4) * 4;
    float4 y = x[u];
    if (w) {
      const float f = w[r];
      y.x *= f, y.y *= f, y.z *= f, y.w *= f;
    }
    uint32_t w0[2], w1[2], w2[2];
    split3(y, w0, w1, w2);
    uint8_t* to = sm + (c >> 6) * (ROWS * 128) + sw128_chunk(r, (c & 63) >> 3) + (c & 4) * 2;
    *reinterpret_cast<uint2*>(to) = make_uint2(w0[0], w0[1]);
    *reinterpret_cast<uint2*>(to + tile) = make_uint2(w1[0], w1[1]);
    *reinterpret_cast<uint2*>(to + 2 * tile) = make_uint2(w2[0], w2[1]);
  }
}

// The six products of terms, the smallest first: f(term of A, term of B, first)
template <typename F>
__device__ __forceinline__ void six(F f) {
  f(2, 0, 0u), f(1, 1, 1u), f(0, 2, 1u), f(1, 0, 1u), f(0, 1, 1u), f(0, 0, 1u);
}

template <int KD, int VD>
struct StateMap32 {
  static constexpr uint32_t kK = KD * 128, kV = VD * 128;   // a term's tile
  static constexpr uint32_t V = 0, K = 3 * kV;
  static constexpr uint32_t Misc = K + 3 * kK, Hi = Misc, Lo = Misc + 256, Wt = Misc + 512;
  static constexpr uint32_t Bar = Misc + 768, Flags = Bar + 8, Bytes = Flags + 56 + 1024;
};

template <int KD, int VD, bool ADJ>
__global__ void __launch_bounds__(kThreads32<KD>, KD == 64 ? 2 : 1)
    states_tc32_kernel(const float* __restrict__ x, int64_t ldx, const float* __restrict__ y, int64_t ldy, Shape d,
                       const float* __restrict__ g, Pieces pc, float factor, float* __restrict__ S,
                       float* __restrict__ total, int32_t* status) {
  using M = StateMap32<KD, VD>;
  constexpr int N = kThreads32<KD>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int c = blockIdx.x / d.Hv, h = blockIdx.x % d.Hv, hq = h / (d.Hv / d.Hqk);
  const Piece p = piece_of(pc, c);
  if (!p.ok) return;
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t s4 = (smem_u32(sm) & 0x3FFFFu) >> 4;
  float *hi = reinterpret_cast<float*>(sm + M::Hi), *lo = reinterpret_cast<float*>(sm + M::Lo);
  float* w = reinterpret_cast<float*>(sm + M::Wt);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + M::Bar);
  uint32_t* flags = reinterpret_cast<uint32_t*>(sm + M::Flags);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    mbar_init(bar, 1);
    mbar_fence_init();
  }
  if (warp == 0) tmem_alloc(flags, KD);
  float4 xs[64 * KD / 4 / N], ys[64 * VD / 4 / N];
  fetch<64, KD, N>(xs, x + p.tok0 * ldx + (int64_t)hq * KD, ldx, p.len);
  fetch<64, VD, N>(ys, y + p.tok0 * ldy + (int64_t)h * VD, ldy, p.len);
  if (warp == 1) {
    chunk_sums(g + (d.g_per_head ? h : p.tok0 * d.Hv + h), d.g_per_head ? 0 : d.Hv, p.len, lane, hi, lo);
    __syncwarp();
#pragma unroll
    for (int r = lane; r < kC; r += 32)
      w[r] = ADJ ? factor * expf(hi[r] + lo[r]) : expf((hi[kC - 1] - hi[r]) + (lo[kC - 1] - lo[r]));
    if (lane == 0) total[blockIdx.x] = expf(hi[kC - 1] + lo[kC - 1]);
  }
  place<64, VD, N>(sm + M::V, ys, nullptr);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(flags);
  place<64, KD, N>(sm + M::K, xs, w);
  fence_proxy_async();
  __syncthreads();
  if (tid == 0) {
    const uint32_t id = idesc_bf16(128, KD, 1, 1, 0);
    six([&](int a, int b, uint32_t first) {
#pragma unroll
      for (int s = 0; s < 4; ++s)
        mma_bf16(tmem, dsw(s4, M::V + a * M::kV + s * 2048, 8192), dsw(s4, M::K + b * M::kK + s * 2048, 8192), id,
                 s > 0 ? 1u : first);
    });
    mma_commit(bar);
  }
  __syncwarp();
  const bool good = mbar_wait(bar, 0, status);
  tc_fence_after();
  const int qd = warp & 3, part = warp >> 2, row = 32 * qd + lane;
  if (good && row < VD) {
    constexpr int COLS = KD / (N / 128);
    float* to = S + ((int64_t)blockIdx.x * KD + part * COLS) * VD + row;
#pragma unroll
    for (int b = 0; b < COLS; b += 16) {
      float v[16];
      tmem_ld16(tmem + (static_cast<uint32_t>(32 * qd) << 16) + part * COLS + b, v);
#pragma unroll
      for (int j = 0; j < 16; ++j) to[(b + j) * VD] = v[j];
    }
  }
  tc_fence_before();
  if (__syncthreads_or(!good) && tid == 0) mbar_wait(bar, 0, status, 100000000ull);
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, KD);
}

template <int KD, int VD>
struct OutMap32 {
  static constexpr uint32_t kQ = KD * 128, kS = KD * VD * 2, kV = VD * 128, kP = 8192;
  static constexpr uint32_t S = 0, V = S;            // V where S0 was
  static constexpr uint32_t Q = S + 3 * kS;
  static constexpr uint32_t K = Q + 3 * kQ, P = K;   // P where K was
  static constexpr uint32_t Misc = K + 3 * kQ, Hi = Misc, Lo = Misc + 256, Up = Misc + 512;
  static constexpr uint32_t Bar = Misc + 768, Flags = Bar + 24, Bytes = Flags + 40 + 1024;
};

// One chunk of one value head a CTA.
template <int KD, int VD>
__global__ void __launch_bounds__(kThreads32<KD>, KD == 64 ? 2 : 1)
    outputs_tc32_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v, Shape d,
                        const float* __restrict__ g, Pieces pc, float scale, const float* __restrict__ S0,
                        float* __restrict__ o, int32_t* status) {
  using M = OutMap32<KD, VD>;
  constexpr int N = kThreads32<KD>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int c = blockIdx.x / d.Hv, h = blockIdx.x % d.Hv, hq = h / (d.Hv / d.Hqk);
  const Piece p = piece_of(pc, c);
  if (!p.ok) return;
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t s4 = (smem_u32(sm) & 0x3FFFFu) >> 4;
  float *hi = reinterpret_cast<float*>(sm + M::Hi), *lo = reinterpret_cast<float*>(sm + M::Lo);
  float* up = reinterpret_cast<float*>(sm + M::Up);
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + M::Bar);   // Q K^T, S0^T Q^T, V^T P^T: one phase each
  uint32_t* flags = reinterpret_cast<uint32_t*>(sm + M::Flags);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int qd = warp & 3, part = warp >> 2, row = 32 * qd + lane;
  constexpr int COLS = 64 / (N / 128);   // tokens of a thread
  const uint32_t lane_off = static_cast<uint32_t>(32 * qd) << 16;

  if (tid == 0) {
#pragma unroll
    for (int i = 0; i < 3; ++i) mbar_init(bars + i, 1);
    mbar_fence_init();
  }
  if (warp == 0) tmem_alloc(flags, 128);
  {
    float4 xq[64 * KD / 4 / N], xk[64 * KD / 4 / N], xs[KD * VD / 4 / N];
    fetch<64, KD, N>(xq, q + p.tok0 * d.ldq + (int64_t)hq * KD, d.ldq, p.len);
    fetch<64, KD, N>(xk, k + p.tok0 * d.ldk + (int64_t)hq * KD, d.ldk, p.len);
    fetch<KD, VD, N>(xs, S0 + (int64_t)blockIdx.x * KD * VD, VD, KD);
    if (warp == 1) {
      chunk_sums(g + (d.g_per_head ? h : p.tok0 * d.Hv + h), d.g_per_head ? 0 : d.Hv, p.len, lane, hi, lo);
      __syncwarp();
#pragma unroll
      for (int r = lane; r < kC; r += 32) up[r] = scale * expf(hi[r] + lo[r]);
    }
    place<64, KD, N>(sm + M::Q, xq, nullptr);
    place<64, KD, N>(sm + M::K, xk, nullptr);
    fence_proxy_async();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0) {
      const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(flags), id = idesc_bf16(128, 64, 0, 0, 0);
      six([&](int a, int b, uint32_t first) {
#pragma unroll
        for (int s = 0; s < KD / 16; ++s) {
          const uint32_t at = (s >> 2) * 8192 + (s & 3) * 32;
          mma_bf16(tmem, dsw(s4, M::Q + a * M::kQ + at, 16), dsw(s4, M::K + b * M::kQ + at, 16), id,
                   s > 0 ? 1u : first);
        }
      });
      mma_commit(bars);
    }
    __syncwarp();
    place<KD, VD, N>(sm + M::S, xs, nullptr);
  }
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(flags);
  fence_proxy_async();
  __syncthreads();
  if (tid == 0) {
    const uint32_t id = idesc_bf16(128, 64, 1, 0, 0);
    six([&](int a, int b, uint32_t first) {
#pragma unroll
      for (int s = 0; s < KD / 16; ++s)
        mma_bf16(tmem + 64, dsw(s4, M::S + a * M::kS + s * 2048, KD * 128),
                 dsw(s4, M::Q + b * M::kQ + (s >> 2) * 8192 + (s & 3) * 32, 16), id, s > 0 ? 1u : first);
    });
    mma_commit(bars + 1);
  }
  __syncwarp();
  float4 xv[64 * VD / 4 / N];
  fetch<64, VD, N>(xv, v + p.tok0 * d.ldv + (int64_t)h * VD, d.ldv, p.len);
  bool good = mbar_wait(bars, 0, status);
  tc_fence_after();
  if (row < 64 && good) {   // P[row][.] of COLS tokens
#pragma unroll
    for (int b = 0; b < COLS; b += 16) {
      float x[16];
      const int j0 = part * COLS + b;
      tmem_ld16(tmem + lane_off + j0, x);
      const float mine = hi[row], rest = lo[row];
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float e = expf((mine - hi[j0 + j]) + (rest - lo[j0 + j]));
        x[j] = j0 + j <= row ? scale * e * x[j] : 0.f;
      }
#pragma unroll
      for (int j = 0; j < 16; j += 8) {
        uint32_t a0[2], a1[2], a2[2], b0[2], b1[2], b2[2];
        split3(make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]), a0, a1, a2);
        split3(make_float4(x[j + 4], x[j + 5], x[j + 6], x[j + 7]), b0, b1, b2);
        uint8_t* to = sm + M::P + sw128_chunk(row, (j0 + j) >> 3);
        *reinterpret_cast<uint4*>(to) = make_uint4(a0[0], a0[1], b0[0], b0[1]);
        *reinterpret_cast<uint4*>(to + M::kP) = make_uint4(a1[0], a1[1], b1[0], b1[1]);
        *reinterpret_cast<uint4*>(to + 2 * M::kP) = make_uint4(a2[0], a2[1], b2[0], b2[1]);
      }
    }
  }
  good = good && mbar_wait(bars + 1, 0, status);
  if (good) place<64, VD, N>(sm + M::V, xv, nullptr);
  fence_proxy_async();
  tc_fence_before();
  const bool all = !__syncthreads_or(!good);
  tc_fence_after();
  if (all) {
    if (tid == 0) {
      const uint32_t id = idesc_bf16(128, 64, 1, 0, 0);
      six([&](int a, int b, uint32_t first) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
          mma_bf16(tmem, dsw(s4, M::V + a * M::kV + s * 2048, 8192), dsw(s4, M::P + b * M::kP + s * 32, 16), id,
                   s > 0 ? 1u : first);
      });
      mma_commit(bars + 2);
    }
    __syncwarp();
    good = mbar_wait(bars + 2, 0, status);
    tc_fence_after();
    if (good && row < VD) {
      float* to = o + ((p.tok0 + part * COLS) * d.Hv + h) * (int64_t)VD + row;
#pragma unroll
      for (int b = 0; b < COLS; b += 16) {
        float x[16], y[16];
        tmem_ld16(tmem + lane_off + part * COLS + b, x);
        tmem_ld16(tmem + lane_off + 64 + part * COLS + b, y);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int i = part * COLS + b + j;
          if (i < p.len) to[(int64_t)(b + j) * d.Hv * VD] = fmaf(up[i], y[j], x[j]);
        }
      }
    }
  }
  tc_fence_before();
  if (__syncthreads_or(!good) && tid == 0) {   // products still under way end before their memory is given back
    for (int b = 0; b < (all ? 3 : 2); ++b) mbar_wait(bars + b, 0, status, 100000000ull);
  }
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 128);
}

template <typename F>
bool allow(F kern, uint32_t bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess;
}

template <int KD, int VD, bool ADJ>
gdn_status states(const Shape& d, const float* x, int64_t ldx, const float* y, int64_t ldy, const float* g,
                  const Pieces& pc, int most, float factor, float* S, float* total, int32_t* status, cudaStream_t s) {
  auto kern = states_tc32_kernel<KD, VD, ADJ>;
  constexpr uint32_t bytes = StateMap32<KD, VD>::Bytes;
  if (!allow(kern, bytes)) return GDN_ERR_CUDA;
  kern<<<(unsigned)((int64_t)most * d.Hv), kThreads32<KD>, bytes, s>>>(x, ldx, y, ldy, d, g, pc, factor, S, total,
                                                                       status);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

template <int KD, int VD>
gdn_status outputs(const Shape& d, const float* q, const float* k, const float* v, const float* g, const Pieces& pc,
                   int most, float scale, const float* S0, float* o, int32_t* status, cudaStream_t s) {
  auto kern = outputs_tc32_kernel<KD, VD>;
  constexpr uint32_t bytes = OutMap32<KD, VD>::Bytes;
  static_assert(bytes <= 232448, "shared memory of one SM");
  if (!allow(kern, bytes)) return GDN_ERR_CUDA;
  kern<<<(unsigned)((int64_t)most * d.Hv), kThreads32<KD>, bytes, s>>>(q, k, v, d, g, pc, scale, S0, o, status);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

#define GDN_HEADS(CALL)                          \
  if (d.K == 64 && d.V == 64) return CALL(64, 64); \
  if (d.K == 64) return CALL(64, 128);           \
  if (d.V == 64) return CALL(128, 64);           \
  return CALL(128, 128)

gdn_status launch_states32(bool adj, const Shape& d, const float* x, int64_t ldx, const float* y, int64_t ldy,
                           const float* g, const Pieces& pc, int most, float factor, float* S, float* total,
                           int32_t* status, cudaStream_t s) {
#define GDN_CALL(K, V)                                                                          \
  adj ? states<K, V, true>(d, x, ldx, y, ldy, g, pc, most, factor, S, total, status, s)         \
      : states<K, V, false>(d, x, ldx, y, ldy, g, pc, most, factor, S, total, status, s)
  GDN_HEADS(GDN_CALL);
#undef GDN_CALL
}

gdn_status launch_outputs32(const Shape& d, const float* q, const float* k, const float* v, const float* g,
                            const Pieces& pc, int most, float scale, const float* S0, float* o, int32_t* status,
                            cudaStream_t s) {
#define GDN_CALL(K, V) outputs<K, V>(d, q, k, v, g, pc, most, scale, S0, o, status, s)
  GDN_HEADS(GDN_CALL);
#undef GDN_CALL
}
#undef GDN_HEADS

}  // namespace lin
}  // namespace gdn
