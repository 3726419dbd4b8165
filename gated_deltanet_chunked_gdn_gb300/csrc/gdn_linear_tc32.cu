// gdn_linear_tc32.cu -- the chunks' own states and the outputs of decayed linear attention on the tensor cores with fp32
// precision throughout (the backward pass also has the states of bf16 inputs with a head dim of 256 from here).
//
//   states:   D[e][d] = V^T (w K)                                (w_j = e^{b_last - b_j}; the adjoint's: q, do)
//   outputs:  P = scale M (Q K^T),   o^T[e][i] = scale e^{b_i} (S0^T Q^T) + V^T P^T
//
// Lanes of the tensor memory are the value columns, so that a warp writes 32 neighbours of a row of S or o.
#include "gdn_linear_tc32.cuh"

namespace gdn {
namespace lin {
namespace {

constexpr int N = 256;   // threads

template <typename T, int KD, int VD>
struct StateMap32 {
  static constexpr uint32_t kK = KD * 128, kV = VD * 128;   // a term's tile
  static constexpr uint32_t V = 0, K = kTerms<T> * kV;
  static constexpr uint32_t Misc = K + 3 * kK, Hi = Misc, Lo = Misc + 256, Wt = Misc + 512;
  static constexpr uint32_t Bar = Misc + 768, Flags = Bar + 8, Bytes = Flags + 56 + 1024;
};

// One chunk of one value head a CTA, KD x VD of its state.  2 x 4096 tokens of 16 fp32 heads of 128: 66 us (3.6 TB/s of
// states and inputs); 37 packed sequences, 12 heads of 64 x 128: 28 (fp32 FMAs: 47).  Bound by the latency of one round
// of loading, splitting and products: two CTAs an SM, tensor pipe 14 to 18 %.
template <typename T, int KD, int VD>
__global__ void __launch_bounds__(N, 2)
    states_tc32_kernel(Side<T> first, Side<T> second, Shape d, const float* __restrict__ g, Pieces pc,
                       Two* __restrict__ total, int32_t* status) {
  using M = StateMap32<T, KD, VD>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int nv = d.V / VD, nb = d.K / KD * nv;
  const int ch = blockIdx.x / nb, blk = blockIdx.x - ch * nb, d0 = blk / nv * KD, e0 = blk % nv * VD;
  const int c = ch / d.Hv, h = ch % d.Hv, hq = h / (d.Hv / d.Hqk);
  const Piece p = piece_of(pc, c);
  if (!p.ok) return;
  const Side<T> m = blockIdx.y ? second : first;
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
  fetch<64, KD, N>(xs, m.x + p.tok0 * m.ldx + (int64_t)hq * d.K + d0, m.ldx, p.len);
  fetch<64, VD, N>(ys, m.y + p.tok0 * m.ldy + (int64_t)h * d.V + e0, m.ldy, p.len);
  if (warp == 1) {
    chunk_sums(g + (d.g_per_head ? h : p.tok0 * d.Hv + h), d.g_per_head ? 0 : d.Hv, p.len, lane, hi, lo);
    __syncwarp();
#pragma unroll
    for (int r = lane; r < kC; r += 32)
      w[r] = m.adj ? m.factor * expf(hi[r] + lo[r]) : expf((hi[kC - 1] - hi[r]) + (lo[kC - 1] - lo[r]));
    if (lane == 0 && blk == 0 && blockIdx.y == 0) total[ch] = exp_two({hi[kC - 1], lo[kC - 1]});
  }
  place<64, VD, kTerms<T>, N>(sm + M::V, ys, nullptr);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(flags);
  place<64, KD, 3, N>(sm + M::K, xs, w);
  fence_proxy_async();
  __syncthreads();
  if (tid == 0) {
    const uint32_t id = idesc_bf16(128, KD, 1, 1, 0);
    products<kTerms<T>, 3>([&](int a, int b, uint32_t more) {
#pragma unroll
      for (int s = 0; s < 4; ++s)
        mma_bf16(tmem, dsw(s4, M::V + a * M::kV + s * 2048, 8192), dsw(s4, M::K + b * M::kK + s * 2048, 8192), id,
                 s > 0 ? 1u : more);
    });
    mma_commit(bar);
  }
  __syncwarp();
  const bool good = warp_wait(bar, 0, status);
  tc_fence_after();
  const int qd = warp & 3, part = warp >> 2, row = 32 * qd + lane;
  if (good && row < VD) {
    float* to = m.S + ((int64_t)ch * d.K + d0 + part * (KD / 2)) * d.V + e0 + row;
#pragma unroll
    for (int b = 0; b < KD / 2; b += 16) {
      float v[16];
      tmem_ld16(tmem + (static_cast<uint32_t>(32 * qd) << 16) + part * (KD / 2) + b, v);
#pragma unroll
      for (int j = 0; j < 16; ++j) to[(int64_t)(b + j) * d.V] = v[j];
    }
  }
  tc_fence_before();
  if (__syncthreads_or(!good) && tid == 0) mbar_wait(bar, 0, status, 100000000ull);
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, KD);
}

template <int VD>
struct OutMap32 {
  static constexpr uint32_t kQ = 8192, kS = 64 * VD * 2, kV = kS, kP = 8192;   // a term's tile
  static constexpr uint32_t S = 0, V = S;                     // V where S0 was
  static constexpr uint32_t Q = S + 3 * kS;
  static constexpr uint32_t K = Q + 3 * kQ, P = K;             // P where K was
  static constexpr uint32_t Misc = K + 3 * kP, Hi = Misc, Lo = Misc + 256, Up = Misc + 512;
  static constexpr uint32_t Bar = Misc + 768, Flags = Bar + 16, Bytes = Flags + 48 + 1024;
};

// VD of the V = NV VD columns of the outputs of one chunk of one value head a CTA, 64 of the summed K at a time (KB of
// them).  With
// more than one 64 of K, the products of first terms and all others have a sum each.  2 x 4096 tokens of 16 heads of
// 128: 131 us (2.6 TB/s); 37 packed sequences, 12 heads of 64 x 128: 60 (fp32 FMAs: 131).  Bound by the latency of its
// three rounds at two CTAs an SM: tensor pipe 19 %, HBM 21 %.
template <int VD, int NV, int KB>
__global__ void __launch_bounds__(N, 2)
    outputs_tc32_kernel(const float* __restrict__ q, const float* __restrict__ k, const float* __restrict__ v, Shape d,
                        const float* __restrict__ g, Pieces pc, float scale, const float* __restrict__ S0,
                        float* __restrict__ o, int32_t* status) {
  using M = OutMap32<VD>;
  constexpr uint32_t kCols = KB > 1 ? 256 : 128, kRest = KB > 1 ? 128 : 0;   // TMEM columns, place of the others' sums
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  constexpr int K = 64 * KB, V = NV * VD;
  const int ch = blockIdx.x / NV, e0 = (blockIdx.x - ch * NV) * VD;
  const int c = ch / d.Hv, h = ch % d.Hv, hq = h / (d.Hv / d.Hqk);
  const Piece p = piece_of(pc, c);
  if (!p.ok) return;
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t s4 = (smem_u32(sm) & 0x3FFFFu) >> 4;
  float *hi = reinterpret_cast<float*>(sm + M::Hi), *lo = reinterpret_cast<float*>(sm + M::Lo);
  float* up = reinterpret_cast<float*>(sm + M::Up);
  // Q K^T and, with the last of them, V^T P^T; S0^T Q^T: a phase for every 64 of K
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + M::Bar);
  uint32_t* flags = reinterpret_cast<uint32_t*>(sm + M::Flags);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int qd = warp & 3, part = warp >> 2, row = 32 * qd + lane;
  const uint32_t lane_off = static_cast<uint32_t>(32 * qd) << 16;

  if (tid == 0) {
    mbar_init(bars, 1);
    mbar_init(bars + 1, 1);
    mbar_fence_init();
  }
  if (warp == 0) tmem_alloc(flags, kCols);
  const float* qp = q + p.tok0 * d.ldq + (int64_t)hq * K;
  const float* kp = k + p.tok0 * d.ldk + (int64_t)hq * K;
  const float* sp = S0 + (int64_t)ch * K * V + e0;
  constexpr int last = KB - 1;
  float4 xv[64 * VD / 4 / N];   // S0's rows, then V's
  bool good = true;
  uint32_t tmem = 0;
  int issued0 = 0, issued1 = 0;   // phases begun
#pragma unroll 1
  for (int kb = 0; kb < KB; ++kb) {
    float4 xq[4], xk[4];
    fetch<64, 64, N>(xq, qp + 64 * kb, d.ldq, p.len);
    fetch<64, 64, N>(xk, kp + 64 * kb, d.ldk, p.len);
    fetch<64, VD, N>(xv, sp + (int64_t)64 * kb * V, V, 64);
    if (kb == 0) {
      if (warp == 1) {
        chunk_sums(g + (d.g_per_head ? h : p.tok0 * d.Hv + h), d.g_per_head ? 0 : d.Hv, p.len, lane, hi, lo);
        __syncwarp();
#pragma unroll
        for (int r = lane; r < kC; r += 32) up[r] = scale * expf(hi[r] + lo[r]);
      }
    } else {   // the tiles before have been read
      good = good && warp_wait(bars, (kb - 1) & 1, status);
      good = good && warp_wait(bars + 1, (kb - 1) & 1, status);
    }
    if (good) {
      place<64, 64, 3, N>(sm + M::Q, xq, nullptr);
      place<64, 64, 3, N>(sm + M::K, xk, nullptr);
    }
    fence_proxy_async();
    tc_fence_before();
    if (__syncthreads_or(!good)) {
      good = false;
      break;
    }
    tc_fence_after();
    tmem = *reinterpret_cast<volatile uint32_t*>(flags);
    if (tid == 0) {
      const uint32_t id = idesc_bf16(128, 64, 0, 0, 0);
      products<3, 3>([&](int a, int b, uint32_t more) {
        const bool main = a + b == 0;
        const uint32_t to = tmem + (main ? 0 : kRest), first = main && KB > 1 ? 0u : more;
#pragma unroll
        for (int s = 0; s < 4; ++s)
          mma_bf16(to, dsw(s4, M::Q + a * M::kQ + s * 32, 16), dsw(s4, M::K + b * M::kQ + s * 32, 16), id,
                   s > 0 || kb > 0 ? 1u : first);
      });
      mma_commit(bars);
    }
    issued0 = kb + 1;
    __syncwarp();
    place<64, VD, 3, N>(sm + M::S, xv, nullptr);
    fence_proxy_async();
    __syncthreads();
    if (tid == 0) {
      const uint32_t id = idesc_bf16(128, 64, 1, 0, 0);
      products<3, 3>([&](int a, int b, uint32_t more) {
        const bool main = a + b == 0;
        const uint32_t to = tmem + 64 + (main ? 0 : kRest), first = main && KB > 1 ? 0u : more;
#pragma unroll
        for (int s = 0; s < 4; ++s)
          mma_bf16(to, dsw(s4, M::S + a * M::kS + s * 2048, 8192), dsw(s4, M::Q + b * M::kQ + s * 32, 16), id,
                   s > 0 || kb > 0 ? 1u : first);
      });
      mma_commit(bars + 1);
    }
    issued1 = kb + 1;
    __syncwarp();
  }
  if (good) {
    fetch<64, VD, N>(xv, v + p.tok0 * d.ldv + (int64_t)h * V + e0, d.ldv, p.len);
    good = warp_wait(bars, last & 1, status);
    tc_fence_after();
  }
  constexpr int COLS = 32;   // tokens of a thread
  if (row < 64 && good) {    // P[row][.]
#pragma unroll
    for (int b = 0; b < COLS; b += 16) {
      float x[16];
      const int j0 = part * COLS + b;
      tmem_ld16(tmem + lane_off + j0, x);
      if (KB > 1) {
        float rest[16];
        tmem_ld16(tmem + kRest + lane_off + j0, rest);
#pragma unroll
        for (int j = 0; j < 16; ++j) x[j] += rest[j];
      }
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
  good = good && warp_wait(bars + 1, last & 1, status);
  if (good) place<64, VD, 3, N>(sm + M::V, xv, nullptr);
  fence_proxy_async();
  tc_fence_before();
  const bool all = !__syncthreads_or(!good);
  tc_fence_after();
  if (all) {
    if (tid == 0) {
      const uint32_t id = idesc_bf16(128, 64, 1, 0, 0);
      products<3, 3>([&](int a, int b, uint32_t more) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
          mma_bf16(tmem, dsw(s4, M::V + a * M::kV + s * 2048, 8192), dsw(s4, M::P + b * M::kP + s * 32, 16), id,
                   s > 0 ? 1u : more);
      });
      mma_commit(bars);
    }
    issued0 = last + 2;
    __syncwarp();
    good = warp_wait(bars, (last + 1) & 1, status);
    tc_fence_after();
    if (good && row < VD) {
      float* to = o + ((p.tok0 + part * COLS) * d.Hv + h) * (int64_t)V + e0 + row;
#pragma unroll
      for (int b = 0; b < COLS; b += 16) {
        float x[16], y[16];
        tmem_ld16(tmem + lane_off + part * COLS + b, x);
        tmem_ld16(tmem + lane_off + 64 + part * COLS + b, y);
        if (KB > 1) {
          float rest[16];
          tmem_ld16(tmem + kRest + lane_off + 64 + part * COLS + b, rest);
#pragma unroll
          for (int j = 0; j < 16; ++j) y[j] += rest[j];
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int i = part * COLS + b + j;
          if (i < p.len) to[(int64_t)(b + j) * d.Hv * V] = fmaf(up[i], y[j], x[j]);
        }
      }
    }
  }
  tc_fence_before();
  if (__syncthreads_or(!good) && tid == 0) {   // products still under way end before their memory is given back
    if (issued0) mbar_wait(bars, (issued0 - 1) & 1, status, 100000000ull);
    if (issued1) mbar_wait(bars + 1, (issued1 - 1) & 1, status, 100000000ull);
  }
  __syncthreads();
  if (warp == 0) tmem_dealloc(*reinterpret_cast<volatile uint32_t*>(flags), kCols);
}

template <typename F>
bool allow(F kern, uint32_t bytes) {
  return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess;
}

template <typename T, int KD, int VD>
gdn_status states(const Shape& d, const Side<T>& first, const Side<T>& second, int sides, const float* g,
                  const Pieces& pc, int most, Two* total, int32_t* status, cudaStream_t s) {
  auto kern = states_tc32_kernel<T, KD, VD>;
  constexpr uint32_t bytes = StateMap32<T, KD, VD>::Bytes;
  if (!allow(kern, bytes)) return GDN_ERR_CUDA;
  const int64_t grid = (int64_t)most * d.Hv * (d.K / KD) * (d.V / VD);
  kern<<<dim3((unsigned)grid, sides), N, bytes, s>>>(first, second, d, g, pc, total, status);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

template <int VD, int NV, int KB>
gdn_status outputs(const Shape& d, const float* q, const float* k, const float* v, const float* g, const Pieces& pc,
                   int most, float scale, const float* S0, float* o, int32_t* status, cudaStream_t s) {
  auto kern = outputs_tc32_kernel<VD, NV, KB>;
  constexpr uint32_t bytes = OutMap32<VD>::Bytes;
  if (!allow(kern, bytes)) return GDN_ERR_CUDA;
  const int64_t grid = (int64_t)most * d.Hv * NV;
  kern<<<(unsigned)grid, N, bytes, s>>>(q, k, v, d, g, pc, scale, S0, o, status);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

template <typename T>
gdn_status launch_states(const Shape& d, const Side<T>& first, const Side<T>& second, int sides, const float* g,
                         const Pieces& pc, int most, Two* total, int32_t* status, cudaStream_t s) {
  if (most == 0) return GDN_OK;
#define GDN_STATES(K, V) return states<T, K, V>(d, first, second, sides, g, pc, most, total, status, s)
  if (d.K == 64 && d.V != 64) GDN_STATES(64, 128);
  if (d.K != 64 && d.V == 64) GDN_STATES(128, 64);
  if constexpr (sizeof(T) == 4) {   // bf16 comes here with a head dim of 256 alone
    if (d.K == 64) GDN_STATES(64, 64);
  }
  GDN_STATES(128, 128);
#undef GDN_STATES
}

gdn_status launch_outputs(const Shape& d, const float* q, const float* k, const float* v, const float* g,
                          const Pieces& pc, int most, float scale, const float* S0, float* o, int32_t* status,
                          cudaStream_t s) {
  if (most == 0) return GDN_OK;
#define GDN_OUTPUTS(KB)                                                                        \
  (d.V == 64 ? outputs<64, 1, KB> : d.V == 128 ? outputs<128, 1, KB> : outputs<128, 2, KB>)(   \
      d, q, k, v, g, pc, most, scale, S0, o, status, s)
  if (d.K == 64) return GDN_OUTPUTS(1);
  return d.K == 128 ? GDN_OUTPUTS(2) : GDN_OUTPUTS(4);
#undef GDN_OUTPUTS
}

template gdn_status launch_states<float>(const Shape&, const Side<float>&, const Side<float>&, int, const float*,
                                         const Pieces&, int, Two*, int32_t*, cudaStream_t);
template gdn_status launch_states<__nv_bfloat16>(const Shape&, const Side<__nv_bfloat16>&, const Side<__nv_bfloat16>&,
                                                 int, const float*, const Pieces&, int, Two*, int32_t*, cudaStream_t);

}  // namespace lin
}  // namespace gdn
