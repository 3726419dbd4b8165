// gdn_linear_tc_bwd.cu -- backward of decayed linear attention for bf16 and K, V in {64, 128} on the tensor cores (the
// formulas are gdn_linear_bwd.cu's).
//
// Two walks (gdn_linear_tc.cu) leave the state S0 before every chunk and the adjoint G of the state behind it in the
// workspace in fp32; then every chunk of every value head is on its own.  S0 and G enter the products in three bf16
// terms each, all of their 24 bits: dg, an fp32 output, is a sum over products with them (with two terms it was off by
// up to 1.2e-5 in sequences without decay).  Persistent CTAs, one an SM (the chunk's tiles, S0 and G fill its shared
// memory), take chunks in turn; the next chunk's S0 comes in while this one's gradients are formed, its tiles and G are
// prefetched to L2.  4 x 4096 tokens of 32 heads of 128: 610 us (3.3 TB/s of S0, G, the inputs and the gradients; HBM
// 36 %, tensor pipe 26 %; 570 with W and P in one term): a chunk takes 20k cycles and more, 5k of products, 5k of their
// operands' shared-memory reads, 2.5k of splitting S0 and G, and barriers between.  Tiles released earlier (561 against
// 570) or a warp that only issues (678, registers) did not help.
// TMEM lane = token: rows 0..63 of every stacked product are keys' rows, 64..127 queries'.
//
//   D1 = [K;Q] [K;Q]^T, D2 = [V;dO] [V;dO]^T   (lanes 0..63: columns 64..127 are K Q^T, V dO^T; lanes 64..127: columns
//                                              0..63 are Q K^T, dO V^T: both orientations in one product each)
//   I1 = [V;dO] S0^T, I2 = [V;dO] G^T          (S0, G in three terms)    lanes 64..127: dO S0^T;  lanes 0..63: V G^T
//   W = scale M (dO V^T), W^T, P^T             from D1, D2, in two bf16 terms (with one dq, dk and dv were off by up to
//                                              2.3e-3, with two by their own rounding, 1.7e-3); row and column sums of
//                                              A = W (Q K^T) in fp32
//   D1 <- [W^T;W] K, D2 <- [W^T;W] Q           lanes 64..127: W K;  lanes 0..63: W^T Q
//   dq_i = scale e^{b_i} I1 + D1,  dk_j = e^{b_last - b_j} I2 + D2
//   I1 <- dO^T P^T | G^T K^T                   lane = value column:  dv_j = I1a + e^{b_last - b_j} I1b
#include "gdn_linear_tc.cuh"

namespace gdn {
namespace lin {
namespace {

constexpr int kGradThreads = 512;

struct GradParams {
  const float* decays;   // [slots][Hv][kDecays]
  const float* states;   // [slots][Hv][K / 8][V][8]
  const float* adjoints;
  void* dq;              // bf16 [B, T, Hqk, K], or fp32 [B, T, Hv, K] (SHARED)
  void* dk;
  __nv_bfloat16* dv;
  float* dg;             // [B, T, Hv], or [chunks][Hv] sums
  int32_t* status;
  Pieces pc;
  int items;             // chunks x Hv (packed: at most)
  int Hqk, Hv, g_per_head;
  float scale;
};

template <int KD, int VD>
struct GradMap {
  static constexpr uint32_t KQ = 0;                              // k rows 0..63, q rows 64..127
  static constexpr uint32_t VO = KQ + KD / 64 * 16384;           // v rows 0..63, do rows 64..127
  static constexpr uint32_t S = VO + VD / 64 * 16384;            // S0 as it lies in memory, then S0^T's first two terms
  static constexpr uint32_t kTile = (uint32_t)KD * VD * 2;
  static constexpr uint32_t G = S + 2 * kTile;
  // the third terms of S0, then of G; then W^T rows 0..63, W rows 64..127 | P^T | sums, float[4][128] each.  (A 64-row
  // tile of G read as 128 rows, the upper half ignored, stays inside as well.)
  static constexpr uint32_t X3 = G + 2 * kTile;
  static constexpr uint32_t W = X3, P = W + 16384, SumA = P + 8192, SumX = SumA + 2048;
  // the second terms of W^T, W: where there is no room of their own, in the place of S0's front, which the next chunk's
  // then takes last; of P^T: in the place of W^T, once that has been read
  static constexpr bool kRoom = KD * VD < 128 * 128;
  static constexpr uint32_t W2 = kRoom ? X3 + 32768 : S, P2 = W;
  static constexpr uint32_t kFront = kRoom ? 0 : 16384;
  static constexpr uint32_t Misc = X3 + 32768 + (kRoom ? 16384 : 0);
  static constexpr uint32_t kGam = 4 * kDecays;
  static constexpr uint32_t Gam = Misc, Down = Misc + 256, Up = Misc + 512, Whole = Misc + 768, Low = Whole + 16;
  static constexpr uint32_t Red = Misc + kGam;   // float[16]
  static constexpr uint32_t Bar = Red + 64, Flags = Bar + 64;
  static constexpr uint32_t Bytes = Flags + 64 + 1024;
};

__device__ __forceinline__ void bulk_prefetch(const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}

template <int KD, int VD, bool SHARED>
__global__ void __launch_bounds__(kGradThreads, 1)
    grads_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                    const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_do,
                    const GradParams prm) {
  using M = GradMap<KD, VD>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t s4 = (smem_u32(sm) & 0x3FFFFu) >> 4;
  const float* gam = reinterpret_cast<const float*>(sm + M::Gam);
  const float* down = reinterpret_cast<const float*>(sm + M::Down);
  const float* up = reinterpret_cast<const float*>(sm + M::Up);
  const float* low = reinterpret_cast<const float*>(sm + M::Low);
  float* suma = reinterpret_cast<float*>(sm + M::SumA);
  float* sumx = reinterpret_cast<float*>(sm + M::SumX);
  float* red = reinterpret_cast<float*>(sm + M::Red);
  // every barrier completes one phase an item, and every thread waits for each of them once an item, in order
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + M::Bar);
  uint64_t *bar_t = bars, *bar_s = bars + 1, *bar_g = bars + 2, *bar_d = bars + 3, *bar_i = bars + 4, *bar_w = bars + 5,
           *bar_v = bars + 6, *bar_x = bars + 7;
  volatile uint32_t* flags = reinterpret_cast<volatile uint32_t*>(sm + M::Flags);   // [0] TMEM base
  volatile uint32_t* count = flags + 1;   // thread 0: phases begun on each barrier

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int qd = warp & 3, part = warp >> 2;   // TMEM lane quadrant, quarter of the columns
  const int row = 32 * qd + lane, tok = row & 63;
  const bool query = row >= 64;

  int total = prm.items;
  if (prm.pc.seq) {
    const int nc = *prm.pc.nc;
    total = nc < 0 ? 0 : nc * prm.Hv;
  }
  if ((int)blockIdx.x >= total) return;

  if (tid == 0) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      mbar_init(bars + i, 1);
      count[i] = 0;
    }
    mbar_fence_init();
    prefetch_tmap(&tm_q);
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    prefetch_tmap(&tm_do);
  }
  if (warp == 0) tmem_alloc(const_cast<uint32_t*>(flags), 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = flags[0];
  const uint32_t D1 = tmem, D2 = tmem + 128, I1 = tmem + 256, I2 = tmem + 384;
  const uint32_t lane_off = static_cast<uint32_t>(32 * qd) << 16;

  bool bad = false;
  auto wait = [&](uint64_t* bar, int n) {
    if (!bad) bad = !mbar_wait(bar, n & 1, prm.status);
  };
  auto commit = [&](int b, int n) {
    mma_commit(bars + b);
    count[b] = n + 1;
  };
  auto cell = [&](const Piece& p, int h) { return (chunk_slot(p) * prm.Hv + h); };
  auto issue_tiles = [&](int item, int n) {
    const int h = item % prm.Hv, hq = h / (prm.Hv / prm.Hqk);
    const Piece p = piece_of(prm.pc, item / prm.Hv);
    const int t = (int)p.tok0;
    count[0] = n + 1;
    mbar_arrive_expect_tx(bar_t, (KD + VD) / 64 * 16384 + M::kGam);
    bulk_load(sm + M::Gam, prm.decays + cell(p, h) * kDecays, M::kGam, bar_t);
#pragma unroll
    for (int a = 0; a < KD / 64; ++a) {
      tma_load_3d(sm + M::KQ + a * 16384, &tm_k, bar_t, 64 * a, hq, t);
      tma_load_3d(sm + M::KQ + a * 16384 + 8192, &tm_q, bar_t, 64 * a, hq, t);
    }
#pragma unroll
    for (int a = 0; a < VD / 64; ++a) {
      tma_load_3d(sm + M::VO + a * 16384, &tm_v, bar_t, 64 * a, h, t);
      tma_load_3d(sm + M::VO + a * 16384 + 8192, &tm_do, bar_t, 64 * a, h, t);
    }
  };
  auto issue_state = [&](int item, int n) {
    const Piece p = piece_of(prm.pc, item / prm.Hv);
    count[1] = n + 1;
    mbar_arrive_expect_tx(bar_s, 2 * M::kTile);
    bulk_load(sm + M::S + M::kFront, prm.states + cell(p, item % prm.Hv) * (KD * VD) + M::kFront / 4,
              2 * M::kTile - M::kFront, bar_s);
  };
  auto issue_front = [&](int item) {   // the rest of it
    if (M::kFront == 0) return;
    const Piece p = piece_of(prm.pc, item / prm.Hv);
    bulk_load(sm + M::S, prm.states + cell(p, item % prm.Hv) * (KD * VD), M::kFront, bar_s);
  };
  auto issue_adjoint = [&](int item, int n) {
    const Piece p = piece_of(prm.pc, item / prm.Hv);
    count[2] = n + 1;
    mbar_arrive_expect_tx(bar_g, 2 * M::kTile);
    bulk_load(sm + M::G, prm.adjoints + cell(p, item % prm.Hv) * (KD * VD), 2 * M::kTile, bar_g);
  };
  if (tid == 0) {
    issue_tiles(blockIdx.x, 0);
    issue_state(blockIdx.x, 0);
    issue_front(blockIdx.x);
    issue_adjoint(blockIdx.x, 0);
  }

  constexpr int NV = KD * VD / 4 / kGradThreads;   // quads of a state a thread holds
  auto tile_at = [&](int u) {   // place of this thread's quad u in a bf16 tile
    const int quad = tid + u * kGradThreads, e = (quad >> 1) % VD, d = (quad >> 1) / VD * 8 + (quad & 1) * 4;
    return (uint32_t)((d >> 6) * (VD * 128)) + sw128_chunk(e, (d & 63) >> 3) + (d & 4) * 2;
  };

  int n = 0;
#pragma unroll 1
  for (int item = blockIdx.x; item < total; item += gridDim.x, ++n) {
    const int h = item % prm.Hv, hq = h / (prm.Hv / prm.Hqk), c = item / prm.Hv;
    const Piece p = piece_of(prm.pc, c);
    const int len = p.len;
    const bool more = item + (int)gridDim.x < total;
    wait(bar_t, n);
    if (len < 64) {
      zero_rows(sm + M::KQ, KD / 64, 16384, len, tid, kGradThreads);
      zero_rows(sm + M::KQ + 8192, KD / 64, 16384, len, tid, kGradThreads);
      zero_rows(sm + M::VO, VD / 64, 16384, len, tid, kGradThreads);
      zero_rows(sm + M::VO + 8192, VD / 64, 16384, len, tid, kGradThreads);
      fence_proxy_async();
      if (__syncthreads_or(bad)) break;
    }
    if (warp == 8 && lane == 0 && more) {
      // the next chunk's tiles and its G, whose places stay taken until this one's end, on their way to L2
      const int next = item + gridDim.x, h1 = next % prm.Hv, hq1 = h1 / (prm.Hv / prm.Hqk);
      const Piece p1 = piece_of(prm.pc, next / prm.Hv);
      const int t = (int)p1.tok0;
      bulk_prefetch(prm.decays + cell(p1, h1) * kDecays, M::kGam);
#pragma unroll
      for (int a = 0; a < KD / 64; ++a) {
        tma_prefetch_3d(&tm_k, 64 * a, hq1, t);
        tma_prefetch_3d(&tm_q, 64 * a, hq1, t);
      }
#pragma unroll
      for (int a = 0; a < VD / 64; ++a) {
        tma_prefetch_3d(&tm_v, 64 * a, h1, t);
        tma_prefetch_3d(&tm_do, 64 * a, h1, t);
      }
      bulk_prefetch(prm.states + cell(p1, h1) * (KD * VD), 2 * M::kTile);
      bulk_prefetch(prm.adjoints + cell(p1, h1) * (KD * VD), 2 * M::kTile);
    }
    // ---- products that need the loads alone
    if (tid == 0 && !bad) {
      tc_fence_after();
      const uint32_t id = idesc_bf16(128, 128, 0, 0, 0);
#pragma unroll
      for (int s = 0; s < KD / 16; ++s) {
        const uint32_t a = M::KQ + (s >> 2) * 16384 + (s & 3) * 32;
        mma_bf16(D1, dsw(s4, a, 16), dsw(s4, a, 16), id, s > 0);
      }
#pragma unroll
      for (int s = 0; s < VD / 16; ++s) {
        const uint32_t a = M::VO + (s >> 2) * 16384 + (s & 3) * 32;
        mma_bf16(D2, dsw(s4, a, 16), dsw(s4, a, 16), id, s > 0);
      }
      commit(3, n);
    }
    __syncwarp();
    // ---- S0 and G: <G, S0>, and their terms in their own places (two lanes eight d of an e)
    wait(bar_s, n);
    wait(bar_g, n);
    uint32_t third[NV][2];   // of G
    {
      float4 s[NV], g[NV];
      float gs = 0.f;
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        s[u] = *reinterpret_cast<const float4*>(sm + M::S + 16 * (tid + u * kGradThreads));
        g[u] = *reinterpret_cast<const float4*>(sm + M::G + 16 * (tid + u * kGradThreads));
        gs = fmaf(s[u].x, g[u].x, fmaf(s[u].y, g[u].y, fmaf(s[u].z, g[u].z, fmaf(s[u].w, g[u].w, gs))));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) gs += __shfl_xor_sync(0xffffffffu, gs, o);
      if (lane == 0) red[warp] = gs;
      if (__syncthreads_or(bad)) break;
#pragma unroll
      for (int u = 0; u < NV; ++u) {
        const uint32_t off = tile_at(u);
        uint32_t w0[2], w1[2], w2[2];
        split3(s[u], w0, w1, w2);
        *reinterpret_cast<uint2*>(sm + M::S + off) = make_uint2(w0[0], w0[1]);
        *reinterpret_cast<uint2*>(sm + M::S + M::kTile + off) = make_uint2(w1[0], w1[1]);
        *reinterpret_cast<uint2*>(sm + M::X3 + off) = make_uint2(w2[0], w2[1]);
        split3(g[u], w0, w1, third[u]);
        *reinterpret_cast<uint2*>(sm + M::G + off) = make_uint2(w0[0], w0[1]);
        *reinterpret_cast<uint2*>(sm + M::G + M::kTile + off) = make_uint2(w1[0], w1[1]);
      }
    }
    fence_proxy_async();
    tc_fence_before();
    if (__syncthreads_or(bad)) break;
    tc_fence_after();
    // B = [e][d] tiles: the summed dimension e outermost
    const uint32_t idi = idesc_bf16(128, KD, 0, 1, 0);
    auto product = [&](uint32_t to, uint32_t tile, uint32_t first) {
#pragma unroll
      for (int e = 0; e < VD / 16; ++e)
        mma_bf16(to, dsw(s4, M::VO + (e >> 2) * 16384 + (e & 3) * 32, 16), dsw(s4, tile + e * 2048, VD * 128), idi,
                 e > 0 ? 1u : first);
    };
    if (tid == 0) {
      product(I1, M::X3, 0);
      commit(7, n);
      product(I1, M::S, 1);
      product(I1, M::S + M::kTile, 1);
      product(I2, M::G, 0);
      product(I2, M::G + M::kTile, 1);
    }
    __syncwarp();
    // ---- W, W^T, P^T and the sums of A
    wait(bar_d, n);
    tc_fence_after();
    uint32_t plow[2][4];   // P^T's second term
    {
      float qk[16], ov[16];
      const uint32_t at = (query ? 0 : 64) + 16 * part;
      tmem_ld16(D1 + lane_off + at, qk);
      tmem_ld16(D2 + lane_off + at, ov);
      const float mine = gam[tok], rest = low[tok];
      float w[16], pt[16], s = 0.f;
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        const int other = 16 * part + u;   // queries: column j of row i; keys: row i of column j
        const float d = (mine - gam[other]) + (rest - low[other]), e = query ? d : -d;
        const uint32_t keep = (query ? other <= tok : other >= tok) ? 0xffffffffu : 0u;
        const float m = prm.scale * ex2_fast(e);
        w[u] = __uint_as_float(__float_as_uint(m * ov[u]) & keep);
        pt[u] = __uint_as_float(__float_as_uint(m * qk[u]) & keep);
        const uint32_t off = other != tok ? 0xffffffffu : 0u;   // a token with itself has no decay between
        s += __uint_as_float(__float_as_uint(w[u] * qk[u]) & keep & off);
      }
      wait(bar_x, n);   // the third term of S0 has been read
#pragma unroll
      for (int u = 0; u < NV; ++u)
        *reinterpret_cast<uint2*>(sm + M::X3 + tile_at(u)) = make_uint2(third[u][0], third[u][1]);
      fence_proxy_async();
      tc_fence_before();
      if (__syncthreads_or(bad)) break;
      tc_fence_after();
      if (tid == 0) {
        product(I2, M::X3, 1);
        commit(4, n);
      }
      __syncwarp();
      wait(bar_i, n);   // S0 and the third term of G have been read
      if (tid == 0 && more && !bad) issue_state(item + gridDim.x, n + 1);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t off = sw128_chunk(row, 2 * part + u);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) split2(w[8 * u + 2 * j], w[8 * u + 2 * j + 1], hi[j], lo[j]);
        *reinterpret_cast<uint4*>(sm + M::W + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        *reinterpret_cast<uint4*>(sm + M::W2 + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) split2(pt[8 * u + 2 * j], pt[8 * u + 2 * j + 1], hi[j], plow[u][j]);
        if (!query) *reinterpret_cast<uint4*>(sm + M::P + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
      }
      suma[part * 128 + row] = s;
    }
    fence_proxy_async();
    tc_fence_before();
    if (__syncthreads_or(bad)) break;
    tc_fence_after();
    if (tid == 0) {
      const uint32_t id = idesc_bf16(128, KD, 0, 1, 0);
#pragma unroll
      for (int s = 0; s < 8; ++s)   // the second terms first
        mma_bf16(D1, dsw(s4, (s >> 2 ? M::W : M::W2) + (s & 3) * 32, 16), dsw(s4, M::KQ + (s & 3) * 2048, 16384), id,
                 s > 0);
#pragma unroll
      for (int s = 0; s < 8; ++s)
        mma_bf16(D2, dsw(s4, (s >> 2 ? M::W : M::W2) + (s & 3) * 32, 16),
                 dsw(s4, M::KQ + 8192 + (s & 3) * 2048, 16384), id, s > 0);
      commit(5, n);
    }
    __syncwarp();
    wait(bar_w, n);
    tc_fence_after();
    if (tid == 0 && more && !bad) issue_front(item + gridDim.x);
    if (!query) {
#pragma unroll
      for (int u = 0; u < 2; ++u)
        *reinterpret_cast<uint4*>(sm + M::P2 + sw128_chunk(row, 2 * part + u)) =
            make_uint4(plow[u][0], plow[u][1], plow[u][2], plow[u][3]);
    }
    // ---- dq (lanes 64..127), dk (lanes 0..63)
    {
      constexpr int COLS = KD / 4;   // of this thread
      const int d0 = part * COLS;
      const float f = query ? up[tok] : down[tok];
      const uint32_t ri = (query ? I1 : I2) + lane_off + d0, rd = (query ? D1 : D2) + lane_off + d0;
      float2 x2 = make_float2(0.f, 0.f);
      const int64_t t = p.tok0 + tok;
      const int64_t to = SHARED ? (t * prm.Hv + h) * KD + d0 : (t * prm.Hqk + hq) * KD + d0;
#pragma unroll
      for (int b = 0; b < COLS; b += 16) {
        float vi[16], vd[16];
        tmem_ld16(ri + b, vi);
        tmem_ld16(rd + b, vd);
        const int col = d0 + b;
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint4 raw = *reinterpret_cast<const uint4*>(sm + M::KQ + (col >> 6) * 16384 +
                                                            sw128_chunk(row, ((col & 63) >> 3) + q));
          const uint32_t rw[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
            x2 = __ffma2_rn(halves(rw[i]), make_float2(vi[8 * q + 2 * i], vi[8 * q + 2 * i + 1]), x2);
        }
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float2 y = __ffma2_rn(make_float2(f, f), make_float2(vi[j], vi[j + 1]), make_float2(vd[j], vd[j + 1]));
          vd[j] = y.x, vd[j + 1] = y.y;
        }
        if (tok < len) {
          if (SHARED) {
            float4* o = reinterpret_cast<float4*>(static_cast<float*>(query ? prm.dq : prm.dk) + to + b);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = make_float4(vd[4 * j], vd[4 * j + 1], vd[4 * j + 2], vd[4 * j + 3]);
          } else {
            uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(query ? prm.dq : prm.dk) + to + b);
#pragma unroll
            for (int j = 0; j < 2; ++j)
              o[j] = make_uint4(pack_bf16(vd[8 * j], vd[8 * j + 1]), pack_bf16(vd[8 * j + 2], vd[8 * j + 3]),
                                pack_bf16(vd[8 * j + 4], vd[8 * j + 5]), pack_bf16(vd[8 * j + 6], vd[8 * j + 7]));
          }
        }
      }
      sumx[part * 128 + row] = (x2.x + x2.y) * f;
    }
    fence_proxy_async();
    tc_fence_before();
    if (__syncthreads_or(bad)) break;
    tc_fence_after();
    // ---- dv
    if (tid == 0) {
      const uint32_t ida = idesc_bf16(128, 64, 1, 0, 0), idb = idesc_bf16(128, 64, 0, 0, 0);
#pragma unroll
      for (int s = 0; s < 8; ++s)
        mma_bf16(I1, dsw(s4, M::VO + 8192 + (s & 3) * 2048, 16384),
                 dsw(s4, (s >> 2 ? M::P : M::P2) + (s & 3) * 32, 16), ida, s > 0);
#pragma unroll
      for (int s = 0; s < 2 * (KD / 16); ++s) {   // two of G's terms
        const int k = s % (KD / 16);
        mma_bf16(I1 + 64, dsw(s4, M::G + s / (KD / 16) * M::kTile + (k >> 2) * (VD * 128) + (k & 3) * 32, 16),
                 dsw(s4, M::KQ + (k >> 2) * 16384 + (k & 3) * 32, 16), idb, s > 0);
      }
      commit(6, n);
    }
    __syncwarp();
    // ---- dg (one warp, under dv's products): sum_{i >= s} row_i + sum_{j < s} out_j + e^{b_last} <G, S0>
    if (warp == 15) {
      float past = lane < 16 ? red[lane] : 0.f;
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) past += __shfl_xor_sync(0xffffffffu, past, o);
      past = __shfl_sync(0xffffffffu, past, 0) * *reinterpret_cast<const float*>(sm + M::Whole);
      const int r = 2 * lane;
      float rw[2], ot[2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        rw[u] = 0.f, ot[u] = 0.f;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          rw[u] += suma[q * 128 + 64 + r + u] - suma[q * 128 + r + u] + sumx[q * 128 + 64 + r + u];
          ot[u] += sumx[q * 128 + r + u];
        }
      }
      float suf = rw[0] + rw[1], pre = ot[0] + ot[1];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const float a = __shfl_down_sync(0xffffffffu, suf, o), b = __shfl_up_sync(0xffffffffu, pre, o);
        if (lane + o < 32) suf += a;
        if (lane >= o) pre += b;
      }
      const float before = __shfl_up_sync(0xffffffffu, pre, 1), after = __shfl_down_sync(0xffffffffu, suf, 1);
      const float b0 = lane ? before : 0.f, a1 = lane < 31 ? after : 0.f;
      const float x0 = (rw[0] + (rw[1] + a1)) + b0 + past, x1 = (rw[1] + a1) + (b0 + ot[0]) + past;
      if (prm.g_per_head) {
        float s = (r < len ? x0 : 0.f) + (r + 1 < len ? x1 : 0.f);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane == 0) prm.dg[item] = s;
      } else {
        float* gp = prm.dg + p.tok0 * prm.Hv + h;
        if (r < len) gp[(int64_t)r * prm.Hv] = x0;
        if (r + 1 < len) gp[(int64_t)(r + 1) * prm.Hv] = x1;
      }
    }
    wait(bar_v, n);
    tc_fence_after();
    if (row < VD) {
      // this thread has value column `row` for 16 tokens; neighbouring lanes exchange values for bf16 pairs
      float a[16], b[16];
      tmem_ld16(I1 + lane_off + 16 * part, a);
      tmem_ld16(I1 + lane_off + 64 + 16 * part, b);
      const bool odd = lane & 1;
      __nv_bfloat16* to = prm.dv + (p.tok0 * prm.Hv + h) * (int64_t)VD + (row & ~1);
#pragma unroll
      for (int pp = 0; pp < 8; ++pp) {
        const int j = 16 * part + 2 * pp;
        const float v0 = fmaf(down[j], b[2 * pp], a[2 * pp]), v1 = fmaf(down[j + 1], b[2 * pp + 1], a[2 * pp + 1]);
        const float other = __shfl_xor_sync(0xffffffffu, odd ? v0 : v1, 1);
        const uint32_t word = odd ? pack_bf16(other, v1) : pack_bf16(v0, other);
        const int jj = j + (odd ? 1 : 0);
        if (jj < len) *reinterpret_cast<uint32_t*>(to + (int64_t)jj * prm.Hv * VD) = word;
      }
    }
    tc_fence_before();
    // every thread has read this chunk's decays, sums and products
    if (__syncthreads_or(bad)) break;
    tc_fence_after();
    if (tid == 0 && more) {
      issue_tiles(item + gridDim.x, n + 1);
      issue_adjoint(item + gridDim.x, n + 1);
    }
  }
  if (__syncthreads_or(bad) && tid == 0) {
    for (int b = 0; b < 8; ++b)
      if (count[b] > 0) mbar_wait(bars + b, (count[b] - 1) & 1, prm.status, 100000000ull);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

struct Layout {
  int seg;
  size_t seg_tables, chunk_tables, decays, total, own, part, states, adjoints, dq, dk, end;
};

Layout layout_of(const gdn_linear_problem& p) {
  Layout L;
  L.seg = segment_tokens(p);
  const size_t segs = L.seg < p.T ? (size_t)pieces_max(p, L.seg) * p.Hv : 0;
  const size_t slots = ((size_t)p.B * p.T / 64 + p.N + 1) * p.Hv, tile = 4 * (size_t)p.K * p.V;
  L.seg_tables = kAlign;
  L.chunk_tables = L.seg_tables + pieces_bytes(p, L.seg);
  L.decays = L.chunk_tables + pieces_bytes(p, 64);
  L.total = L.decays + decays_bytes(p);
  L.own = L.total + align_up(sizeof(Two) * segs);
  L.part = L.own + segs * tile;
  L.states = L.part + (p.g_per_head ? align_up(4 * (size_t)pieces_max(p, 64) * p.Hv) : 0);
  L.adjoints = L.states + slots * tile;
  L.dq = L.adjoints + slots * tile;
  const size_t heads = p.Hv == p.Hqk ? 0 : align_up(4 * (size_t)p.B * p.T * p.Hv * p.K);
  L.dk = L.dq + heads;
  L.end = L.dk + heads;
  return L;
}

template <int KD, int VD, bool SHARED>
gdn_status launch_grads(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& td,
                        const GradParams& prm, cudaStream_t s) {
  auto kern = grads_tc_kernel<KD, VD, SHARED>;
  constexpr int bytes = (int)GradMap<KD, VD>::Bytes;
  static_assert(bytes <= 232448, "shared memory of one SM");
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return GDN_ERR_CUDA;
  const int sms = sm_count();
  kern<<<prm.items < sms ? prm.items : sms, kGradThreads, bytes, s>>>(tq, tk, tv, td, prm);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace

bool tc_bwd_supported(const gdn_linear_problem& p) { return p.dt == GDN_BF16 && p.K <= 128 && p.V <= 128; }

size_t tc_bwd_bytes(const gdn_linear_problem& p) { return layout_of(p).end; }

gdn_status tc_bwd(const gdn_linear_problem& p, const void* q, const void* k, const void* v, const float* g, float scale,
                  const float* h0, const int32_t* cu, const void* dout, const float* dht, void* dq, void* dk, void* dv,
                  float* dg, float* dh0, void* ws, cudaStream_t s) {
  uint8_t* at = static_cast<uint8_t*>(ws);
  int32_t* status = reinterpret_cast<int32_t*>(at);
  const Layout L = layout_of(p);
  if (launch_pieces(p, L.seg, cu, at + L.seg_tables, status, true, s) != cudaSuccess) return GDN_ERR_CUDA;
  if (launch_pieces(p, 64, cu, at + L.chunk_tables, status, false, s) != cudaSuccess) return GDN_ERR_CUDA;
  const Pieces segs = pieces_at(p, L.seg, at + L.seg_tables), chunks = pieces_at(p, 64, at + L.chunk_tables);
  gdn_status st = launch_empty(p, segs, cu, dht, dh0, nullptr, 0, s);
  if (st != GDN_OK) return st;
  const int64_t tokens = (int64_t)p.B * p.T;
  float* part = reinterpret_cast<float*>(at + L.part);
  if (tokens > 0) {
    float* decays = reinterpret_cast<float*>(at + L.decays);
    st = launch_decays(p, segs, L.seg, g, scale, decays, s);
    const int64_t ldo = (int64_t)p.Hv * p.V;
    TcParams prm = tc_params(p, segs, cu, scale, decays, status);
    prm.total = reinterpret_cast<Two*>(at + L.total);
    prm.own = reinterpret_cast<float*>(at + L.own);
    const bool cut = L.seg < p.T;
    if (st == GDN_OK && cut) {
      st = launch_walk(p, kOwn, false, nullptr, k, p.ld_k, v, p.ld_v, nullptr, prm, L.seg, s);
      if (st == GDN_OK)
        st = launch_sums(shape_of(p), segs, p.N, prm.total, Sum{h0, prm.own, nullptr, nullptr, 0, false}, s);
    }
    TcParams walk = prm;
    walk.start = cut ? prm.own : nullptr;
    walk.h0 = h0;
    walk.emit = reinterpret_cast<float*>(at + L.states);
    if (st == GDN_OK) st = launch_walk(p, kEmit, false, nullptr, k, p.ld_k, v, p.ld_v, nullptr, walk, L.seg, s);
    if (st == GDN_OK && cut) {
      st = launch_walk(p, kOwn, true, nullptr, q, p.ld_q, dout, ldo, nullptr, prm, L.seg, s);
      if (st == GDN_OK)
        st = launch_sums(shape_of(p), segs, p.N, prm.total, Sum{dht, prm.own, nullptr, nullptr, 0, true}, s);
    }
    walk.h0 = dht;
    walk.ht = dh0;
    walk.emit = reinterpret_cast<float*>(at + L.adjoints);
    if (st == GDN_OK) st = launch_walk(p, kEmit, true, nullptr, q, p.ld_q, dout, ldo, nullptr, walk, L.seg, s);
    if (st != GDN_OK) return st;

    CUtensorMap tq, tk, tv, td;
    const uint32_t box[3] = {64, 1, 64};
    const uint64_t kd[3] = {(uint64_t)p.K, (uint64_t)p.Hqk, (uint64_t)tokens};
    const uint64_t vd[3] = {(uint64_t)p.V, (uint64_t)p.Hv, (uint64_t)tokens};
    const uint64_t sq[2] = {(uint64_t)p.K * 2, (uint64_t)p.ld_q * 2}, sk[2] = {(uint64_t)p.K * 2, (uint64_t)p.ld_k * 2};
    const uint64_t sv[2] = {(uint64_t)p.V * 2, (uint64_t)p.ld_v * 2}, so[2] = {(uint64_t)p.V * 2, (uint64_t)ldo * 2};
    if (!make_tmap_bf16(&tq, q, 3, kd, sq, box) || !make_tmap_bf16(&tk, k, 3, kd, sk, box) ||
        !make_tmap_bf16(&tv, v, 3, vd, sv, box) || !make_tmap_bf16(&td, dout, 3, vd, so, box))
      return GDN_ERR_CUDA;
    const bool shared = p.Hv != p.Hqk;
    GradParams gp;
    memset(&gp, 0, sizeof(gp));
    gp.decays = decays;
    gp.states = reinterpret_cast<const float*>(at + L.states);
    gp.adjoints = reinterpret_cast<const float*>(at + L.adjoints);
    gp.dq = shared ? at + L.dq : dq;
    gp.dk = shared ? at + L.dk : dk;
    gp.dv = static_cast<__nv_bfloat16*>(dv);
    gp.dg = p.g_per_head ? part : dg;
    gp.status = status;
    gp.pc = chunks;
    gp.items = pieces_max(p, 64) * p.Hv;
    gp.Hqk = p.Hqk;
    gp.Hv = p.Hv;
    gp.g_per_head = p.g_per_head;
    gp.scale = scale;
#define GDN_GRADS(K, V)                                                                                              \
  st = shared ? launch_grads<K, V, true>(tq, tk, tv, td, gp, s) : launch_grads<K, V, false>(tq, tk, tv, td, gp, s)
    if (p.K == 64 && p.V == 64) GDN_GRADS(64, 64);
    else if (p.K == 64) GDN_GRADS(64, 128);
    else if (p.V == 64) GDN_GRADS(128, 64);
    else GDN_GRADS(128, 128);
#undef GDN_GRADS
    if (st != GDN_OK) return st;
    if (shared) {
      st = launch_heads<__nv_bfloat16>(p, reinterpret_cast<const float*>(at + L.dq),
                                       reinterpret_cast<const float*>(at + L.dk), chunks.nc,
                                       static_cast<__nv_bfloat16*>(dq), static_cast<__nv_bfloat16*>(dk), s);
      if (st != GDN_OK) return st;
    }
  }
  return p.g_per_head ? launch_head_decays(p, part, chunks.nc, dg, s) : GDN_OK;
}

}  // namespace lin
}  // namespace gdn
