// gdn_linear_bwd.cu -- backward of decayed linear attention with fp32 precision throughout, for fp32 and for bf16 with
// a head dim of 256 (other bf16 problems: gdn_linear_tc_bwd.cu).
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
#include "gdn_linear_tc32.cuh"

namespace gdn {
namespace lin {
namespace {

constexpr int kGradThreads = 512;

// Over a warp: x[j] summed over the lanes, in lane sum_of16(lane) = j (and in the lane beside it).
__device__ __forceinline__ int sum_of16(int lane) {
  return (lane >> 4 & 1) * 8 + (lane >> 3 & 1) * 4 + (lane >> 2 & 1) * 2 + (lane >> 1 & 1);
}
__device__ __forceinline__ float reduce16(float (&x)[16], int lane) {
#pragma unroll
  for (int n = 8; n >= 1; n >>= 1) {
    const bool upper = lane & (2 * n);
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const float give = upper ? x[j] : x[j + n], keep = upper ? x[j + n] : x[j];
      x[j] = keep + __shfl_xor_sync(0xffffffffu, give, 2 * n);
    }
  }
  return x[0] + __shfl_xor_sync(0xffffffffu, x[0], 1);
}

// A term's tile of 64 rows of 64: 8 KB.  DB, EB: columns of K, of V a stage takes.
template <typename T, int DB, int EB>
struct GradMap32 {
  static constexpr int TERMS = kTerms<T>;
  static constexpr uint32_t kT = 8192;
  // stages: Q | K;  dO | V | S0 [d][e] | G;  K | Q, DB columns each;  G [d][e] | K | dO
  static constexpr uint32_t kKQ = 64 * DB * 2, kSG = DB * 128, kGE = 64 * EB * 2;
  static constexpr uint32_t S = 2 * TERMS * kT, G = S + 3 * kSG;
  static constexpr uint32_t KE = 3 * kGE, OE = KE + TERMS * kT;
  static constexpr uint32_t kEnd1 = G + 3 * kSG, kEnd2 = 2 * TERMS * kKQ, kEnd3 = OE + TERMS * kGE;
  static constexpr uint32_t W = kEnd1 > kEnd2 ? (kEnd1 > kEnd3 ? kEnd1 : kEnd3) : (kEnd2 > kEnd3 ? kEnd2 : kEnd3);
  static constexpr uint32_t P = W + 3 * kT;
  static constexpr uint32_t Misc = P + 3 * kT;
  static constexpr uint32_t Hi = Misc, Lo = Misc + 256, Up = Misc + 512, Down = Misc + 768;
  static constexpr uint32_t RowA = Misc + 1024, ColA = RowA + 1024;   // [4 parts][64], [2 warps' rows][64]
  static constexpr uint32_t SumQ = ColA + 512, SumK = SumQ + 1024;    // [4 warps' rows][64] each
  static constexpr uint32_t Red = SumK + 1024, Bar = Red + 64, Flags = Bar + 8;
  static constexpr uint32_t Bytes = Flags + 56 + 1024;
};

// Gradients of one chunk of one value head.  TMEM lane = token (Q K^T, dO V^T) or column of K or V (all else, so that a
// warp writes 32 neighbours of a row); one batch of products at a time, the next tiles' loads under it.  Bound by those
// rounds of loading, splitting, products and a wait (seven for K = V = 128, 10k cycles each; tensor pipe 15 %, HBM 16 %,
// issue 27 % with 16 warps).  2 x 4096 tokens of 16 heads: fp32 of 128 500 us (fp32 FMAs on 64 x 64 tiles: 950), bf16 of
// 256 877 (3040).  Prefetching the states of the CTA behind to L2 changed nothing (498 against 494, 916 against 866).
// DROP (a test's): the waits for one batch of products run out in some warps of the first CTA.
template <typename T, typename TG, int DB, int EB, bool DROP>
__global__ void __launch_bounds__(kGradThreads, 1) grads_kernel(
    const T* __restrict__ q, const T* __restrict__ k, const T* __restrict__ v, const T* __restrict__ dout, Shape d,
    const float* __restrict__ g, Pieces pc, float scale, const float* __restrict__ S0, const float* __restrict__ G,
    TG* __restrict__ dq, TG* __restrict__ dk, T* __restrict__ dv, float* __restrict__ dg, int32_t* status,
    int drop_batch, uint32_t drop_warps) {
  using M = GradMap32<T, DB, EB>;
  constexpr int TERMS = M::TERMS, N = kGradThreads;
  constexpr uint32_t kT = M::kT;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int c = blockIdx.x / d.Hv, h = blockIdx.x % d.Hv, hq = h / (d.Hv / d.Hqk);
  const Piece p = piece_of(pc, c);
  if (!p.ok) return;
  uint8_t* sm = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t s4 = (smem_u32(sm) & 0x3FFFFu) >> 4;
  float *hi = reinterpret_cast<float*>(sm + M::Hi), *lo = reinterpret_cast<float*>(sm + M::Lo);
  float *up = reinterpret_cast<float*>(sm + M::Up), *down = reinterpret_cast<float*>(sm + M::Down);
  float *rowa = reinterpret_cast<float*>(sm + M::RowA), *cola = reinterpret_cast<float*>(sm + M::ColA);
  float *sumq = reinterpret_cast<float*>(sm + M::SumQ), *sumk = reinterpret_cast<float*>(sm + M::SumK);
  float* red = reinterpret_cast<float*>(sm + M::Red);
  uint64_t* bar = reinterpret_cast<uint64_t*>(sm + M::Bar);
  uint32_t* flags = reinterpret_cast<uint32_t*>(sm + M::Flags);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int qd = warp & 3, part = warp >> 2, row = 32 * qd + lane, t0 = 16 * part;   // lane of TMEM, first of 16 columns
  if (tid == 0) {
    mbar_init(bar, 1);
    mbar_fence_init();
  }
  if (warp == 0) tmem_alloc(flags, 512);
  if (warp == 1) {
    chunk_sums(g + (d.g_per_head ? h : p.tok0 * d.Hv + h), d.g_per_head ? 0 : d.Hv, p.len, lane, hi, lo);
    __syncwarp();
#pragma unroll
    for (int r = lane; r < kC; r += 32) {
      up[r] = scale * expf(hi[r] + lo[r]);
      down[r] = expf((hi[kC - 1] - hi[r]) + (lo[kC - 1] - lo[r]));
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(flags);
  const uint32_t mine = tmem + (static_cast<uint32_t>(32 * qd) << 16) + t0;
  // columns; a sum over several tiles has another accumulator 64 behind, for all but the products of first terms
  constexpr uint32_t QK = 0, OV = 128, IQ = 256, IK = 384, WK = OV, WQ = OV + 64, IV = QK, PO = OV;

  const T* qp = q + p.tok0 * d.ldq + (int64_t)hq * d.K;
  const T* kp = k + p.tok0 * d.ldk + (int64_t)hq * d.K;
  const T* vp = v + p.tok0 * d.ldv + (int64_t)h * d.V;
  const int64_t ldo = (int64_t)d.Hv * d.V, ldg = (int64_t)d.Hv * d.K;
  const T* op = dout + p.tok0 * ldo + (int64_t)h * d.V;
  const float* sp = S0 + ((int64_t)c * d.Hv + h) * d.K * d.V;
  const float* gp = G + ((int64_t)c * d.Hv + h) * d.K * d.V;

  // A warp's waits can run out when another's do not.  `good` is the warp's own from drained() to the next ready(), which
  // makes it the CTA's: no loop begins, ends or is left on it but behind ready(), or warps would meet different barriers.
  int n = 0;          // batches of products issued
  bool good = true;
  auto drained = [&] {   // they have been read and summed
    if (good && n > 0) good = warp_wait(bar, (n - 1) & 1, status);
    if constexpr (DROP)
      if (blockIdx.x == 0 && n - 1 == drop_batch && (drop_warps >> warp & 1)) {
        good = false;
        if (lane == 0) atomicExch(status, GDN_DEV_WAIT_TIMEOUT);
      }
  };
  auto ready = [&] {     // tiles are in place, TMEM has been read
    fence_proxy_async();
    tc_fence_before();
    if (__syncthreads_or(!good)) good = false;
    tc_fence_after();
    return good;
  };
  // one step of 16 of a sum over tiles at column `at`: products of terms a and b, in products()'s order
  auto tiles = [&](uint32_t at, uint64_t A, uint64_t B, uint32_t id, int a, int b, uint32_t more, bool begun) {
    const bool first = a + b == 0;
    mma_bf16(tmem + at + (first ? 0 : 64), A, B, id, begun ? 1u : (first ? 0u : more));
  };
  auto sum_ld = [&](uint32_t at, float (&x)[16], bool rest) {
    tmem_ld16(mine + at, x);
    if (rest) {
      float y[16];
      tmem_ld16(mine + at + 64, y);
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] += y[j];
    }
  };

  // ---- Q K^T
#pragma unroll 1
  for (int kb = 0; kb < d.K / 64; ++kb) {
    float4 xq[2], xk[2];
    fetch<64, 64, N>(xq, qp + 64 * kb, d.ldq, p.len);
    fetch<64, 64, N>(xk, kp + 64 * kb, d.ldk, p.len);
    drained();
    if (good) {
      place<64, 64, TERMS, N>(sm, xq, nullptr);
      place<64, 64, TERMS, N>(sm + TERMS * kT, xk, nullptr);
    }
    if (!ready()) break;
    if (tid == 0) {
      const uint32_t id = idesc_bf16(128, 64, 0, 0, 0);
      products<TERMS, TERMS>([&](int a, int b, uint32_t more) {
#pragma unroll
        for (int s = 0; s < 4; ++s)
          tiles(QK, dsw(s4, a * kT + s * 32, 16), dsw(s4, (TERMS + b) * kT + s * 32, 16), id, a, b, more,
                kb > 0 || s > 0);
      });
      mma_commit(bar);
    }
    ++n;
    __syncwarp();
  }
  // ---- DB columns of dq, dk at a time
  float gs = 0.f;   // <G, S0>
#pragma unroll 1
  for (int db = 0; db < d.K / DB; ++db) {
#pragma unroll 1
    for (int vb = 0; vb < d.V / 64; ++vb) {
      float4 xo[2], xv[2], xs[DB / 32], xg[DB / 32];
      fetch<64, 64, N>(xo, op + 64 * vb, ldo, p.len);
      fetch<64, 64, N>(xv, vp + 64 * vb, d.ldv, p.len);
      fetch<DB, 64, N>(xs, sp + (int64_t)db * DB * d.V + 64 * vb, d.V, DB);
      fetch<DB, 64, N>(xg, gp + (int64_t)db * DB * d.V + 64 * vb, d.V, DB);
#pragma unroll
      for (int u = 0; u < DB / 32; ++u)
        gs = fmaf(xs[u].x, xg[u].x, fmaf(xs[u].y, xg[u].y, fmaf(xs[u].z, xg[u].z, fmaf(xs[u].w, xg[u].w, gs))));
      drained();
      if (good) {
        place<64, 64, TERMS, N>(sm, xo, nullptr);
        place<64, 64, TERMS, N>(sm + TERMS * kT, xv, nullptr);
        place<DB, 64, 3, N>(sm + M::S, xs, nullptr);
        place<DB, 64, 3, N>(sm + M::G, xg, nullptr);
      }
      if (!ready()) break;
      if (tid == 0) {
        const uint32_t id = idesc_bf16(128, 64, 0, 0, 0);
        if (db == 0)
          products<TERMS, TERMS>([&](int a, int b, uint32_t more) {
#pragma unroll
            for (int s = 0; s < 4; ++s)
              tiles(OV, dsw(s4, a * kT + s * 32, 16), dsw(s4, (TERMS + b) * kT + s * 32, 16), id, a, b, more,
                    vb > 0 || s > 0);
          });
        products<3, TERMS>([&](int a, int b, uint32_t more) {
#pragma unroll
          for (int s = 0; s < 4; ++s)
            tiles(IQ, dsw(s4, M::S + a * M::kSG + s * 32, 16), dsw(s4, b * kT + s * 32, 16), id, a, b, more,
                  vb > 0 || s > 0);
        });
        products<3, TERMS>([&](int a, int b, uint32_t more) {
#pragma unroll
          for (int s = 0; s < 4; ++s)
            tiles(IK, dsw(s4, M::G + a * M::kSG + s * 32, 16), dsw(s4, (TERMS + b) * kT + s * 32, 16), id, a, b, more,
                  vb > 0 || s > 0);
        });
        mma_commit(bar);
      }
      ++n;
      __syncwarp();
    }
    if (!good) break;
    float4 xk[DB / 32], xq[DB / 32];
    fetch<64, DB, N>(xk, kp + db * DB, d.ldk, p.len);
    fetch<64, DB, N>(xq, qp + db * DB, d.ldq, p.len);
    drained();
    tc_fence_after();
    if (db == 0 && qd < 2 && good) {   // W, P and the sums of A: 16 columns of row `row`
      float qk[16], ov[16];
      sum_ld(QK, qk, TERMS > 1);
      sum_ld(OV, ov, TERMS > 1);
      const float b0 = hi[row], b1 = lo[row];
      float rs = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int col = t0 + j;
        const float m = scale * expf((b0 - hi[col]) + (b1 - lo[col]));
        const float w = col <= row ? m * ov[j] : 0.f, a = col < row ? w * qk[j] : 0.f;   // a token with itself has no
        qk[j] = col <= row ? m * qk[j] : 0.f;                                            // decay between
        rs += a;
        ov[j] = w;
      }
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const float(&x)[16] = m ? qk : ov;
        uint8_t* at = sm + (m ? M::P : M::W);
#pragma unroll
        for (int j = 0; j < 16; j += 8) {
          uint32_t a0[2], a1[2], a2[2], c0[2], c1[2], c2[2];
          split3(make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]), a0, a1, a2);
          split3(make_float4(x[j + 4], x[j + 5], x[j + 6], x[j + 7]), c0, c1, c2);
          uint8_t* to = at + sw128_chunk(row, (t0 + j) >> 3);
          *reinterpret_cast<uint4*>(to) = make_uint4(a0[0], a0[1], c0[0], c0[1]);
          *reinterpret_cast<uint4*>(to + kT) = make_uint4(a1[0], a1[1], c1[0], c1[1]);
          *reinterpret_cast<uint4*>(to + 2 * kT) = make_uint4(a2[0], a2[1], c2[0], c2[1]);
        }
      }
      // A's columns: w (q k) again, from the products
      float x[16];
      sum_ld(QK, x, TERMS > 1);
#pragma unroll
      for (int j = 0; j < 16; ++j) x[j] = t0 + j < row ? ov[j] * x[j] : 0.f;
      rowa[part * 64 + row] = rs;
      const float cs = reduce16(x, lane);
      if (!(lane & 1)) cola[qd * 64 + t0 + sum_of16(lane)] = cs;
    }
    if (good) {
      place<64, DB, TERMS, N>(sm, xk, nullptr);
      place<64, DB, TERMS, N>(sm + TERMS * M::kKQ, xq, nullptr);
    }
    if (!ready()) break;
    if (tid == 0) {
      const uint32_t idn = idesc_bf16(128, 64, 1, 0, 0), idt = idesc_bf16(128, 64, 1, 1, 0);
      products<TERMS, 3>([&](int a, int b, uint32_t more) {   // (W K)^T: lanes d, columns i
#pragma unroll
        for (int s = 0; s < 4; ++s)
          mma_bf16(tmem + WK, dsw(s4, a * M::kKQ + s * 2048, kT), dsw(s4, M::W + b * kT + s * 32, 16), idn,
                   s > 0 ? 1u : more);
      });
      products<TERMS, 3>([&](int a, int b, uint32_t more) {   // (W^T Q)^T: lanes d, columns j
#pragma unroll
        for (int s = 0; s < 4; ++s)
          mma_bf16(tmem + WQ, dsw(s4, (TERMS + a) * M::kKQ + s * 2048, kT), dsw(s4, M::W + b * kT + s * 2048, kT), idt,
                   s > 0 ? 1u : more);
      });
      mma_commit(bar);
    }
    ++n;
    __syncwarp();
    drained();
    tc_fence_after();
    if (good) {
#pragma unroll
      for (int m = 0; m < 2; ++m) {   // dq, dk: column db DB + row of 16 tokens
        const T* src = (m ? kp : qp) + db * DB + row;
        const int64_t ld = m ? d.ldk : d.ldq;
        TG* to = (m ? dk : dq) + p.tok0 * ldg + (int64_t)h * d.K + db * DB + row;
        const float* f = m ? down : up;
        float in[16], own[16];
        sum_ld(m ? IK : IQ, in, true);
        tmem_ld16(mine + (m ? WQ : WK), own);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int t = t0 + j;
          const bool is = t < p.len && row < DB;
          const float y = f[t] * in[j];
          if (is) to[t * ldg] = from_f<TG>(own[j] + y);
          in[j] = is ? to_f(src[t * ld]) * y : 0.f;
        }
        const float s = reduce16(in, lane);
        float* at = (m ? sumk : sumq) + qd * 64 + t0 + sum_of16(lane);
        if (!(lane & 1)) *at = db ? *at + s : s;
      }
    }
  }
  // ---- EB columns of dv at a time
#pragma unroll 1
  for (int eb = 0; eb < d.V / EB; ++eb) {
#pragma unroll 1
    for (int kb = 0; kb < d.K / 64; ++kb) {
      float4 xg[EB / 32], xk[2], xo[EB / 32];
      fetch<64, EB, N>(xg, gp + (int64_t)64 * kb * d.V + eb * EB, d.V, 64);
      fetch<64, 64, N>(xk, kp + 64 * kb, d.ldk, p.len);
      if (kb == 0) fetch<64, EB, N>(xo, op + eb * EB, ldo, p.len);
      drained();
      if (good) {
        place<64, EB, 3, N>(sm, xg, nullptr);
        place<64, 64, TERMS, N>(sm + M::KE, xk, nullptr);
        if (kb == 0) place<64, EB, TERMS, N>(sm + M::OE, xo, nullptr);
      }
      if (!ready()) break;
      if (tid == 0) {
        const uint32_t idn = idesc_bf16(128, 64, 1, 0, 0), idt = idesc_bf16(128, 64, 1, 1, 0);
        products<3, TERMS>([&](int a, int b, uint32_t more) {   // (K G)^T: lanes e, columns j
#pragma unroll
          for (int s = 0; s < 4; ++s)
            tiles(IV, dsw(s4, a * M::kGE + s * 2048, kT), dsw(s4, M::KE + b * kT + s * 32, 16), idn, a, b, more,
                  kb > 0 || s > 0);
        });
        if (kb == 0)
          products<TERMS, 3>([&](int a, int b, uint32_t more) {   // (P^T dO)^T
#pragma unroll
            for (int s = 0; s < 4; ++s)
              mma_bf16(tmem + PO, dsw(s4, M::OE + a * M::kGE + s * 2048, kT), dsw(s4, M::P + b * kT + s * 2048, kT), idt,
                       s > 0 ? 1u : more);
          });
        mma_commit(bar);
      }
      ++n;
      __syncwarp();
    }
    if (!good) break;
    drained();
    tc_fence_after();
    if (good) {
      float in[16], own[16];
      sum_ld(IV, in, true);
      tmem_ld16(mine + PO, own);
      T* to = dv + p.tok0 * ldo + (int64_t)h * d.V + eb * EB + row;
#pragma unroll
      for (int j = 0; j < 16; ++j)
        if (t0 + j < p.len && row < EB) to[(t0 + j) * ldo] = from_f<T>(fmaf(down[t0 + j], in[j], own[j]));
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) gs += __shfl_xor_sync(0xffffffffu, gs, o);
  if (lane == 0) red[warp] = gs;
  tc_fence_before();
  const bool stop = __syncthreads_or(!good);
  if (stop && tid == 0 && n > 0) mbar_wait(bar, (n - 1) & 1, status, 100000000ull);   // products under way end first
  if (!stop && warp == 1) {
    // dg_s = sum_{i >= s} row_i + sum_{j < s} out_j + e^{b_last} <G, S0>
    double past = 0.0;
#pragma unroll
    for (int w = 0; w < N / 32; ++w) past += red[w];
    const Two whole = exp_two({hi[kC - 1], lo[kC - 1]});
    past *= (double)whole.h + whole.l;
    const int r = 2 * lane;
    double rw[2], ot[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      rw[u] = -(double)cola[r + u] - cola[64 + r + u], ot[u] = 0.0;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        rw[u] += (double)rowa[w * 64 + r + u];
        if (32 * w < DB) rw[u] += (double)sumq[w * 64 + r + u], ot[u] += (double)sumk[w * 64 + r + u];
      }
    }
    double suf = rw[0] + rw[1], pre = ot[0] + ot[1];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const double a = __shfl_down_sync(0xffffffffu, suf, o), b = __shfl_up_sync(0xffffffffu, pre, o);
      if (lane + o < 32) suf += a;
      if (lane >= o) pre += b;
    }
    pre -= ot[0] + ot[1];
    const double x0 = suf + pre + past, x1 = suf - rw[0] + pre + ot[0] + past;
    if (d.g_per_head) {
      double s = (r < p.len ? x0 : 0.0) + (r + 1 < p.len ? x1 : 0.0);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
      if (lane == 0) dg[(int64_t)c * d.Hv + h] = (float)s;
    } else {
      float* to = dg + p.tok0 * d.Hv + h;
      if (r < p.len) to[(int64_t)r * d.Hv] = (float)x0;
      if (r + 1 < p.len) to[(int64_t)(r + 1) * d.Hv] = (float)x1;
    }
  }
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, 512);
}

// What a test drops of the first CTA's waits (-1: nothing).
struct Drop {
  int batch;
  uint32_t warps;
};

template <typename T, typename TG, int DB, int EB, bool DROP>
gdn_status launch_grads(int most, const T* q, const T* k, const T* v, const T* dout, const Shape& d, const float* g,
                        const Pieces& pc, float scale, const float* S, const float* G, TG* dq, TG* dk, T* dv,
                        float* dg, int32_t* status, Drop drop, cudaStream_t s) {
  auto kern = grads_kernel<T, TG, DB, EB, DROP>;
  constexpr int bytes = (int)GradMap32<T, DB, EB>::Bytes;
  static_assert(bytes <= 232448, "shared memory of one SM");
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
    return GDN_ERR_CUDA;
  kern<<<(unsigned)((int64_t)most * d.Hv), kGradThreads, bytes, s>>>(q, k, v, dout, d, g, pc, scale, S, G, dq, dk, dv,
                                                                     dg, status, drop.batch, drop.warps);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

template <typename T, typename TG>
gdn_status run_grads(int most, const T* q, const T* k, const T* v, const T* dout, const Shape& d, const float* g,
                     const Pieces& pc, float scale, const float* S, const float* G, TG* dq, TG* dk, T* dv, float* dg,
                     int32_t* status, Drop drop, cudaStream_t s) {
#define GDN_GRADS_DROP(DB, EB, DROP) \
  return launch_grads<T, TG, DB, EB, DROP>(most, q, k, v, dout, d, g, pc, scale, S, G, dq, dk, dv, dg, status, drop, s)
#define GDN_GRADS(DB, EB) GDN_GRADS_DROP(DB, EB, false)
  if constexpr (sizeof(T) == 4 && sizeof(TG) == 4) {
    if (drop.batch >= 0) GDN_GRADS_DROP(128, 128, true);
  }
  if (d.K == 64 && d.V != 64) GDN_GRADS(64, 128);
  if (d.K != 64 && d.V == 64) GDN_GRADS(128, 64);
  if constexpr (sizeof(T) == 4) {   // bf16 comes here with a head dim of 256 alone
    if (d.K == 64) GDN_GRADS(64, 64);
  }
  GDN_GRADS(128, 128);
#undef GDN_GRADS
#undef GDN_GRADS_DROP
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

struct Layout {
  size_t tables, total, part, states, adjoints, dq, dk, end;
};

Layout layout_of(const gdn_linear_problem& p) {
  const size_t cells = (size_t)pieces_max(p, kC) * p.Hv;
  Layout L;
  L.tables = kAlign;
  L.total = L.tables + pieces_bytes(p, kC);
  L.part = L.total + align_up(sizeof(Two) * cells);
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
                 const Pieces& pc, const Layout& L, uint8_t* ws, Drop drop, cudaStream_t s) {
  const Shape d = shape_of(p);
  const int most = pieces_max(p, kC);
  int32_t* status = reinterpret_cast<int32_t*>(ws);
  Two* total = reinterpret_cast<Two*>(ws + L.total);
  float* S = reinterpret_cast<float*>(ws + L.states);
  float* G = reinterpret_cast<float*>(ws + L.adjoints);
  const Side<T> states{k, v, p.ld_k, p.ld_v, 1.f, S, false};
  const Side<T> adjoints{q, dout, p.ld_q, (int64_t)p.Hv * p.V, scale, G, true};
  gdn_status st = launch_states(d, states, adjoints, 2, g, pc, most, total, status, s);
  const Sum forth{h0, S, nullptr, nullptr, 0, false}, back{dht, G, dh0, nullptr, 0, true};
  if (dh0 && dh0 == h0) {   // read before it is written
    if (st == GDN_OK) st = launch_sums(d, pc, p.N, total, forth, s);
    if (st == GDN_OK) st = launch_sums(d, pc, p.N, total, back, s);
  } else if (st == GDN_OK) {
    st = launch_sums(d, pc, p.N, total, forth, back, 2, s);
  }
  if (st != GDN_OK) return st;
  float* part = reinterpret_cast<float*>(ws + L.part);
  const bool shared = p.Hv != p.Hqk;
  if (most > 0) {
    float* dgp = p.g_per_head ? part : dg;
    if (shared)
      st = run_grads<T, float>(most, q, k, v, dout, d, g, pc, scale, S, G, reinterpret_cast<float*>(ws + L.dq),
                               reinterpret_cast<float*>(ws + L.dk), dv, dgp, status, drop, s);
    else
      st = run_grads<T, T>(most, q, k, v, dout, d, g, pc, scale, S, G, dq, dk, dv, dgp, status, drop, s);
    if (st != GDN_OK) return st;
  }
  if (shared && (int64_t)p.B * p.T > 0) {
    st = launch_heads<T>(p, reinterpret_cast<const float*>(ws + L.dq), reinterpret_cast<const float*>(ws + L.dk), pc.nc,
                         dq, dk, s);
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

size_t bwd32_bytes(const gdn_linear_problem& p) { return layout_of(p).end; }

gdn_status bwd32(const gdn_linear_problem& p, const void* q, const void* k, const void* v, const float* g, float scale,
                 const float* h0, const int32_t* cu, const void* dout, const float* dht, void* dq, void* dk, void* dv,
                 float* dg, float* dh0, void* ws, Drop drop, cudaStream_t s) {
  uint8_t* at = static_cast<uint8_t*>(ws);
  int32_t* status = reinterpret_cast<int32_t*>(at);
  const Layout L = layout_of(p);
  if (launch_pieces(p, kC, cu, at + L.tables, status, true, s) != cudaSuccess) return GDN_ERR_CUDA;
  const Pieces pc = pieces_at(p, kC, at + L.tables);
  if (p.dt == GDN_F32)
    return bwd_t<float>(p, (const float*)q, (const float*)k, (const float*)v, g, scale, h0, (const float*)dout, dht,
                        (float*)dq, (float*)dk, (float*)dv, dg, dh0, pc, L, at, drop, s);
  using T = __nv_bfloat16;
  return bwd_t<T>(p, (const T*)q, (const T*)k, (const T*)v, g, scale, h0, (const T*)dout, dht, (T*)dq, (T*)dk, (T*)dv,
                  dg, dh0, pc, L, at, drop, s);
}

}  // namespace lin

size_t linear_bwd_workspace_bytes(const gdn_linear_problem& p) {
  return lin::tc_bwd_supported(p) ? lin::tc_bwd_bytes(p) : lin::bwd32_bytes(p);
}

gdn_status run_linear_bwd(const gdn_linear_problem& p, const void* q, const void* k, const void* v, const float* g,
                          float scale, const float* h0, const int32_t* cu, const void* dout, const float* dht,
                          void* dq, void* dk, void* dv, float* dg, float* dh0, void* ws, cudaStream_t s) {
  if (lin::tc_bwd_supported(p))
    return lin::tc_bwd(p, q, k, v, g, scale, h0, cu, dout, dht, dq, dk, dv, dg, dh0, ws, s);
  return lin::bwd32(p, q, k, v, g, scale, h0, cu, dout, dht, dq, dk, dv, dg, dh0, ws, lin::Drop{-1, 0}, s);
}

gdn_status run_linear_bwd_drop(const gdn_linear_problem& p, const void* q, const void* k, const void* v, const float* g,
                               float scale, const void* dout, void* dq, void* dk, void* dv, float* dg, void* ws,
                               int batch, unsigned warps, cudaStream_t s) {
  return lin::bwd32(p, q, k, v, g, scale, nullptr, nullptr, dout, nullptr, dq, dk, dv, dg, nullptr, ws,
                    lin::Drop{batch, warps}, s);
}

}  // namespace gdn
