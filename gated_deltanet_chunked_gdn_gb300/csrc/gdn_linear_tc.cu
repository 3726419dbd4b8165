// gdn_linear_tc.cu -- decayed linear attention of bf16 prompts and training batches on the tensor cores.
//
// A CTA walks a segment of a (sequence, value head, 128 columns of V) chain in chunks of 64 tokens.  Everything is
// transposed so that every tcgen05.mma has M = 128 (TMEM lane = value column e, or token):
//
//   [K;Q] K^T                -> lanes 64..127: Q K^T                              (M128 N64)
//   OQ^T = S^T Q^T           S^T: copy of the state before the chunk, two bf16 terms (M128 N64)
//   OP^T = V^T P^T           P = lower(scale e^{b_i - b_j} Q K^T), two bf16 terms (M128 N64)
//   U^T  = V''^T K           V'' = diag(e^{b_last - b_j}) V in three bf16 terms   (M128 N K)
//   o_i  = scale e^{b_i} OQ_i + OP_i,   S^T <- e^{b_last} S^T + U^T
//
// The state itself stays in fp32 registers (a thread holds K / 2 columns of one row of S^T), and what a chunk adds to
// it comes out of the tensor cores complete: V'' keeps all 24 bits of the weighted values (with two terms the final
// state was off by 2.4e-6, with three by 1e-7), and no sum longer than a chunk is left to the tensor cores'
// accumulation.  o reads a copy of the state in two bf16 terms, as its weights P are (with one term of either o was off by
// 2.3e-3 where that part made it up, with two by its own rounding, 1.7e-3).  The copy lies in tensor memory, where U^T was
// before the registers took it and will be again: in shared memory its second term has no room beside two CTAs, or takes
// that of P and o and makes their phases wait (4 x 8192 tokens of 32 heads: 499 us; so 470; one term 456).
// Two CTAs share an SM: one's loads and SIMT phases run under the other's products.
//
// Chains that do not fill the device are cut into segments of whole chunks: a launch before forms every segment's own
// contribution and decay (no q, no outputs), and the sums along the sequence give the states the segments start from.
//
// Rows past a sequence's end are zeroed in the K and V tiles (they may hold another sequence's values, NaN among them)
// and their weights are selected to zero; their outputs are not stored.
#include "gdn_linear_tc.cuh"

namespace gdn {
namespace lin {
namespace {

constexpr int kTcThreads = 256;

// Shared memory, byte offsets from its start.
template <int KD, int VD, bool FULL>
struct Map {
  static constexpr uint32_t KQ = 0;                               // k rows 0..63, q rows 64..127; 64 columns an atom column
  static constexpr uint32_t V = KQ + KD / 64 * 16384;
  static constexpr uint32_t P = V + VD / 64 * 8192;               // two terms
  static constexpr uint32_t X = P + (FULL ? 16384 : 0);           // the first two terms of V'' [j][e]
  static constexpr uint32_t OS = X + (uint32_t)VD * 64 * 2 * 2;   // the third, then o
  static constexpr uint32_t Tail = OS + VD / 64 * 8192;
  // rows 64..127 of a 64-row A tile are read (and ignored): they stay inside
  static constexpr uint32_t Misc = Tail < OS + 16384 ? OS + 16384 : Tail;
  static constexpr uint32_t kGam = 4 * kWalkDecays;
  static constexpr uint32_t Gam = Misc;   // a chunk's decays, as they lie in memory; without outputs two chunks'
  static constexpr uint32_t Bar = Misc + (FULL ? 1 : 2) * kGam, Flags = Bar + 64;
  static constexpr uint32_t Bytes = Flags + 64;
  static constexpr int Cols = KD + 128 <= 256 ? 256 : 512;        // TMEM: U^T and S^T's copy, Q K^T / OP^T, OQ^T
  static constexpr int Ctas = KD == 256 ? 1 : 2;
  static_assert(Ctas * (Bytes + 1024) <= 228 * 1024, "shared memory of an SM");
};

// A whole 32-byte sector a thread; a warp's lanes write 1 KB side by side.
__device__ __forceinline__ void store32(float* p, const float* v) {
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
               "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
               : "memory");
}

// V'' = diag(down) V in three terms (packed pairs throughout: a chunk's instructions bound the kernel): a thread takes
// 8 columns of a row at a time, units [u, end) in steps of n; zeros where down is 0.
template <int VD>
__device__ __forceinline__ void weigh_values(uint8_t* sm, uint32_t v, uint32_t x, uint32_t x2, uint32_t x3,
                                             const float* down, int u, int end, int n) {
  const float2 minus = make_float2(-1.f, -1.f);
#pragma unroll 2
  for (; u < end; u += n) {
    const int j = u / (VD / 8), c = u % (VD / 8);
    const uint32_t off = (c >> 3) * 8192 + sw128_chunk(j, c & 7);
    const uint4 w = *reinterpret_cast<const uint4*>(sm + v + off);
    const float2 f = make_float2(down[j], down[j]);
    const uint32_t in[4] = {w.x, w.y, w.z, w.w};
    uint32_t hi[4], lo[4], rest[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float2 a = __fmul2_rn(f, halves(in[i]));
      hi[i] = pack_bf16(a.x, a.y);
      a = __ffma2_rn(halves(hi[i]), minus, a);
      lo[i] = pack_bf16(a.x, a.y);
      a = __ffma2_rn(halves(lo[i]), minus, a);
      rest[i] = pack_bf16(a.x, a.y);
    }
    *reinterpret_cast<uint4*>(sm + x + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(sm + x2 + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
    *reinterpret_cast<uint4*>(sm + x3 + off) = make_uint4(rest[0], rest[1], rest[2], rest[3]);
  }
}

__device__ __forceinline__ Two add(Two a, float bh, float bl) {
  const float s = a.h + bh, v = s - a.h, e = ((a.h - (s - v)) + (bh - v)) + (a.l + bl);
  const float h = s + e;
  return {h, e - (h - s)};
}
__device__ __forceinline__ Two log2_units(Two a) {
  constexpr float kLow = (float)(1.4426950408889634 - (double)kLog2e);   // log2(e) = kLog2e + kLow
  const float h = a.h * kLog2e;
  return {h, fmaf(a.h, kLog2e, -h) + fmaf(a.l, kLog2e, a.h * kLow)};
}

// Decays of every chunk and head: log2(e) b_i, e^{b_last - b_j} (0 past the end), scale e^{b_i}, e^{b_last} in two floats
// and what the first lacks to 48 bits; the sums in pairs of floats (so that e^{b_last - b_j} keeps fp32 accuracy behind a
// strong decay, and differences of the sums do; with sums in double, fp64 being scarce here, 4 x 8192 tokens of 32 heads
// take 28 us, as they are 8).  o's weights take the first 24 bits: behind 64 tokens at the cut the difference of two sums
// is off by 2^-11, behind one by 2^-17, under the 2^-8 of o's own rounding.  A warp takes a chunk and head at a time.
// (Within the kernels below it was one warp's work for 2000 cycles a chunk, while the others waited.)  4 MB read, 17 MB
// written: the 8 us are latency.
__global__ void __launch_bounds__(256) decays_kernel(const float* __restrict__ g, int g_per_head, int Hv, Pieces pc,
                                                     float scale, float* __restrict__ out) {
  const Piece p = piece_of(pc, blockIdx.x);
  if (!p.ok) return;
  const int lane = threadIdx.x & 31, r = 2 * lane, chunks = (p.len + 63) / 64;
  for (int64_t w = (int64_t)blockIdx.y * 8 + (threadIdx.x >> 5); w < (int64_t)chunks * Hv; w += 8 * gridDim.y) {
    const int i = (int)(w / Hv), h = (int)(w % Hv), len = p.len - 64 * i;
    const float* gp = g + (g_per_head ? h : (p.tok0 + 64 * i + r) * Hv + h);
    const float ga = r < len ? gp[0] : 0.f, gb = r + 1 < len ? gp[g_per_head ? 0 : Hv] : 0.f;
    // e^-150 is 0 in fp32: stronger decays are cut there, and -infinity never meets itself in a difference
    const float a = ga < -150.f ? -150.f : ga, b = gb < -150.f ? -150.f : gb;
    Two s = add({a, 0.f}, b, 0.f);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const float th = __shfl_up_sync(0xffffffffu, s.h, o), tl = __shfl_up_sync(0xffffffffu, s.l, o);
      if (lane >= o) s = add(s, th, tl);
    }
    const float lh = __shfl_sync(0xffffffffu, s.h, 31), ll = __shfl_sync(0xffffffffu, s.l, 31);
    const Two s0 = add(s, -b, 0.f), x0 = log2_units(s0), x1 = log2_units(s);
    float* to = out + ((chunk_slot(p) + i) * Hv + h) * kDecays + r;
    *reinterpret_cast<float2*>(to) = make_float2(x0.h, x1.h);
    *reinterpret_cast<float2*>(to + kWalkDecays) = make_float2(x0.l, x1.l);
    if (lane == 0) {
      const Two whole = exp_two({lh, ll});
      *reinterpret_cast<float4*>(to + 192) = make_float4(whole.h, whole.l, 0.f, 0.f);
    }
    *reinterpret_cast<float2*>(to + 64) = make_float2(r < len ? expf((lh - s0.h) + (ll - s0.l)) : 0.f,
                                                      r + 1 < len ? expf((lh - s.h) + (ll - s.l)) : 0.f);
    *reinterpret_cast<float2*>(to + 128) = make_float2(scale * expf(s0.h + s0.l), scale * expf(s.h + s.l));
  }
}

// The walk over a segment's chunks.  ADJ: backwards, x = q, y = do, weights scale e^{b_i}: the adjoint of the state.
// 32 heads of 128: with outputs (kFull), 314 us for 4 x 8192 tokens and 86 for 8192 (3.4 TB/s of q, k, v and o); the
// segments' own (kOwn) before it 122 and 37; states for the backward pass (kEmit), 138 us for 4 x 4096 tokens (5.8 TB/s,
// 537 MB of them written: rows of S^T a lane took 152).  All but the last are bound by the chain of a chunk's phases:
// tensor pipe 28 to 33 %, HBM 30 %, the schedulers issue a third of the time with two CTAs an SM.  A third CTA has no
// room.
template <int KD, int VD, int MODE, bool ADJ>
__global__ void __launch_bounds__(kTcThreads, (Map<KD, VD, MODE == kFull>::Ctas))
    lin_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                  const TcParams prm) {
  constexpr bool FULL = MODE == kFull;
  using M = Map<KD, VD, FULL>;
  constexpr int KH = KD / 2;   // columns of S^T a thread holds
  extern __shared__ __align__(1024) uint8_t sm[];
  const uint32_t s4 = (smem_u32(sm) & 0x3FFFFu) >> 4;
  // Every barrier completes one phase a chunk, and every thread that waits for it does so once a chunk, in order.
  // Without outputs there is room for two chunks' loads, each with barriers of its own (bars 0, 1 and 2, 3).
  uint64_t* bars = reinterpret_cast<uint64_t*>(sm + M::Bar);
  uint64_t *bar_k = bars, *bar_v = bars + 1, *bar_qk = bars + 2, *bar_qs = bars + 3, *bar_pv = bars + 4,
           *bar_u = bars + 5, *bar_q = bars + 6;
  volatile uint32_t* flags = reinterpret_cast<volatile uint32_t*>(sm + M::Flags);   // [0] TMEM base
  volatile uint32_t* count = flags + 1;   // thread 0: phases begun on each barrier (what an abort has to wait for)

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int qd = warp & 3, hf = warp >> 2;   // TMEM lane quadrant, half of the columns
  const int row = 32 * qd + lane;
  const int slices = prm.V / VD;
  const int slice = blockIdx.x % slices, ch = blockIdx.x / slices;
  const int c = ch / prm.Hv, h = ch % prm.Hv, hq = h / (prm.Hv / prm.Hqk), e0 = slice * VD;
  const Piece p = piece_of(prm.pc, c);
  if (!p.ok) return;
  const int64_t seq0 = prm.varlen ? prm.cu[p.seq] : (int64_t)p.seq * prm.T;
  const int64_t seq1 = prm.varlen ? prm.cu[p.seq + 1] : seq0 + prm.T;
  const bool ends = ADJ ? p.tok0 == seq0 : p.tok0 + p.len == seq1;   // the walk's last segment of its sequence
  if (MODE == kOwn && ends) return;   // nobody starts behind it
  const int nchunks = (p.len + 63) / 64;
  auto chunk_at = [&](int i) { return ADJ ? nchunks - 1 - i : i; };

  if (tid == 0) {
#pragma unroll
    for (int i = 0; i < 7; ++i) mbar_init(bars + i, 1);
    mbar_fence_init();
#pragma unroll
    for (int i = 0; i < 7; ++i) count[i] = 0;
    prefetch_tmap(&tm_k);
    prefetch_tmap(&tm_v);
    if (FULL) {
      prefetch_tmap(&tm_q);
      prefetch_tmap(&tm_o);
    }
  }
  if (warp == 0) tmem_alloc(const_cast<uint32_t*>(flags), M::Cols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = flags[0];
  const uint32_t R_U = tmem, R_a = tmem + KD, R_b = tmem + KD + 64;
  const uint32_t lane_off = static_cast<uint32_t>(32 * qd) << 16;

  bool bad = false;   // one of this thread's waits ran out
  constexpr bool TWO = !FULL;
  auto buffer = [&](int i) { return TWO ? i & 1 : 0; };
  auto k_tile = [&](int i) { return M::KQ + 8192u * buffer(i); };   // the second in the place of Q
  auto v_tile = [&](int i) { return buffer(i) ? M::X : M::V; };     // the second in the place of the first term of V''
  auto load_bar = [&](int which, int i) { return bars + which + 2 * buffer(i); };
  auto load_no = [&](int i) { return TWO ? i >> 1 : i; };
  auto decays_of = [&](int i) { return reinterpret_cast<const float*>(sm + M::Gam + M::kGam * buffer(i)); };
  auto issue_k = [&](int i) {
    const int at = chunk_at(i), t = (int)(p.tok0 + 64 * at);
    uint64_t* bar = load_bar(0, i);
    count[2 * buffer(i)] = load_no(i) + 1;
    mbar_arrive_expect_tx(bar, KD / 64 * 8192 + M::kGam);
    bulk_load(sm + M::Gam + M::kGam * buffer(i), prm.decays + ((chunk_slot(p) + at) * prm.Hv + h) * kDecays, M::kGam, bar);
#pragma unroll
    for (int a = 0; a < KD / 64; ++a) tma_load_3d(sm + k_tile(i) + a * 16384, &tm_k, bar, 64 * a, hq, t);
  };
  auto issue_q = [&](int i) {
    const int t = (int)(p.tok0 + 64 * chunk_at(i));
    count[6] = i + 1;
    mbar_arrive_expect_tx(bar_q, KD / 64 * 8192);
#pragma unroll
    for (int a = 0; a < KD / 64; ++a) tma_load_3d(sm + M::KQ + a * 16384 + 8192, &tm_q, bar_q, 64 * a, hq, t);
  };
  auto issue_v = [&](int i) {
    const int t = (int)(p.tok0 + 64 * chunk_at(i));
    uint64_t* bar = load_bar(1, i);
    count[1 + 2 * buffer(i)] = load_no(i) + 1;
    mbar_arrive_expect_tx(bar, VD / 64 * 8192);
#pragma unroll
    for (int a = 0; a < VD / 64; ++a) tma_load_3d(sm + v_tile(i) + a * 8192, &tm_v, bar, e0 + 64 * a, h, t);
  };
  auto wait = [&](uint64_t* bar, int i) {
    if (!bad) bad = !mbar_wait(bar, i & 1, prm.status);
  };
  auto commit = [&](int b, int i) {
    mma_commit(bars + b);
    count[b] = i + 1;
  };
  if (tid == 0) {
    if (FULL) issue_q(0);
    issue_k(0);
    issue_v(0);
    if (TWO && nchunks > 1) {
      issue_k(1);
      issue_v(1);
    }
  }

  // S^T[e = row][d = hf KH + i]
  float S[KH];
  {
    const int64_t kv = (int64_t)KD * prm.V;
    const float* from = nullptr;
    if (MODE != kOwn) {
      // cut sequences start from a copy of h0, which another segment's CTA may be overwriting with the final state
      if (prm.start) from = prm.start + (int64_t)ch * kv;
      else if (prm.h0) from = prm.h0 + ((int64_t)p.seq * prm.Hv + h) * kv;
    }
    if (from && row < VD) {
      from += (int64_t)hf * KH * prm.V + e0 + row;
#pragma unroll
      for (int i = 0; i < KH; ++i) S[i] = from[(int64_t)i * prm.V];
    } else {
#pragma unroll
      for (int i = 0; i < KH; ++i) S[i] = 0.f;
    }
  }
  Two dec{1.f, 0.f}, total{1.f, 0.f};

#pragma unroll 1
  for (int i = 0; i < nchunks; ++i) {
    const int at = chunk_at(i), len = p.len - 64 * at < 64 ? p.len - 64 * at : 64;
    // ---- the state: what the chunk before added, and its bf16 copy
    if (i > 0) {
      wait(bar_u, i - 1);
      tc_fence_after();
      if (tid == 0 && !bad) {   // the tiles of the chunk before have been read
        if (FULL) issue_k(i);
        if (TWO && i + 1 < nchunks) {
          issue_k(i + 1);
          issue_v(i + 1);
        }
      }
#pragma unroll
      for (int b = 0; b < KH; b += 32) {
        float u[32];
        tmem_ld32(R_U + lane_off + hf * KH + b, u);
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const float2 y = make_float2(S[b + j], S[b + j + 1]);
          const float2 x = __ffma2_rn(make_float2(dec.h, dec.h), y,
                                      __ffma2_rn(make_float2(dec.l, dec.l), y, make_float2(u[j], u[j + 1])));
          S[b + j] = x.x, S[b + j + 1] = x.y;
        }
      }
    }
    if (FULL) {
      // in the place of U^T, whose columns of this half this thread has just read: KH / 2 columns for the first terms,
      // then as many for the second
      if (tid == 0) bulk_wait_read();   // the o staging has been read: its place takes a term of V''
#pragma unroll
      for (int b = 0; b < KH; b += 32) {
        uint32_t hi[16], lo[16];
#pragma unroll
        for (int u = 0; u < 16; ++u) split2(S[b + 2 * u], S[b + 2 * u + 1], hi[u], lo[u]);
        tmem_st16(R_U + lane_off + hf * KH + b / 2, hi);
        tmem_st16(R_U + lane_off + hf * KH + KH / 2 + b / 2, lo);
      }
      tmem_wait_st();
    }
    if (MODE == kEmit && row < VD) {
      float* to = prm.emit + ((chunk_slot(p) + at) * prm.Hv + h) * (int64_t)(KD * VD) + hf * KH * VD + row * 8;
#pragma unroll
      for (int b = 0; b < KH; b += 8) store32(to + b * VD, S + b);
    }
    if (len < 64) {
      wait(load_bar(0, i), load_no(i));
      wait(load_bar(1, i), load_no(i));
      zero_rows(sm + k_tile(i), KD / 64, 16384, len, tid, kTcThreads);
      zero_rows(sm + v_tile(i), VD / 64, 8192, len, tid, kTcThreads);
    }
    if (FULL || len < 64) {
      fence_proxy_async();
      tc_fence_before();
      if (__syncthreads_or(bad)) break;
      tc_fence_after();
    }
    const float *gam = decays_of(i), *down = gam + 64, *up = gam + 128;

    if (FULL && warp == 6 && lane == 0 && i + 1 < nchunks) {   // the next chunk's tiles on their way to L2
      const int t = (int)(p.tok0 + 64 * chunk_at(i + 1));
#pragma unroll
      for (int a = 0; a < KD / 64; ++a) tma_prefetch_3d(&tm_k, 64 * a, hq, t);
#pragma unroll
      for (int a = 0; a < VD / 64; ++a) tma_prefetch_3d(&tm_v, e0 + 64 * a, h, t);
    }
    if (FULL) {
      if (tid == 0) {
        const uint32_t id = idesc_bf16(128, 64, 0, 0, 0);
        wait(bar_q, i);
        wait(bar_k, i);
        if (!bad) {
          tc_fence_after();
#pragma unroll
          for (int s = 0; s < KD / 16; ++s) {
            const uint32_t a = M::KQ + (s >> 2) * 16384 + (s & 3) * 32;
            mma_bf16(R_a, dsw(s4, a, 16), dsw(s4, a, 16), id, s > 0);
          }
          commit(2, i);
#pragma unroll
          for (int s = 0; s < 2 * (KD / 16); ++s) {   // the second terms first
            const int d = s % (KD / 16), half = 16 * d / KH;
            const uint32_t a = R_U + half * KH + (16 * d - half * KH) / 2 + (s < KD / 16 ? KH / 2 : 0);
            mma_bf16_ta(R_b, a, dsw(s4, M::KQ + 8192 + (d >> 2) * 16384 + (d & 3) * 32, 16), id, s > 0);
          }
          commit(3, i);
        }
      }
      __syncwarp();
      if (qd >= 2) {
        // P row i2, columns 32 hf ..
        wait(bar_k, i);   // every thread that reads the decays waits for them
        wait(bar_qk, i);
        tc_fence_after();
        float v[32];
        const int i2 = row - 64;
        if (qd == 2 && hf == 1) {   // above the diagonal
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = 0.f;
        } else {
          tmem_ld32(R_a + lane_off + 32 * hf, v);
          const float gi = gam[i2];
#pragma unroll
          for (int j4 = 0; j4 < 8; ++j4) {
            const float4 g4 = *reinterpret_cast<const float4*>(gam + 32 * hf + 4 * j4);
            const float gj[4] = {g4.x, g4.y, g4.z, g4.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const int j = 4 * j4 + u;
              // above the diagonal cleared by its bits: a branch an element would cost ten times the products
              const uint32_t keep = 32 * hf + j <= i2 ? 0xffffffffu : 0u;
              v[j] = __uint_as_float(__float_as_uint(prm.scale * ex2_fast(gi - gj[u]) * v[j]) & keep);
            }
          }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) split2(v[8 * q + 2 * u], v[8 * q + 2 * u + 1], hi[u], lo[u]);
          const uint32_t off = sw128_chunk(i2, 4 * hf + q);
          *reinterpret_cast<uint4*>(sm + M::P + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(sm + M::P + 8192 + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
      }
      // V'': the warps without weights begin with five eighths of it, the one whose weights are all zero takes as
      // much as the three others behind theirs
      wait(bar_k, i);
      wait(bar_v, i);
      constexpr int n = 64 * (VD / 8);
      constexpr uint32_t x2 = M::X + VD / 64 * 8192;
      if (qd < 2) weigh_values<VD>(sm, M::V, M::X, x2, M::OS, down, 64 * hf + row, n * 5 / 8, 128);
      else if (warp == 6) weigh_values<VD>(sm, M::V, M::X, x2, M::OS, down, n * 13 / 16 + lane, n, 32);
      else
        weigh_values<VD>(sm, M::V, M::X, x2, M::OS, down, n * 5 / 8 + 32 * (warp == 7 ? 2 : warp - 2) + lane, n * 13 / 16,
                         96);
    } else {
      wait(load_bar(0, i), load_no(i));
      wait(load_bar(1, i), load_no(i));
      // the first term in the place of V
      weigh_values<VD>(sm, v_tile(i), v_tile(i), M::X + VD / 64 * 8192, M::OS, ADJ ? up : down, tid, 64 * (VD / 8),
                       kTcThreads);
    }
    dec = {gam[192], gam[193]};   // before the barrier behind which the next chunk's decays may come in
    if (MODE == kOwn) total = times(total, dec);
    fence_proxy_async();
    tc_fence_before();
    if (__syncthreads_or(bad)) break;
    tc_fence_after();
    if (FULL && tid == 0) {   // U^T takes the place of S^T's copy (products of different shapes need not end in order)
      wait(bar_qs, i);
      tc_fence_after();
    }
    if (tid == 0 && !bad) {
      const uint32_t idu = idesc_bf16(128, KD, 1, 1, 0);
      // the third term first: its place takes o, which is written once V^T P^T, issued behind it, is complete
#pragma unroll
      for (int s = 0; s < 4; ++s)
        mma_bf16(R_U, dsw(s4, M::OS + s * 2048, 8192), dsw(s4, k_tile(i) + s * 2048, 16384), idu, s > 0);
      if (FULL) {
        const uint32_t id = idesc_bf16(128, 64, 1, 0, 0);
#pragma unroll
        for (int s = 0; s < 8; ++s)
          mma_bf16(R_a, dsw(s4, M::V + (s & 3) * 2048, 8192),
                   dsw(s4, M::P + (s >> 2) * 8192 + (s & 3) * 32, 16), id, s > 0);
        commit(4, i);
      }
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const uint32_t term = s >> 2 ? M::X + VD / 64 * 8192 : (FULL ? M::X : v_tile(i));
        mma_bf16(R_U, dsw(s4, term + (s & 3) * 2048, 8192), dsw(s4, k_tile(i) + (s & 3) * 2048, 16384), idu, 1);
      }
      commit(5, i);
    }
    __syncwarp();
    if (FULL) {
      // o_i = up_i OQ_i + OP_i: this thread has column e0 + row of o for 32 rows; neighbouring lanes exchange values
      // so that each writes bf16 pairs
      const int ecol = (row & 63) & ~1;
      const bool odd = lane & 1;
      uint8_t* lbase = sm + M::OS + (row >> 6) * 8192 + (odd ? 128 : 0) + (ecol & 7) * 2;
      const uint32_t xsw = (static_cast<uint32_t>((ecol >> 3) ^ (odd ? 1 : 0))) << 4;
      float oq[32];
      wait(bar_qs, i);
      tc_fence_after();
      tmem_ld32(R_b + lane_off + 32 * hf, oq);
      wait(bar_pv, i);
      tc_fence_after();
      if (tid == 0 && i + 1 < nchunks && !bad) {
        issue_q(i + 1);
        issue_v(i + 1);
      }
      if (row < VD) {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          float b[16];
          const uint32_t col = 32 * hf + 16 * q;
          tmem_ld16(R_a + lane_off + col, b);
          uint8_t* qb = lbase + col * 128;
#pragma unroll
          for (int pp = 0; pp < 8; ++pp) {
            const float2 f = *reinterpret_cast<const float2*>(up + col + 2 * pp);
            const float2 v = __ffma2_rn(f, make_float2(oq[16 * q + 2 * pp], oq[16 * q + 2 * pp + 1]),
                                        make_float2(b[2 * pp], b[2 * pp + 1]));
            const float other = __shfl_xor_sync(0xffffffffu, odd ? v.x : v.y, 1);
            const uint32_t word = odd ? pack_bf16(other, v.y) : pack_bf16(v.x, other);
            const uint32_t off = (2 * pp) * 128 + (xsw ^ (static_cast<uint32_t>((2 * pp) & 7) << 4));
            *reinterpret_cast<uint32_t*>(qb + off) = word;
          }
        }
      }
      fence_proxy_async();
      tc_fence_before();
      __syncthreads();
      const int64_t t0 = p.tok0 + 64 * (int64_t)at;
      if (len == 64) {
        if (tid == 0) {
#pragma unroll
          for (int a = 0; a < VD / 64; ++a) tma_store_3d(&tm_o, sm + M::OS + a * 8192, e0 + 64 * a, h, (int)t0);
          bulk_commit();
        }
      } else {
        for (int u = tid; u < len * (VD / 8); u += kTcThreads) {
          const int r = u / (VD / 8), q = u % (VD / 8);
          const uint4 val = *reinterpret_cast<const uint4*>(sm + M::OS + (q >> 3) * 8192 + sw128_chunk(r, q & 7));
          *reinterpret_cast<uint4*>(prm.o + ((t0 + r) * prm.Hv + h) * (int64_t)prm.V + e0 + q * 8) = val;
        }
      }
    }
  }

  // what the last chunk added; after an abort (every thread left the loop at the same barrier) nothing is written
  if (!__syncthreads_or(bad)) {
    wait(bar_u, nchunks - 1);
    tc_fence_after();
#pragma unroll
    for (int b = 0; b < KH; b += 32) {
      float u[32];
      tmem_ld32(R_U + lane_off + hf * KH + b, u);
#pragma unroll
      for (int j = 0; j < 32; ++j) S[b + j] = fmaf(dec.h, S[b + j], fmaf(dec.l, S[b + j], u[j]));
    }
    float* to = nullptr;
    const int64_t kv = (int64_t)KD * prm.V;
    if (MODE == kOwn) {
      to = prm.own + (int64_t)ch * kv;
      if (tid == 0 && slice == 0) prm.total[ch] = total;
    } else if (ends && prm.ht) {
      int64_t at = p.seq;
      if (prm.idx) {
        at = prm.idx[p.seq];
        if (at < 0 || at >= prm.slots) at = -1;
      }
      if (at >= 0) to = prm.ht + (at * prm.Hv + h) * kv;
    }
    if (to && row < VD && !bad) {
      to += (int64_t)hf * KH * prm.V + e0 + row;
#pragma unroll
      for (int i = 0; i < KH; ++i) to[(int64_t)i * prm.V] = S[i];
    }
  }
  if (tid == 0) bulk_wait_read();
  if (__syncthreads_or(bad) && tid == 0) {
    // abort: loads and products in flight finish (bounded) before their memory is released
    for (int b = 0; b < 7; ++b)
      if (count[b] > 0) mbar_wait(bars + b, (count[b] - 1) & 1, prm.status, 100000000ull);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) tmem_dealloc(tmem, M::Cols);
}

// Final states of sequences without tokens: the initial ones.
__global__ void __launch_bounds__(256) empty_kernel(const int32_t* __restrict__ cu, const int32_t* __restrict__ nc,
                                                    int Hv, int64_t kv, const float* __restrict__ h0,
                                                    float* __restrict__ ht, const int32_t* __restrict__ idx,
                                                    int slots) {
  const int n = blockIdx.x;
  if (*nc < 0 || cu[n] != cu[n + 1]) return;
  int64_t to = n;
  if (idx) {
    to = idx[n];
    if (to < 0 || to >= slots) return;
  }
  const int64_t size = Hv * kv;
  for (int64_t i = 4 * (int64_t)threadIdx.x; i < size; i += 1024)
    *reinterpret_cast<float4*>(ht + to * size + i) =
        h0 ? load4(h0 + n * size + i) : make_float4(0.f, 0.f, 0.f, 0.f);
}

int slice_width(const gdn_linear_problem& p) { return p.V >= 128 ? 128 : 64; }

struct Maps {
  CUtensorMap q, x, y, o;
};

template <int KD, int VD, int MODE, bool ADJ>
gdn_status launch_one(unsigned grid, const Maps& m, const TcParams& prm, cudaStream_t s) {
  auto kern = lin_tc_kernel<KD, VD, MODE, ADJ>;
  constexpr int bytes = (int)Map<KD, VD, MODE == kFull>::Bytes;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return GDN_ERR_CUDA;
  kern<<<grid, kTcThreads, bytes, s>>>(m.q, m.x, m.y, m.o, prm);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

template <int KD, int VD>
gdn_status launch_dims(int mode, bool adj, unsigned grid, const Maps& m, const TcParams& prm, cudaStream_t s) {
  if (mode == kFull) return launch_one<KD, VD, kFull, false>(grid, m, prm, s);
  if (mode == kOwn && !adj) return launch_one<KD, VD, kOwn, false>(grid, m, prm, s);
  if constexpr (KD <= 128) {   // the head dims of the tensor-core backward pass
    if (mode == kOwn) return launch_one<KD, VD, kOwn, true>(grid, m, prm, s);
    if (adj) return launch_one<KD, VD, kEmit, true>(grid, m, prm, s);
    return launch_one<KD, VD, kEmit, false>(grid, m, prm, s);
  }
  return GDN_ERR_UNSUPPORTED;
}

}  // namespace

// Tokens a segment.  Equal lengths: the number of segments a sequence that costs least in chunks on the busiest CTA
// slot: full walks in rounds of the slots' segments (and half as much for the segments' own contributions, where there
// is more than one), about two chunks for a segment's start and end.  32 heads, K = V = 128: 8192 tokens take 9
// segments, 4 x 8192 take 7.  Packed batches, whose lengths the host does not know: half of a slot's even share.
int segment_tokens(const gdn_linear_problem& p) {
  const int64_t slots = (p.K == 256 ? 1 : 2) * (int64_t)sm_count();
  const int64_t heads = (int64_t)p.Hv * (p.V / slice_width(p));
  const int64_t whole = ceil_div(p.T > 0 ? p.T : 1, 64);
  if (p.varlen) {
    const int64_t m = ceil_div((p.T / 64 + p.N) * heads, 2 * slots);
    return (int)(64 * (m < 4 ? (whole < 4 ? whole : 4) : (m > whole ? whole : m)));
  }
  const int64_t chains = p.N * heads;
  int64_t best = whole, least = ceil_div(chains, slots) * (whole + 2) * 2;
  for (int64_t n = 2; n <= 2 * slots && 4 * n <= whole + 3; n += 1 + n / 16) {
    const int64_t m = ceil_div(whole, n), cut = ceil_div(whole, m);
    const int64_t cost = (m + 2) * (2 * ceil_div(chains * cut, slots) + ceil_div(chains * (cut - 1), slots));
    if (cost < least) least = cost, best = m;
  }
  return (int)(64 * best);
}

size_t decays_bytes(const gdn_linear_problem& p) {
  return align_up(4 * kDecays * (size_t)((int64_t)p.B * p.T / 64 + p.N + 1) * p.Hv);
}

gdn_status launch_decays(const gdn_linear_problem& p, const Pieces& pc, int size, const float* g, float scale,
                         float* decays, cudaStream_t s) {
  const int64_t share = ceil_div((int64_t)(size / 64) * p.Hv, 8);   // CTAs a piece
  decays_kernel<<<dim3(pieces_max(p, size), (unsigned)(share < 64 ? share : 64)), 256, 0, s>>>(g, p.g_per_head, p.Hv,
                                                                                              pc, scale, decays);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status launch_empty(const gdn_linear_problem& p, const Pieces& pc, const int32_t* cu, const float* h0, float* ht,
                        const int32_t* idx, int slots, cudaStream_t s) {
  if (!p.varlen || !ht) return GDN_OK;
  empty_kernel<<<p.N, 256, 0, s>>>(cu, pc.nc, p.Hv, (int64_t)p.K * p.V, h0, ht, idx, slots);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

TcParams tc_params(const gdn_linear_problem& p, const Pieces& pc, const int32_t* cu, float scale, const float* decays,
                   int32_t* status) {
  TcParams prm;
  memset(&prm, 0, sizeof(prm));
  prm.pc = pc;
  prm.decays = decays;
  prm.status = status;
  prm.cu = cu;
  prm.Hqk = p.Hqk;
  prm.Hv = p.Hv;
  prm.V = p.V;
  prm.varlen = p.varlen;
  prm.T = p.T;
  prm.scale = scale;
  return prm;
}

gdn_status launch_walk(const gdn_linear_problem& p, int mode, bool adj, const void* q, const void* x, int64_t ld_x,
                       const void* y, int64_t ld_y, void* o, TcParams prm, int size, cudaStream_t s) {
  const int64_t tokens = (int64_t)p.B * p.T;
  Maps m;
  memset(&m, 0, sizeof(m));
  const uint32_t box[3] = {64, 1, 64};
  const uint64_t kd[3] = {(uint64_t)p.K, (uint64_t)p.Hqk, (uint64_t)tokens};
  const uint64_t vd[3] = {(uint64_t)p.V, (uint64_t)p.Hv, (uint64_t)tokens};
  const uint64_t sx[2] = {(uint64_t)p.K * 2, (uint64_t)ld_x * 2}, sy[2] = {(uint64_t)p.V * 2, (uint64_t)ld_y * 2};
  if (!make_tmap_bf16(&m.x, x, 3, kd, sx, box) || !make_tmap_bf16(&m.y, y, 3, vd, sy, box)) return GDN_ERR_CUDA;
  if (mode == kFull) {
    const uint64_t sq[2] = {(uint64_t)p.K * 2, (uint64_t)p.ld_q * 2};
    const uint64_t so[2] = {(uint64_t)p.V * 2, (uint64_t)p.Hv * p.V * 2};
    if (!make_tmap_bf16(&m.q, q, 3, kd, sq, box) || !make_tmap_bf16(&m.o, o, 3, vd, so, box)) return GDN_ERR_CUDA;
    prm.o = static_cast<__nv_bfloat16*>(o);
  }
  const unsigned grid = (unsigned)((int64_t)pieces_max(p, size) * p.Hv * (p.V / slice_width(p)));
  if (p.V == 64) {
    if (p.K == 64) return launch_dims<64, 64>(mode, adj, grid, m, prm, s);
    if (p.K == 128) return launch_dims<128, 64>(mode, adj, grid, m, prm, s);
    return launch_dims<256, 64>(mode, adj, grid, m, prm, s);
  }
  if (p.K == 64) return launch_dims<64, 128>(mode, adj, grid, m, prm, s);
  if (p.K == 128) return launch_dims<128, 128>(mode, adj, grid, m, prm, s);
  return launch_dims<256, 128>(mode, adj, grid, m, prm, s);
}

// [status][tables][decays][the segments' decays: segments x Hv][states: segments x Hv x K x V]
size_t tc_fwd_bytes(const gdn_linear_problem& p) {
  const int seg = segment_tokens(p);
  const size_t cells = seg < p.T ? (size_t)pieces_max(p, seg) * p.Hv : 0;
  return kAlign + pieces_bytes(p, seg) + decays_bytes(p) + align_up(sizeof(Two) * cells) + 4 * cells * p.K * p.V;
}

gdn_status tc_fwd(const gdn_linear_problem& p, const void* q, const void* k, const void* v, const float* g,
                  float scale, const float* h0, const int32_t* cu, void* o, float* ht, const int32_t* idx, int slots,
                  void* ws, cudaStream_t s) {
  uint8_t* at = static_cast<uint8_t*>(ws);
  int32_t* status = reinterpret_cast<int32_t*>(at);
  const int seg = segment_tokens(p);
  void* tables = at + kAlign;
  if (launch_pieces(p, seg, cu, tables, status, true, s) != cudaSuccess) return GDN_ERR_CUDA;
  const Pieces pc = pieces_at(p, seg, tables);
  gdn_status st = launch_empty(p, pc, cu, h0, ht, idx, slots, s);
  if (st != GDN_OK || (int64_t)p.B * p.T == 0) return st;
  float* decays = reinterpret_cast<float*>(at + kAlign + pieces_bytes(p, seg));
  st = launch_decays(p, pc, seg, g, scale, decays, s);
  TcParams prm = tc_params(p, pc, cu, scale, decays, status);
  prm.h0 = h0;
  if (st == GDN_OK && seg < p.T) {
    prm.total = reinterpret_cast<Two*>(decays + decays_bytes(p) / 4);
    prm.own = decays + (decays_bytes(p) + align_up(sizeof(Two) * (size_t)pieces_max(p, seg) * p.Hv)) / 4;
    st = launch_walk(p, kOwn, false, nullptr, k, p.ld_k, v, p.ld_v, nullptr, prm, seg, s);
    if (st == GDN_OK) st = launch_sums(shape_of(p), pc, p.N, prm.total, Sum{h0, prm.own, nullptr, nullptr, 0, false}, s);
    prm.start = prm.own;
  }
  if (st != GDN_OK) return st;
  prm.ht = ht;
  prm.idx = idx;
  prm.slots = slots;
  return launch_walk(p, kFull, false, q, k, p.ld_k, v, p.ld_v, o, prm, seg, s);
}

}  // namespace lin
}  // namespace gdn
