// gdn_linear.cuh -- pieces shared by the kernels of decayed linear attention
//
//   S_t = e^{g_t} S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t            (S is [K][V], one per value head)
//
// in chunks of 64 tokens.  With b_i the sum of g over the chunk's tokens up to i, and S0 the state before the chunk,
//
//   o_i  = scale (e^{b_i} S0^T q_i + sum_{j <= i} e^{b_i - b_j} (q_i . k_j) v_j)
//   S_64 = e^{b_last} S0 + sum_j e^{b_last - b_j} k_j v_j^T
#pragma once

#include "gdn_internal.h"

namespace gdn {
namespace lin {

constexpr int kC = 64;   // tokens a chunk

// Chunks (or segments of chunks) of a batch.  Packed batches: tables that a launch before builds from cu_seqlens
// (nc < 0: malformed); equal lengths: arithmetic.
struct Pieces {
  const int32_t* seq;    // null: equal lengths
  const int32_t* tok0;
  const int32_t* len;
  const int32_t* first;  // [N + 1] first piece of each sequence
  const int32_t* nc;
  int T, per;            // equal lengths: tokens a sequence, pieces a sequence
  int size;              // tokens a piece
};

struct Piece {
  int seq, len;
  int64_t tok0;
  bool ok;
};

__device__ __forceinline__ Piece piece_of(const Pieces& t, int c) {
  Piece p;
  if (t.seq) {
    p.ok = c < *t.nc;
    p.seq = p.ok ? t.seq[c] : 0;
    p.tok0 = p.ok ? t.tok0[c] : 0;
    p.len = p.ok ? t.len[c] : 0;
  } else {
    p.ok = true;
    p.seq = c / t.per;
    const int at = (c - p.seq * t.per) * t.size;
    p.tok0 = (int64_t)p.seq * t.T + at;
    p.len = t.T - at < t.size ? t.T - at : t.size;
  }
  return p;
}

// Decays below e^-700 are 0 in fp32 (and -infinity among the sums would make differences of them NaN); NaN passes.
__device__ __forceinline__ double log_decay(float g) { return g < -700.f ? -700.0 : (double)g; }

// A sum of two floats that holds twice a float's bits.
struct Two {
  float h, l;
};

// e^{x.h + x.l} as a sum of two floats.  A state is multiplied by such a factor once a chunk (in the step once a token),
// with slow decays by nearly the same one for as long as its memory lasts, so that an error of the factor adds up.  Final
// states of 100000 tokens with decays of -1e-4 against 64 bits: 5.6e-6 with ex2.approx, 2.1e-6 with expf, 2.3e-7 with
// this; 20000 single steps with -1e-5: 5.1e-4 with expf, 2.5e-6.
// x = n ln 2 + r with n ln 2 in two parts (Cody and Waite's reduction), the first of 15 bits, so that its multiples are
// exact; e^r = 1 + r + r^2 / 2 + ... + r^8 / 8! for |r| <= ln 2 / 2, where the rest, below 2e-10, meets factors that are
// forgotten after a few chunks, as r's own rounding does; for small r all of it is exact to 2^-24 r^2.
__device__ __forceinline__ Two exp_two(Two x) {
  if (x.h < -150.f) return {0.f, 0.f};   // below fp32, above it (NaN goes on)
  if (x.h > 89.f) return {__int_as_float(0x7f800000), 0.f};
  constexpr double kLn2 = 0.693147180559945309;
  constexpr float kHigh = (float)((int)(kLn2 * 32768) / 32768.0), kRest = (float)(kLn2 - (int)(kLn2 * 32768) / 32768.0);
  const float n = rintf(x.h * (float)(1 / kLn2));
  const float t = fmaf(-n, kHigh, x.h), r = fmaf(-n, kRest, t), rl = fmaf(-n, kRest, t - r) + x.l;
  float q = 1.f / 40320;
  q = fmaf(q, r, 1.f / 5040);
  q = fmaf(q, r, 1.f / 720);
  q = fmaf(q, r, 1.f / 120);
  q = fmaf(q, r, 1.f / 24);
  q = fmaf(q, r, 1.f / 6);
  q = fmaf(q, r, 0.5f);
  const float s = 1.f + r, rest = (r - (s - 1.f)) + fmaf(q, r * r, fmaf(rl, r, rl));
  const float h = s + rest;
  const int half = (int)n / 2;   // 2^n in two factors: n down to -217
  const float a = __int_as_float((127 + half) << 23), b = __int_as_float((127 + (int)n - half) << 23);
  return {h * a * b, (rest - (h - s)) * a * b};
}

__device__ __forceinline__ Two times(Two a, Two b) {
  const float h = a.h * b.h, l = fmaf(a.h, b.h, -h) + fmaf(a.h, b.l, a.l * b.h), s = h + l;
  return {s, l - (s - h)};
}

// One warp: sums of the log decays of a chunk, as pairs of floats (hi + lo has the double's first 48 bits: the
// difference of two sums keeps its precision behind a strong decay).  Rows past len add nothing.
__device__ __forceinline__ void chunk_sums(const float* g, int64_t stride, int len, int lane, float* hi, float* lo) {
  const int r = 2 * lane;
  const double a = r < len ? log_decay(g[r * stride]) : 0.0;
  const double b = r + 1 < len ? log_decay(g[(r + 1) * stride]) : 0.0;
  double s = a + b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const double t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += t;
  }
  const double s0 = s - b;
  hi[r] = (float)s0, lo[r] = (float)(s0 - (double)(float)s0);
  hi[r + 1] = (float)s, lo[r + 1] = (float)(s - (double)(float)s);
}

}  // namespace lin

// Workspace layout and launches shared by the forward and the backward pass (gdn_linear.cu).
namespace lin {
size_t pieces_bytes(const gdn_linear_problem& p, int size);   // 0 for equal lengths
int pieces_max(const gdn_linear_problem& p, int size);
// Status word, then (packed batches) the tables of pieces of `size` tokens.
Pieces pieces_at(const gdn_linear_problem& p, int size, void* tables);
// Their launch (none for equal lengths); the one that begins a call clears the status word, with a launch less for packed
// batches.
cudaError_t launch_pieces(const gdn_linear_problem& p, int size, const int32_t* cu, void* tables, int32_t* status,
                          bool begin, cudaStream_t s);

// The tensor-core backward pass (gdn_linear_tc_bwd.cu).
bool tc_bwd_supported(const gdn_linear_problem& p);
size_t tc_bwd_bytes(const gdn_linear_problem& p);
gdn_status tc_bwd(const gdn_linear_problem& p, const void* q, const void* k, const void* v, const float* g, float scale,
                  const float* h0, const int32_t* cu, const void* dout, const float* dht, void* dq, void* dk, void* dv,
                  float* dg, float* dh0, void* ws, cudaStream_t s);

// The forward pass in bf16 (gdn_linear_tc.cu).
size_t tc_fwd_bytes(const gdn_linear_problem& p);
gdn_status tc_fwd(const gdn_linear_problem& p, const void* q, const void* k, const void* v, const float* g,
                  float scale, const float* h0, const int32_t* cu, void* o, float* ht, const int32_t* idx, int slots,
                  void* ws, cudaStream_t s);
}  // namespace lin

}  // namespace gdn
