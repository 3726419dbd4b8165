// gdn_scan.cuh -- pieces shared by the selective state space scan's forward
// (gdn_scan.cu) and backward (gdn_scan_bwd.cu): arguments, the cut of the
// sequences into segments, the layout of a warp's channels and states, and the
// scalar functions.
//
// The scan, for a channel d of group g(d) and a state n:
//     dt_t   = softplus(delta_t + dt_bias)     (or delta_t + dt_bias)
//     h_t[n] = e^{dt_t A[n]} h_{t-1}[n] + dt_t x_t B_t[n]
//     y_t    = (sum_n C_t[n] h_t[n] + D x_t) silu(z_t)
//
// Layout.  A warp owns kCpw(RL) = 2 * 32 / RL channels of one group and all of
// their states: RL lanes stand side by side over the states of a channel pair
// (four states each, S <= 4 RL), the 32 / RL lanes of one state quarter over the
// channel pairs, so a lane keeps 2 x 4 states in registers.  Two channels a
// lane: B_t and C_t are read from shared memory as one 16-byte vector each
// (two cycles of the SM's shared-memory port a warp, measured) and serve eight
// state updates, which cost eight cycles of the ex2 unit and of the FMA pipe;
// with one channel a lane the reads would take as long as the arithmetic.  The
// lanes of a state quarter are adjacent: a 16-byte read costs two cycles when
// neighbouring lanes read one address and four when they do not.
#pragma once

#include <cfloat>
#include <type_traits>

#include "gdn_internal.h"
#include "gdn_sm100.cuh"

namespace gdn {
namespace scan {

constexpr int kTileMax = 16;   // tokens a tile

struct Args {
  const void *x, *dl, *z, *B, *C;
  const float *A, *Dp, *bias, *h0;
  const int32_t* cu;
  int bx, bd, bz, bb, bc;            // bytes from one token's row to the next
  int64_t T;                         // tokens of a sequence, or of the packed batch
  int N, D, S, G, Dg;                // Dg = D / G channels a group
  int cbg;                           // warp channel blocks a group
  int softplus;
  bool vin;     // pairs of neighbouring channels of x, delta and z can be loaded at once
  bool vbc;     // vectors of B and C (RowVec) can be loaded at once
  int rows;     // Rows
  // segments
  int nseg;                 // of a sequence (equal lengths)
  int seglen;               // tokens, a multiple of kTileMax
  const int32_t* seg0;      // packed: [N] first segment of every sequence, the number of segments (< 0:
                            // malformed), the number of sequences with several, and which they are
  float* hseg;              // [segments][D][S]: local end states, then the states the segments start from
  float* dtsum;             // [segments][D]: sum of dt over the segment
  // forward outputs
  void* y;
  float* ht;                // [N][D][S], or a pool of `slots` such rows
  const int32_t* slot;      // row of every sequence's final state (outside the pool: not kept), or null (row n)
  int slots;
  bool vy;
};

struct Unit {
  int n;
  int64_t tok0;
  int len;
  bool first, last;   // of its sequence
};

// Segment u of the batch; false past the last one (or for malformed cu_seqlens).
__device__ __forceinline__ bool unit_of(const Args& a, int64_t u, Unit& r) {
  int64_t s, e, j;
  if (a.cu) {
    if (u >= a.seg0[a.N]) return false;
    int lo = 0, hi = a.N - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.seg0[mid] <= u) lo = mid; else hi = mid - 1;
    }
    r.n = lo;
    j = u - a.seg0[lo];
    s = a.cu[lo];
    e = a.cu[lo + 1];
  } else {
    r.n = (int)(u / a.nseg);
    j = u % a.nseg;
    s = (int64_t)r.n * a.T;
    e = s + a.T;
  }
  r.tok0 = s + j * a.seglen;
  const int64_t left = e - r.tok0;
  r.len = (int)(left < a.seglen ? left : a.seglen);
  r.first = j == 0;
  r.last = left <= a.seglen;
  return true;
}

// Four consecutive elements as loaded, entries at or past n as 0.
template <typename T> struct Raw4;
template <> struct Raw4<__nv_bfloat16> {
  uint2 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, int n, bool vec) {
    if (vec) {
      v = __ldg(reinterpret_cast<const uint2*>(p));
    } else {
      uint32_t e[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = i < n ? __ldg(reinterpret_cast<const uint16_t*>(p) + i) : 0u;
      v = make_uint2(e[0] | (e[1] << 16), e[2] | (e[3] << 16));
    }
  }
  __device__ __forceinline__ float2 lo() const { return make_float2(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xffff0000u)); }
  __device__ __forceinline__ float2 hi() const { return make_float2(__uint_as_float(v.y << 16), __uint_as_float(v.y & 0xffff0000u)); }
};
template <> struct Raw4<float> {
  float4 v;
  __device__ __forceinline__ void load(const float* p, int n, bool vec) {
    if (vec) {
      v = __ldg(reinterpret_cast<const float4*>(p));
    } else {
      v.x = 0 < n ? __ldg(p) : 0.f, v.y = 1 < n ? __ldg(p + 1) : 0.f;
      v.z = 2 < n ? __ldg(p + 2) : 0.f, v.w = 3 < n ? __ldg(p + 3) : 0.f;
    }
  }
  __device__ __forceinline__ float2 lo() const { return make_float2(v.x, v.y); }
  __device__ __forceinline__ float2 hi() const { return make_float2(v.z, v.w); }
};

// Row t of a tensor whose rows are `stride` bytes apart (one multiply-add).
template <typename T>
__device__ __forceinline__ const T* row(const T* p, int t, int stride) {
  return reinterpret_cast<const T*>(reinterpret_cast<const char*>(p) + (int64_t)t * stride);
}

// Two neighbouring elements as loaded (converted when they are used, so that
// the loads of the next tile stay in flight).
template <typename T> struct Raw2;
template <> struct Raw2<__nv_bfloat16> {
  uint32_t v;
  __device__ __forceinline__ void zero() { v = 0u; }
  __device__ __forceinline__ void load_shared(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint32_t*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint32_t*>(p) = v; }
  __device__ __forceinline__ void load(const __nv_bfloat16* p, bool vec, bool ok0, bool ok1) {
    if (vec && ok1) {
      v = __ldg(reinterpret_cast<const uint32_t*>(p));
    } else {
      const uint32_t lo = ok0 ? __ldg(reinterpret_cast<const uint16_t*>(p)) : 0u;
      const uint32_t hi = ok1 ? __ldg(reinterpret_cast<const uint16_t*>(p) + 1) : 0u;
      v = lo | (hi << 16);
    }
  }
  __device__ __forceinline__ float2 f() const {
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
  }
};
template <> struct Raw2<float> {
  float2 v;
  __device__ __forceinline__ void zero() { v = make_float2(0.f, 0.f); }
  __device__ __forceinline__ void load_shared(const float* p) { v = *reinterpret_cast<const float2*>(p); }
  __device__ __forceinline__ void store(float* p) const { *reinterpret_cast<float2*>(p) = v; }
  __device__ __forceinline__ void load(const float* p, bool vec, bool ok0, bool ok1) {
    if (vec && ok1) {
      v = __ldg(reinterpret_cast<const float2*>(p));
    } else {
      v.x = ok0 ? __ldg(p) : 0.f;
      v.y = ok1 ? __ldg(p + 1) : 0.f;
    }
  }
  __device__ __forceinline__ float2 f() const { return v; }
};

// A tile's rows of B (or C, padded to SP states) move in vectors of VE elements,
// 16 bytes where a row has as many; NV of them.
template <typename T, int RL>
struct RowVec {
  static constexpr int SP = 4 * RL, VE = 16 / (int)sizeof(T) < SP ? 16 / (int)sizeof(T) : SP;
  static constexpr int NV = (RL >= 4 ? 16 : 4 * RL) * SP / VE;
};
// VE elements of a row from element n on (of `len`), one by one when they cannot be
// loaded at once.
template <typename T, int VE>
__device__ __forceinline__ uint4 load_row16(const T* p, int n, int len, bool vec) {
  if (VE * sizeof(T) == 16 && vec) return __ldg(reinterpret_cast<const uint4*>(p + n));
  uint32_t v[4] = {0u, 0u, 0u, 0u};
#pragma unroll
  for (int i = 0; i < VE; ++i)
    if (n + i < len) {
      if constexpr (sizeof(T) == 4) v[i] = __float_as_uint(__ldg(p + n + i));
      else v[i / 2] |= (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(p) + n + i) << (16 * (i % 2));
    }
  return make_uint4(v[0], v[1], v[2], v[3]);
}
// .. to shared memory as floats.
template <typename T, int VE>
__device__ __forceinline__ void put_row16(float* o, uint4 q) {
  float4* p = reinterpret_cast<float4*>(o);
  if constexpr (sizeof(T) == 4) {
    p[0] = make_float4(__uint_as_float(q.x), __uint_as_float(q.y), __uint_as_float(q.z), __uint_as_float(q.w));
  } else {
    p[0] = make_float4(__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xffff0000u), __uint_as_float(q.y << 16),
                       __uint_as_float(q.y & 0xffff0000u));
    if (VE == 8) p[1] = make_float4(__uint_as_float(q.z << 16), __uint_as_float(q.z & 0xffff0000u), __uint_as_float(q.w << 16),
                       __uint_as_float(q.w & 0xffff0000u));
  }
}

// BYTES (8 or 16) of a register vector to and from shared memory.
template <int BYTES>
__device__ __forceinline__ void copy_vec(void* p, uint4 q) {
  if constexpr (BYTES == 16) *reinterpret_cast<uint4*>(p) = q;
  else *reinterpret_cast<uint2*>(p) = make_uint2(q.x, q.y);
}
template <int BYTES>
__device__ __forceinline__ uint4 get_vec(const void* p) {
  if constexpr (BYTES == 16) return *reinterpret_cast<const uint4*>(p);
  const uint2 q = *reinterpret_cast<const uint2*>(p);
  return make_uint4(q.x, q.y, 0u, 0u);
}

// Asynchronous copy of CH (4, 8 or 16) bytes to shared memory; only the first `bytes`
// of them are read, the rest become zero.
template <int CH>
__device__ __forceinline__ void copy_async(void* dst, const void* src, int bytes) {
  if constexpr (CH == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm100::smem_u32(dst)), "l"(src), "r"(bytes) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(sm100::smem_u32(dst)), "l"(src), "r"(bytes), "n"(CH)
                 : "memory");
}

// How rows come to shared memory: copies of 16 bytes (or a shorter row), of 4 bytes,
// or loads through registers where not even pairs of bf16 are aligned.
enum Rows { kRegs = 0, kWide = 1, kNarrow = 2 };
template <int ROWS, int ROW>
constexpr int chunk() { return ROWS == kNarrow ? 4 : ROW < 16 ? ROW : 16; }
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

template <typename T>
__device__ __forceinline__ void store2(T* p, float2 v) {
  if constexpr (std::is_same<T, float>::value) *reinterpret_cast<float2*>(p) = v;
  else *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
}
template <typename T>
__device__ __forceinline__ void store2(T* p, float2 v, bool vec, bool ok0, bool ok1) {
  if constexpr (std::is_same<T, float>::value) {
    if (vec && ok1) {
      *reinterpret_cast<float2*>(p) = v;
      return;
    }
  } else {
    if (vec && ok1) {
      *reinterpret_cast<__nv_bfloat162*>(p) = __floats2bfloat162_rn(v.x, v.y);
      return;
    }
  }
  if (ok0) p[0] = from_f<T>(v.x);
  if (ok1) p[1] = from_f<T>(v.y);
}

// Up to four consecutive floats, entries at or past `n` read as 0 / not written.
__device__ __forceinline__ void load4(const float* p, int n, bool vec, float (&v)[4]) {
  if (vec && n >= 4) {
    const float4 q = *reinterpret_cast<const float4*>(p);
    v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = i < n ? p[i] : 0.f;
  }
}
__device__ __forceinline__ void store4(float* p, int n, bool vec, const float (&v)[4]) {
  if (vec && n >= 4) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < n) p[i] = v[i];
  }
}

// A decay rate in base 2.  An infinite one (or one that overflows here) becomes the
// largest: a step of zero, which pads the tiles, keeps the state (0 * -inf would be a
// NaN), and any other still makes the decay 0.
__device__ __forceinline__ float rate2(float a) {
  const float r = a * sm100::kLog2e;
  return r < -FLT_MAX ? -FLT_MAX : r;
}

// Decays e^{dt A}, from the rate in base 2.  ex2.approx of a negative argument is low on
// average: by 5e-9 to 8e-9 for arguments of 2e-4 to 4e-3, by 1.6e-8 to 2.7e-8 for 4e-3
// to 1/2 (relative, 2^20 arguments a range against 64 bits, one GB300; its largest error
// is 1.4e-7).  A state is multiplied once a token, so this bias adds up over its memory,
// and made most of the gradients' error (13 packed sequences in fp32: dA 1.1e-6, with
// exact decays 2.4e-7).  The exponent's multiply-add puts 1.4e-8 of it back: 5.3e-7.
// 2^kEx2Bias itself is 1, so that a step or a rate of zero still keeps the state.
constexpr float kEx2Bias = 2e-8f;   // 1.4e-8 log2 e
__device__ __forceinline__ float decay(float dt, float rate) { return sm100::ex2_fast(fmaf(dt, rate, kEx2Bias)); }
__device__ __forceinline__ float2 decay2(float2 dt, float2 rate) {
  const float2 e = __ffma2_rn(dt, rate, make_float2(kEx2Bias, kEx2Bias));
  return make_float2(sm100::ex2_fast(e.x), sm100::ex2_fast(e.y));
}

__device__ __forceinline__ float rcp_approx(float y) {   // about 1 ulp; 1 / inf = 0
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
  return r;
}

// softplus(v) = max(v, 0) + log(1 + e^{-|v|}).  log(1 + e) / e on [0, 1] is a
// polynomial of degree 8, fitted here by Remez's exchange for least relative
// error, so that tiny steps (v << 0) keep their relative accuracy: 6.4e-8 with
// these rounded coefficients (the last one alone is 6e-8 below 1), 1.8e-7 for
// log(1 + e) with the rounding of the fp32 steps.  e_out = e^{-|v|}.
__device__ __forceinline__ float2 softplus2(float2 v, float2& e_out) {
  const float2 e = make_float2(sm100::ex2_fast(-sm100::kLog2e * fabsf(v.x)), sm100::ex2_fast(-sm100::kLog2e * fabsf(v.y)));
  constexpr float k[9] = {0.00523269409f, -0.0295052379f, 0.0782259554f, -0.136632457f, 0.191060066f,
                          -0.24842982f, 0.333190978f, -0.499994934f, 0.99999994f};
  float2 p = make_float2(k[0], k[0]);
#pragma unroll
  for (int i = 1; i < 9; ++i) p = __ffma2_rn(p, e, make_float2(k[i], k[i]));
  e_out = e;
  return __ffma2_rn(p, e, make_float2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)));
}
__device__ __forceinline__ float softplus(float v) {
  float2 e;
  return softplus2(make_float2(v, v), e).x;
}

// sigmoid(v)
__device__ __forceinline__ float sigmoid(float v) {
  return rcp_approx(1.f + sm100::ex2_fast(-sm100::kLog2e * v));
}

__host__ __device__ constexpr int log2i(int v) { return v <= 1 ? 0 : 1 + log2i(v / 2); }

// A warp's lanes over channel pairs and states, and which tokens of a group of
// four a lane finishes (converts on the way in, writes on the way out).
template <int RL>
struct Lanes {
  static constexpr int CL = 32 / RL;              // lanes over channel pairs
  static constexpr int LR = log2i(RL);
  static constexpr int SP = 4 * RL;               // states with padding
  static constexpr int CPW = 2 * CL;              // channels a warp
  static constexpr int TPL = RL >= 4 ? 1 : 4 / RL;    // tokens of a group a lane finishes
  static constexpr int TT = RL >= 4 ? 16 : 4 * RL;    // tokens a tile: four a lane
  static constexpr int NG = TT / 4;
  int lane, chl, sl, own;
  bool dup;   // another lane finishes the same tokens
  __device__ __forceinline__ Lanes() {
    lane = threadIdx.x & 31;
    chl = lane & (CL - 1);
    sl = lane / CL;
    own = RL >= 4 ? sl >> (LR >= 2 ? LR - 2 : 0) : sl;
    dup = RL > 4 && (sl & (RL / 4 - 1)) != 0;
  }
  // token (within a tile) of this lane's slot k
  __device__ __forceinline__ int token(int k) const { return (k / TPL) * 4 + own * TPL + k % TPL; }
};

// Sums over the state lanes of four tokens' values v[tok * NV + i]: lane `own`
// ends with its tokens' sums in v[0 .. TPL * NV).
template <int RL, int NV>
__device__ __forceinline__ void reduce_states(float (&v)[4 * NV], int lane) {
  if constexpr (RL >= 2) {
    const bool up = lane & 16;
#pragma unroll
    for (int i = 0; i < 2 * NV; ++i) {
      const float send = up ? v[i] : v[i + 2 * NV];
      const float keep = up ? v[i + 2 * NV] : v[i];
      v[i] = keep + __shfl_xor_sync(~0u, send, 16);
    }
  }
  if constexpr (RL >= 4) {
    const bool up = lane & 8;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const float send = up ? v[i] : v[i + NV];
      const float keep = up ? v[i + NV] : v[i];
      v[i] = keep + __shfl_xor_sync(~0u, send, 8);
    }
  }
#pragma unroll
  for (int m = 4; m >= 32 / RL && RL >= 8; m >>= 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] += __shfl_xor_sync(~0u, v[i], m);
  }
}

// Rows t0 .. of a tile from a tensor (`first` its row 0, `stride` bytes a row) to
// dst[TT][ROW bytes]: `valid` bytes of a row exist, rows from `len` on become zero.
template <int TT, int ROW, int CH>
__device__ __forceinline__ void copy_rows(char* dst, const char* first, int stride, int t0, int len, int valid, int lane) {
  constexpr int PER = ROW / CH, N = TT * PER;
#pragma unroll
  for (int i = 0; i < (N + 31) / 32; ++i) {
    const int q = lane + 32 * i, t = q / PER, o = q % PER * CH;
    if (N % 32 == 0 || q < N) {
      int bytes = t0 + t < len ? min(valid - o, CH) : 0;
      if (bytes < 0) bytes = 0;
      copy_async<CH>(dst + q * CH, bytes > 0 ? first + (int64_t)(t0 + t) * stride + o : first, bytes);
    }
  }
}

// Host side ---------------------------------------------------------------

inline bool aligned_rows(const void* p, int64_t stride, size_t to) {
  return reinterpret_cast<uintptr_t>(p) % to == 0 && stride % (int64_t)to == 0;
}

// The widest copies that rows allow: x-like rows of xrow bytes a warp at px (stride bytes
// apart), B and C rows of srow bytes.
struct RowsOf {
  int xrow, srow;
  bool groups;   // several groups: chunks may not leave a group's channels or states
  int64_t xg, sg;   // bytes of a group's channels, states
  int rows = kWide;
  void use(const void* p, int64_t stride, int row, int64_t group) {
    if (!p) return;
    const int wide = row < 16 ? row : 16;
    if (rows == kWide && !(aligned_rows(p, stride, wide) && (!groups || group % wide == 0))) rows = kNarrow;
    if (rows == kNarrow && !(aligned_rows(p, stride, 4) && (!groups || group % 4 == 0))) rows = kRegs;
  }
  void x(const void* p, int64_t stride) { use(p, stride, xrow, xg); }
  void s(const void* p, int64_t stride) { use(p, stride, srow, sg); }
};

inline int lanes_for(int S) { return S <= 4 ? 1 : S <= 8 ? 2 : S <= 16 ? 4 : S <= 32 ? 8 : 16; }

// How a problem's sequences are cut: segments of seglen tokens, at most
// max_units of them in all.
struct Plan {
  int RL, cpw, cbg;
  int nseg, seglen;
  int64_t max_units;
  bool cut;   // some sequence may have several segments
};

// Packed sequences longer than a segment: fewer than this.
inline int64_t max_cut(int64_t N, int64_t T, int64_t seglen) {
  const int64_t m = T / seglen;
  return m < 1 ? 1 : m < N ? m : N;
}
inline size_t seg0_bytes(int64_t N, int64_t T, int64_t seglen) {
  return sizeof(int32_t) * (size_t)(N + 2 + max_cut(N, T, seglen));
}

Plan make_plan(const gdn_scan_problem& p);
Args base_args(const gdn_scan_problem& p, const Plan& pl, const void* x, const void* delta, const float* A,
               const void* B, const void* C, const float* Dp, const void* z, const float* dt_bias, const float* h0,
               const int32_t* cu);
// Packed batches: validates cu_seqlens into *status and writes seg0.
cudaError_t launch_prepare_segments(const int32_t* cu, int N, int64_t T, int seglen, int32_t* seg0, int32_t* status,
                                    cudaStream_t s);
// Start states of every segment into hseg (two launches); dtsum is kept.
cudaError_t launch_segment_states(const Args& a, const Plan& pl, gdn_dtype dt, cudaStream_t s);

}  // namespace scan
}  // namespace gdn
