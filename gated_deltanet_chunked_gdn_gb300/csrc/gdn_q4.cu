// gdn_q4.cu -- a few rows times a matrix of 4-bit weights with group scales:
//     y[m][n] = sum_k x[m][k] (code[n][k] - zero[n][k / g]) scale[n][k / g] + bias[n]
// (the projections of a decode step).  Bound by the weights' bytes, N K / 2.
//
// Codes are read as they are stored (rows of K nibbles) and become tensor-core
// operands in registers: a nibble j in the low bits of a bf16's mantissa on top of
// 1/2 is 1/2 + j/256, exactly, so two codes take one AND-OR (and a shift), and one
// packed subtraction of 1/2 + zero/256 leaves (code - zero)/256, again exactly.
// mma.sync m16n8k16 then multiplies 16 weight rows by 8 columns of x with fp32 sums;
// 256 times the group's scale multiplies the fp32 sum, so no weight is ever rounded
// (and codes below 1 keep large fp32 x from overflowing before the scale).  mma.sync
// and not tcgen05: the weights are used once, and the way through shared memory
// and the accumulators' way through tensor memory would cost more than the
// products, which are far below the tensor units' rate; what bounds the loop beside
// HBM is turning codes into operands.
//
// The k order inside an mma is free as long as both operands share it: lane c of a
// row's four takes WL consecutive words (8 WL codes), 16 bytes a load when the
// group size allows (all lanes of an mma have to be in one group), and the four
// code pairs that a word's shifts yield are (0,4), (1,5), (2,6), (3,7), so x's words
// are permuted to match.
//
// fp32 x: each value is split into three bf16 (24 bits in all), which take three of
// the mma's columns; the three sums are added at the end, so fp32 accuracy is kept.
//
// A CTA computes 16 rows; its eight warps split K and add up through shared
// memory in a fixed order.
#include <type_traits>

#include "gdn_internal.h"
#include "gdn_sm100.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 8;

struct Q4Args {
  const void* x;
  const uint8_t* w;
  const void* scale;
  const uint8_t* zero;
  const float* bias;
  void* y;
  int64_t ldx;
  int M, N, K, group;
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four code pairs of a word, less their zero point, over 256 (off: 1/2 + zero/256).
__device__ __forceinline__ void decode(uint32_t w, __nv_bfloat162 off, uint32_t (&p)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint32_t v = ((w >> (4 * j)) & 0x000f000fu) | 0x3f003f00u;
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&v), off);
    p[j] = *reinterpret_cast<const uint32_t*>(&d);
  }
}

template <int WL> struct Words;
template <> struct Words<4> {
  uint4 v;
  __device__ __forceinline__ void load(const uint8_t* p) { v = __ldcs(reinterpret_cast<const uint4*>(p)); }
  __device__ __forceinline__ uint32_t at(int i) const { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
};
template <> struct Words<2> {
  uint2 v;
  __device__ __forceinline__ void load(const uint8_t* p) { v = __ldcs(reinterpret_cast<const uint2*>(p)); }
  __device__ __forceinline__ uint32_t at(int i) const { return i == 0 ? v.x : v.y; }
};
template <> struct Words<1> {
  uint32_t v;
  __device__ __forceinline__ void load(const uint8_t* p) { v = __ldcs(reinterpret_cast<const uint32_t*>(p)); }
  __device__ __forceinline__ uint32_t at(int) const { return v; }
};

// Columns of the mma that a row of x takes.
template <typename T> constexpr int kParts = std::is_same<T, float>::value ? 3 : 1;

// The x operand of a word's eight codes, for one column: pairs (0,4), (1,5), (2,6), (3,7).
__device__ __forceinline__ void load_x(const __nv_bfloat16* p, bool vec, int, uint32_t (&b)[4]) {
  uint32_t v[4];
  if (vec) {
    const uint4 q = __ldg(reinterpret_cast<const uint4*>(p));
    v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
  } else {
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __ldg(h + 2 * i) | ((uint32_t)__ldg(h + 2 * i + 1) << 16);
  }
  b[0] = __byte_perm(v[0], v[2], 0x5410), b[1] = __byte_perm(v[0], v[2], 0x7632);
  b[2] = __byte_perm(v[1], v[3], 0x5410), b[3] = __byte_perm(v[1], v[3], 0x7632);
}
__device__ __forceinline__ void load_x(const float* p, bool vec, int part, uint32_t (&b)[4]) {
  float f[8];
  if (vec) {
    const float4 q = __ldg(reinterpret_cast<const float4*>(p)), r = __ldg(reinterpret_cast<const float4*>(p) + 1);
    f[0] = q.x, f[1] = q.y, f[2] = q.z, f[3] = q.w, f[4] = r.x, f[5] = r.y, f[6] = r.z, f[7] = r.w;
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __ldg(p + i);
  }
  // the first, second or third 8 bits (cut, not rounded, so that none overflows; an
  // infinity has no rest)
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float hi = __uint_as_float(__float_as_uint(f[i]) & 0xffff0000u);
    const float r1 = hi == f[i] ? 0.f : f[i] - hi;
    const float mid = __uint_as_float(__float_as_uint(r1) & 0xffff0000u);
    f[i] = part == 0 ? hi : part == 1 ? mid : r1 - mid;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) b[i] = sm100::pack_bf16(f[i], f[i + 4]);
}

// NT: column tiles of 8.  WL: words a lane reads at once.
template <typename T, typename ST, int NT, int WL>
__global__ void __launch_bounds__(32 * kWarps) q4_matvec_kernel(const Q4Args a, int m0) {
  constexpr int KB = 32 * WL;   // codes of a row a step covers
  constexpr int P = kParts<T>;
  __shared__ float red[kWarps][16][NT * 8 + 1];
  const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
  const int r = lane >> 2, c = lane & 3;
  const int row0 = 16 * blockIdx.x;
  const int ra = min(row0 + r, a.N - 1), rb = min(row0 + r + 8, a.N - 1);   // past the end: not stored
  const int64_t rowbytes = a.K / 2, groups = a.K / a.group;
  const uint8_t* wa = a.w + ra * rowbytes + 4 * WL * c;
  const uint8_t* wb = a.w + rb * rowbytes + 4 * WL * c;
  const ST* scale = static_cast<const ST*>(a.scale);
  const ST* sa = scale + ra * groups;
  const ST* sb = scale + rb * groups;
  const uint8_t* za = a.zero ? a.zero + ra * groups : nullptr;
  const uint8_t* zb = a.zero ? a.zero + rb * groups : nullptr;
  // this lane's columns of x (the b operand): column lane / 4 of each tile
  const T* xp[NT];
  int part[NT];
  bool has[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const int col = 8 * t + r;
    part[t] = col % P;
    has[t] = m0 + col / P < a.M;
    xp[t] = static_cast<const T*>(a.x) + (has[t] ? (int64_t)(m0 + col / P) * a.ldx : 0) + 8 * WL * c;
  }
  const bool vec = (reinterpret_cast<uintptr_t>(a.x) % 16 == 0) && (a.ldx * sizeof(T)) % 16 == 0;

  const int nb = a.K / KB;
  const int b0 = (int)((int64_t)nb * wp / kWarps), b1 = (int)((int64_t)nb * (wp + 1) / kWarps);
  float total[NT][4], acc[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) total[t][i] = acc[t][i] = 0.f;
  const int per = a.group / KB;   // steps a group
  constexpr int U = NT >= 4 ? 2 : 4;
  for (int b = b0; b < b1; b += U) {
    Words<WL> qa[U], qb[U];
    float fa[U], fb[U];
    __nv_bfloat162 oa[U], ob[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int s = min(b + u, b1 - 1);
      qa[u].load(wa + (int64_t)s * (KB / 2));
      qb[u].load(wb + (int64_t)s * (KB / 2));
      const int g = s / per;
      fa[u] = 256.f * to_f(sa[g]), fb[u] = 256.f * to_f(sb[g]);
      oa[u] = __float2bfloat162_rn(0.53125f), ob[u] = oa[u];
      if (za) {
        oa[u] = __float2bfloat162_rn(fmaf((float)za[g], 0.00390625f, 0.5f));
        ob[u] = __float2bfloat162_rn(fmaf((float)zb[g], 0.00390625f, 0.5f));
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b + u >= b1) break;
#pragma unroll
      for (int i = 0; i < WL; ++i) {
        uint32_t pa[4], pb[4];
        decode(qa[u].at(i), oa[u], pa);
        decode(qb[u].at(i), ob[u], pb);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          uint32_t xb[4] = {0u, 0u, 0u, 0u};
          if (has[t]) load_x(xp[t] + (int64_t)(b + u) * KB + 8 * i, vec, part[t], xb);
          mma_bf16(acc[t], pa[0], pb[0], pa[1], pb[1], xb[0], xb[1]);
          mma_bf16(acc[t], pa[2], pb[2], pa[3], pb[3], xb[2], xb[3]);
        }
      }
      if ((b + u + 1) % per == 0 || b + u + 1 == b1) {   // the group (or this warp's share of it) ends
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          total[t][0] = fmaf(fa[u], acc[t][0], total[t][0]);
          total[t][1] = fmaf(fa[u], acc[t][1], total[t][1]);
          total[t][2] = fmaf(fb[u], acc[t][2], total[t][2]);
          total[t][3] = fmaf(fb[u], acc[t][3], total[t][3]);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[t][i] = 0.f;
        }
      }
    }
  }
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    red[wp][r][8 * t + 2 * c] = total[t][0], red[wp][r][8 * t + 2 * c + 1] = total[t][1];
    red[wp][r + 8][8 * t + 2 * c] = total[t][2], red[wp][r + 8][8 * t + 2 * c + 1] = total[t][3];
  }
  __syncthreads();
  const int rows = min(NT * 8 / P, a.M - m0);
  for (int i = threadIdx.x; i < 16 * rows; i += 32 * kWarps) {
    const int n = i % 16, m = i / 16;
    if (row0 + n >= a.N) continue;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k)
#pragma unroll
      for (int q = P - 1; q >= 0; --q) s += red[k][n][m * P + q];
    if (a.bias) s += a.bias[row0 + n];
    static_cast<T*>(a.y)[(int64_t)(m0 + m) * a.N + row0 + n] = from_f<T>(s);
  }
}

template <typename T, typename ST, int NT>
void launch_q4(const Q4Args& a, int m0, cudaStream_t s) {
  const unsigned grid = (unsigned)ceil_div(a.N, 16);
  if (a.group % 128 == 0) q4_matvec_kernel<T, ST, NT, 4><<<grid, 32 * kWarps, 0, s>>>(a, m0);
  else if (a.group % 64 == 0) q4_matvec_kernel<T, ST, NT, 2><<<grid, 32 * kWarps, 0, s>>>(a, m0);
  else q4_matvec_kernel<T, ST, NT, 1><<<grid, 32 * kWarps, 0, s>>>(a, m0);
}

template <typename T, typename ST>
void run_rows(const Q4Args& a, cudaStream_t s) {
  constexpr int P = kParts<T>;
  for (int m0 = 0; m0 < a.M;) {   // 32 columns at a time: the weights come from HBM or L2 again for each
    const int cols = (a.M - m0) * P;
    if (cols <= 8) launch_q4<T, ST, 1>(a, m0, s), m0 += 8 / P;
    else if (cols <= 16) launch_q4<T, ST, 2>(a, m0, s), m0 += 16 / P;
    else launch_q4<T, ST, 4>(a, m0, s), m0 += 32 / P;
  }
}

}  // namespace

gdn_status run_q4_matvec(const void* x, int64_t ldx, const uint8_t* qweight, const void* scales, gdn_dtype sdt,
                         const uint8_t* zeros, const float* bias, int M, int N, int K, int group, gdn_dtype dt,
                         void* y, cudaStream_t s) {
  Q4Args a = {x, qweight, scales, zeros, bias, y, ldx, M, N, K, group};
  using B = __nv_bfloat16;
  if (dt == GDN_F32) sdt == GDN_F32 ? run_rows<float, float>(a, s) : run_rows<float, B>(a, s);
  else sdt == GDN_F32 ? run_rows<B, float>(a, s) : run_rows<B, B>(a, s);
  return cudaGetLastError() == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace gdn
