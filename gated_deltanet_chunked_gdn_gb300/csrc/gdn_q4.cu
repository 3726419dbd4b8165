// gdn_q4.cu -- a few rows times a matrix of 4-bit weights with group scales:
//     y[m][n] = sum_k x[m][k] (code[n][k] - zero[n][k / g]) scale[n][k / g] + bias[n]
// (the projections of a decode step).  Its floor is the weights' bytes, N K / 2.
//
// Codes are read as they are stored (rows of K nibbles) and become tensor-core
// operands in registers: a nibble j in the low bits of a bf16's mantissa on top of
// 1/2 is 1/2 + j/256, exactly, so two neighbouring codes take a byte permutation and
// one AND-OR, and one packed subtraction of 1/2 + zero/256 leaves (code - zero)/256,
// again exactly.  mma.sync m16n8k16 then multiplies 16 weight rows by 8 columns of x
// with fp32 sums; 256 times the group's scale multiplies the fp32 sum, so no weight is
// ever rounded (and codes below 1 keep large fp32 x from overflowing before the scale).
// mma.sync and not tcgen05: for a few rows the weights are used once, and they stay in
// registers on their way to the products.  What bounds the loop at one row is turning
// codes into operands (16384 x 8192, by ncu: ALU pipe 70 %, mma.sync pipe 15 %, DRAM
// 31 %).  At 32 rows no unit is full (mma.sync 29 %, ALU 32 %, IPC 1.4 of 4): latency at
// 8 warps an SM.
//
// The k order inside an mma is free as long as both operands share it, but all its
// products have to be of one group.  A lane loads 16 bytes (32 codes) of a row, the
// four lanes of a row 128 codes (a block).  Groups of 64 or 32 are smaller than that:
// the four lanes exchange words (2 or 4 shuffles a 16 bytes) so that each mma's words
// come from one group, and keep the wide loads.
//
// Weights and x come by asynchronous copies into rings of blocks; every lane
// copies the weights that it reads itself.  x stands in pieces of eight values,
// swizzled so that the operands' reads meet no bank twice.  fp32 x (and rows that are
// not aligned) go through registers: each fp32 value is cut into three bf16 (24 bits
// in all), which take three of the mma's columns; the three sums are added at the end,
// so fp32 accuracy is kept.
//
// A CTA's eight warps are RW rows of warps over 16 MT weight rows each times 8 / RW
// shares of K, which add up through shared memory in a fixed order.  The warps of a
// share use one copy of x: many columns of x would otherwise be brought and read once a
// 16 weight rows, at four times their bytes.
#include <type_traits>

#include "gdn_internal.h"
#include "gdn_sm100.cuh"

namespace gdn {
namespace {

constexpr int kBlock = 128;   // codes of a row that its four lanes load at once

struct Q4Args {
  const void* x;
  const uint8_t* w;
  const void* scale;
  const uint8_t* zero;
  const float* bias;
  void* y;
  int64_t ldx;
  int M, N, K, groups;   // groups a row
  unsigned gmagic;       // 2^32 / (group / 32), rounded up (0 for 1): a code's group by a multiplication
  bool vec;              // rows of x in whole 16-byte pieces
};

__device__ __forceinline__ void mma_bf16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_bf16_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// The codes of a word as four pairs of neighbours, less their zero point, over 256
// (off: 1/2 + zero/256).
__device__ __forceinline__ void decode(uint32_t w, __nv_bfloat162 off, uint32_t (&p)[4]) {
  const uint32_t h = w >> 4;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    // byte j of w (its low nibble is the first code) and of h (the second)
    uint32_t v;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;"   // (a & b) | c
        : "=r"(v)
        : "r"(__byte_perm(w, h, 0x0400 + 0x1111 * j)), "r"(0x000f000fu), "r"(0x3f003f00u));
    const __nv_bfloat162 d = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&v), off);
    p[j] = *reinterpret_cast<const uint32_t*>(&d);
  }
}

// Columns of the mma that a row of x takes.
template <typename T> constexpr int kParts = std::is_same<T, float>::value ? 3 : 1;

// Eight values of x for one column, as loaded.
template <typename T> struct X8;
template <> struct X8<__nv_bfloat16> {
  uint4 q;
  __device__ __forceinline__ void load(const __nv_bfloat16* p, bool vec) {
    if (vec) {
      q = __ldg(reinterpret_cast<const uint4*>(p));
    } else {
      const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
      uint32_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __ldg(h + 2 * i) | ((uint32_t)__ldg(h + 2 * i + 1) << 16);
      q = make_uint4(v[0], v[1], v[2], v[3]);
    }
  }
  __device__ __forceinline__ void zero() { q = make_uint4(0u, 0u, 0u, 0u); }
  __device__ __forceinline__ uint4 operand(int) const { return q; }
};
template <> struct X8<float> {
  float f[8];
  __device__ __forceinline__ void load(const float* p, bool vec) {
    if (vec) {
      const float4 q = __ldg(reinterpret_cast<const float4*>(p)), r = __ldg(reinterpret_cast<const float4*>(p) + 1);
      f[0] = q.x, f[1] = q.y, f[2] = q.z, f[3] = q.w, f[4] = r.x, f[5] = r.y, f[6] = r.z, f[7] = r.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __ldg(p + i);
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 0.f;
  }
  // the first, second or third 8 bits (cut, not rounded, so that none overflows; an
  // infinity has no rest)
  __device__ __forceinline__ uint4 operand(int part) const {
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float hi = __uint_as_float(__float_as_uint(f[i]) & 0xffff0000u);
      const float r1 = hi == f[i] ? 0.f : f[i] - hi;
      const float mid = __uint_as_float(__float_as_uint(r1) & 0xffff0000u);
      v[i] = part == 0 ? hi : part == 1 ? mid : r1 - mid;
    }
    return make_uint4(sm100::pack_bf16(v[0], v[1]), sm100::pack_bf16(v[2], v[3]), sm100::pack_bf16(v[4], v[5]),
                      sm100::pack_bf16(v[6], v[7]));
  }
};

// NT: column tiles of 8.  MT: tiles of 16 weight rows a warp.  RW: rows of warps, of
// NW in all.  R: blocks in a ring, one in use, the others on their way.
template <int NT_, int MT_, int RW_, int NW_, int R_>
struct Conf {
  static constexpr int NT = NT_, MT = MT_, RW = RW_, NW = NW_, R = R_;
  static constexpr int KW = NW / RW, COLS = 8 * NT, ROWS = 16 * MT * RW;
  static constexpr size_t W = sizeof(uint4) * NW * R * MT * 64;             // rings of weights
  static constexpr size_t SUM = sizeof(float) * KW * ROWS * (COLS + 1);     // the shares' sums
  // .. and of x, NCP columns to a piece
  static constexpr size_t bytes(int ncp) {
    const size_t b = W + sizeof(uint4) * KW * R * 16 * ncp;
    return b > SUM ? b : SUM;
  }
};

// GM: group size a multiple of 128 (0), 64 (1), 32 (2).  NCP: ncol, the columns there
// are, rounded up to a power of two (what a piece's columns take in shared memory; the
// other lanes of an mma read one of these, for columns of the result that nobody
// stores).  ASYNC: bf16 x in rows of whole 16-byte pieces.
template <typename T, typename ST, typename F, int GM, int NCP, bool ASYNC>
__global__ void __launch_bounds__(32 * F::NW) q4_matvec_kernel(const Q4Args a, int m0, int ncol) {
  constexpr int NT = F::NT, MT = F::MT, RW = F::RW, kRing = F::R;
  constexpr int P = kParts<T>, KW = F::KW, COLS = F::COLS;
  constexpr int SLOTS = GM == 0 ? 1 : GM == 1 ? 2 : 4;   // groups a block can meet
  constexpr int QB = 4 / SLOTS;                          // blocks whose groups a row's four lanes hold
  extern __shared__ __align__(16) char raw_smem[];
  const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
  const int rw = wp % RW, kw = wp / RW;
  const int r = lane >> 2, c = lane & 3;
  uint4* ring = reinterpret_cast<uint4*>(raw_smem) + wp * (kRing * MT * 64) + lane;   // [kRing][MT][2][32 lanes]
  uint4* xring = reinterpret_cast<uint4*>(raw_smem + F::W) + kw * (kRing * 16 * NCP);   // [kRing][16 words][NCP]

  const int nb = (a.K + kBlock - 1) / kBlock;   // the last block may be short (groups of 32 or 64)
  const int b0 = (int)((int64_t)nb * kw / KW), b1 = (int)((int64_t)nb * (kw + 1) / KW);
  // 32-bit offsets from the CTA's first row (at most 128 rows of 2^20 codes): addresses
  // and predicates would otherwise cost as much as the codes' conversion
  const int first = F::ROWS * blockIdx.x;
  const uint8_t* wbase = a.w + (int64_t)first * (a.K / 2);
  const ST* sbase = static_cast<const ST*>(a.scale) + (int64_t)first * a.groups;
  const uint8_t* zbase = a.zero ? a.zero + (int64_t)first * a.groups : nullptr;
  uint32_t woff[MT][2], soff[MT][2];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int row = min(16 * (MT * rw + t) + r + 8 * h, a.N - 1 - first);   // past the end: not stored
      woff[t][h] = row * (uint32_t)(a.K / 2) + 16 * c;
      soff[t][h] = row * (uint32_t)a.groups;
    }
  const int bw = min(b1, (a.K - 32 * c + kBlock - 1) / kBlock);   // blocks in which this lane's codes exist

  // word kc's pieces stand in the order col ^ swz(kc): the reads below take two
  // neighbouring columns of four words at a time
  auto swz = [](int kc) { return GM == 0 ? (kc / 4 & 3) * 2 : GM == 1 ? ((kc / 4 & 1) + 2 * (kc / 2 & 1)) * 2 : (kc & 3) * 2; };
  // x of a block: this lane brings word kcol of columns col0, col0 + 2 RW, ..
  const int kcol = lane % 16, col0 = 2 * rw + lane / 16, sw = swz(kcol) & (NCP - 1);
  const T* xsrc = static_cast<const T*>(a.x) + (m0 + col0 / P) * a.ldx + b0 * (int64_t)kBlock + 8 * kcol;
  const int bx = (a.K - 8 * kcol + kBlock - 1) / kBlock;   // .. its words of x
  auto fetch = [&](int b, int slot) {
    // (what stands behind the last codes of a short block meets zeros of x)
    if (b < bw) {
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                           sm100::smem_u32(ring + (slot * MT * 2 + t * 2 + h) * 32)),
                       "l"(wbase + (woff[t][h] + (uint32_t)b * (kBlock / 2)))
                       : "memory");
    }
    if (b < b1) {
      const bool have = b < bx;
      uint4* dst = xring + (slot * 16 + kcol) * NCP;
      const T* src = xsrc;
#pragma unroll
      for (int j = 0; j < (NCP + 2 * RW - 1) / (2 * RW); ++j) {
        const int col = col0 + j * 2 * RW;
        if (col >= ncol) break;
        if constexpr (ASYNC) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(sm100::smem_u32(dst + (col ^ sw))),
                       "l"(have ? src : static_cast<const T*>(a.x)), "r"(have ? 16 : 0)
                       : "memory");
          src += 2 * RW * a.ldx;
        } else {
          X8<T> x;
          x.zero();
          if (have) x.load(xsrc + (col / P - col0 / P) * a.ldx, a.vec);
          dst[col ^ sw] = x.operand(col % P);
        }
      }
      xsrc += kBlock;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll 1
  for (int i = 0; i < kRing - 1; ++i) fetch(b0 + i, i);

  // scales (and zero points) of QB blocks from b on: lane c has the c-th group's.  Two
  // such steps are on their way, as loaded: a conversion would wait for them.
  float s0[MT][2];      // 256 times the scale
  uint32_t o0[MT][2];   // 1/2 + zero/256, twice
  ST s1[MT][2], s2[MT][2];
  uint8_t z1[MT][2], z2[MT][2];
  auto load_scales = [&](int b, ST (&sc)[MT][2], uint8_t (&ze)[MT][2]) {
    // past the end (an empty share's too) some group of the row: x is zero there
    const int k = max(0, min(b * kBlock + c * (kBlock / SLOTS), a.K - 32));
    const unsigned g = a.gmagic ? __umulhi((unsigned)k / 32, a.gmagic) : (unsigned)k / 32;
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        sc[t][h] = sbase[soff[t][h] + g];
        ze[t][h] = zbase ? zbase[soff[t][h] + g] : 8;
      }
  };
  load_scales(b0, s1, z1);
  load_scales(b0 + QB, s2, z2);

  // this lane's column of x among a word's pieces, and its first word (see below)
  const int xlane = ((r ^ (2 * c)) & (NCP - 1)) + NCP * (GM == 0 ? 4 * c : GM == 1 ? 4 * (c & 1) + 2 * (c >> 1) : c);

  float total[MT][NT][4];
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) total[t][n][i] = 0.f;

  int slot = 0, q = 0;   // ring slot; the block's place among those whose scales are here
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 2) : "memory");
    if constexpr (RW == 1) __syncwarp();
    else asm volatile("bar.sync %0, %1;" ::"r"(1 + kw), "n"(32 * RW) : "memory");
    fetch(b + kRing - 1, slot == 0 ? kRing - 1 : slot - 1);   // into the slot of the block before
    if (q == 0) {
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          s0[t][h] = 256.f * to_f(s1[t][h]);
          o0[t][h] = 0x3f003f00u + 0x10001u * z1[t][h];
          s1[t][h] = s2[t][h], z1[t][h] = z2[t][h];
        }
      load_scales(b + 2 * QB, s2, z2);
    }
    uint32_t wd[MT][2][4];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 v = ring[(slot * MT * 2 + t * 2 + h) * 32];
        uint32_t w0 = v.x, w1 = v.y, w2 = v.z, w3 = v.w;
        if constexpr (GM >= 1) {   // lanes 0, 1 hand their upper two words to lanes 2, 3 for the lower two
          const bool up = c & 2;
          const uint32_t e0 = __shfl_xor_sync(~0u, up ? w0 : w2, 2), e1 = __shfl_xor_sync(~0u, up ? w1 : w3, 2);
          if (up) w0 = e0, w1 = e1; else w2 = e0, w3 = e1;
        }
        if constexpr (GM == 2) {   // .. and the lanes of a pair one word of each two
          const bool up = c & 1;
          const uint32_t e0 = __shfl_xor_sync(~0u, up ? w0 : w1, 1), e1 = __shfl_xor_sync(~0u, up ? w2 : w3, 1);
          if (up) w0 = e0, w2 = e1; else w1 = e0, w3 = e1;
        }
        wd[t][h][0] = w0, wd[t][h][1] = w1, wd[t][h][2] = w2, wd[t][h][3] = w3;
      }
    const uint4* xrow = xring + slot * 16 * NCP + xlane;
#pragma unroll
    for (int g = 0; g < SLOTS; ++g) {   // the words of one group
      constexpr int CH = NT == 1 ? 2 : 1;   // independent sums: an mma waits for its accumulator
      float acc[CH][MT][NT][4], f[MT][2];
      __nv_bfloat162 o[MT][2];
#pragma unroll
      for (int t = 0; t < MT; ++t) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f[t][h] = __shfl_sync(~0u, s0[t][h], q * SLOTS + g, 4);
          const uint32_t os = a.zero ? __shfl_sync(~0u, o0[t][h], q * SLOTS + g, 4) : 0x3f083f08u;
          o[t][h] = *reinterpret_cast<const __nv_bfloat162*>(&os);
        }
      }
#pragma unroll
      for (int i = g * (4 / SLOTS); i < (g + 1) * (4 / SLOTS); ++i) {
        // this lane's word i is the block's word 4 c + i (GM 0), 8 (i / 2) + 4 (c % 2) +
        // 2 (c / 2) + i % 2 (1) or 4 i + c (2); its swizzle is 2 c
        const int word = GM == 0 ? i : GM == 1 ? 8 * (i / 2) + (i & 1) : 4 * i;
        uint4 xb[NT];
#pragma unroll
        for (int n = 0; n < NT; ++n) xb[n] = xrow[word * NCP + (8 * n & (NCP - 1))];
#pragma unroll
        for (int t = 0; t < MT; ++t) {
          uint32_t pa[4], pb[4];
          decode(wd[t][0][i], o[t][0], pa);
          decode(wd[t][1][i], o[t][1], pb);
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const bool first = i == g * (4 / SLOTS);
            if (first) mma_bf16_zero(acc[0][t][n], pa[0], pb[0], pa[1], pb[1], xb[n].x, xb[n].y);
            else mma_bf16(acc[0][t][n], pa[0], pb[0], pa[1], pb[1], xb[n].x, xb[n].y);
            if (first && CH == 2) mma_bf16_zero(acc[CH - 1][t][n], pa[2], pb[2], pa[3], pb[3], xb[n].z, xb[n].w);
            else mma_bf16(acc[CH - 1][t][n], pa[2], pb[2], pa[3], pb[3], xb[n].z, xb[n].w);
          }
        }
      }
#pragma unroll
      for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float v = acc[0][t][n][i];
            if (CH == 2) v += acc[CH - 1][t][n][i];
            total[t][n][i] = fmaf(f[t][i / 2], v, total[t][n][i]);
          }
    }
    slot = slot + 1 == kRing ? 0 : slot + 1;
    q = q + 1 == QB ? 0 : q + 1;
  }

  // the shares' sums, in order
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncthreads();
  float* red = reinterpret_cast<float*>(raw_smem);   // [KW][ROWS][COLS + 1]
  constexpr int ROWS = F::ROWS, LD = COLS + 1;
#pragma unroll
  for (int t = 0; t < MT; ++t)
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        red[(kw * ROWS + 16 * (MT * rw + t) + r + 8 * (i / 2)) * LD + 8 * n + 2 * c + i % 2] = total[t][n][i];
  __syncthreads();
  const int rows = ncol / P, n0 = ROWS * blockIdx.x;
  for (int i = threadIdx.x; i < ROWS * rows; i += 32 * F::NW) {
    const int n = i % ROWS, m = i / ROWS;
    if (n0 + n >= a.N) continue;
    float s = 0.f;
#pragma unroll
    for (int k = 0; k < KW; ++k)
#pragma unroll
      for (int e = P - 1; e >= 0; --e) s += red[(k * ROWS + n) * LD + m * P + e];
    if (a.bias) s += a.bias[n0 + n];
    static_cast<T*>(a.y)[(int64_t)(m0 + m) * a.N + n0 + n] = from_f<T>(s);
  }
}

template <typename T, typename ST, typename F, int NCP>
cudaError_t launch_q4(const Q4Args& a, int m0, int ncol, cudaStream_t s) {
  constexpr size_t bytes = F::bytes(NCP);
  auto go = [&](auto* k) {
    if constexpr (bytes > 48 * 1024) {
      const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
      if (e != cudaSuccess) return e;
    }
    k<<<(unsigned)ceil_div(a.N, F::ROWS), 32 * F::NW, bytes, s>>>(a, m0, ncol);
    return cudaGetLastError();
  };
  auto by_vec = [&](auto gm) {
    constexpr int GM = decltype(gm)::value;
    if constexpr (kParts<T> == 1) {
      if (a.vec) return go(q4_matvec_kernel<T, ST, F, GM, NCP, true>);
    }
    return go(q4_matvec_kernel<T, ST, F, GM, NCP, false>);
  };
  const int group = a.K / a.groups;
  if (group % 128 == 0) return by_vec(std::integral_constant<int, 0>());
  if (group % 64 == 0) return by_vec(std::integral_constant<int, 1>());
  return by_vec(std::integral_constant<int, 2>());
}

// Which configuration.  One GB300, us a call in a graph, the kept side and the other
// one in the same code; bf16 x, groups of 128, no zero points, unless said.
//   One row of x: 16 weight rows a warp and short rings, so that three CTAs share an SM
//     (the other: 32 rows and rings of six).  16384 x 8192 24.6 / 25.6, in groups of 32
//     30.4 / 34.5; 4096 x 4096 6.1 / 6.1.
//   Up to 4 columns: warps in pairs on one copy of x (alone).  2 rows of 4096 x 4096 8.1 /
//     9.2; 4 rows of 16384 x 8192 30.6 / 37.3.
//   Up to 8: 32 rows a warp (16) from 96 weight rows an SM on.  8 rows of 16384 x 8192 29.7 /
//     38.7, 24576 x 8192 42.1 / 54.6; 5 rows of 16384 x 4096 in groups of 32 23.3 / 26.4;
//     2 fp32 rows of 16384 x 8192 34.2 / 57.5.  16 rows a warp (32) below.  5 rows of 12288 x
//     4096 in groups of 32 21.6 / 22.2; but of 8192 x 4096 15.9 / 14.9, and 8 rows of 12288 x
//     8192 34.1 / 29.4, 14336 x 8192 36.2 / 29.5: the limit is too high for those.
//   Up to 16: 32 rows a warp, four warps on one x (16 rows, two warps).  16 rows of 16384 x
//     8192 36.6 / 57.1, 12288 x 4096 in groups of 32 26.2 / 34.2; but 4096 x 4096 18.7 / 12.6,
//     9 rows 17.2 / 10.9: few weight rows leave SMs idle this way.
//   Up to 16 columns of fp32 x, cut by the warps that bring it: fewer warps to a share (the
//     bf16 choice).  4 rows of 4096 x 4096 21.8 / 35.0; but 5 rows of 16384 x 8192 102 / 72.
//   17 to 32: 17 rows of 16384 x 8192 48.8, 32 rows 57.9; 32 of 12288 x 4096 in groups of 32
//     38.2 (nothing else measured).
template <typename T, typename ST>
cudaError_t run_rows(const Q4Args& a, cudaStream_t s) {
  constexpr int P = kParts<T>;
  for (int m0 = 0; m0 < a.M;) {   // 32 columns at a time: the weights come from HBM or L2 again for each
    const int left = (a.M - m0) * P;
    cudaError_t e;
    int rows = a.M - m0;
    if (left <= 1) {
      e = launch_q4<T, ST, Conf<1, 1, 1, 8, 4>, 1>(a, m0, left, s);
    } else if (left <= 4) {
      e = launch_q4<T, ST, Conf<1, 1, 2, 8, 4>, 4>(a, m0, left, s);
    } else if (left <= 8 && a.N < 96 * sm_count()) {
      e = launch_q4<T, ST, Conf<1, 1, 2, 8, 4>, 8>(a, m0, left, s);
    } else if (left <= 8) {
      e = launch_q4<T, ST, Conf<1, 2, 2, 8, 4>, 8>(a, m0, left, s);
    } else if (left <= 16 && P > 1) {
      e = launch_q4<T, ST, Conf<2, 1, 2, 8, 4>, 16>(a, m0, left, s);
    } else if (left <= 16) {
      e = launch_q4<T, ST, Conf<2, 2, 4, 8, 4>, 16>(a, m0, left, s);
    } else {
      if (rows > 32 / P) rows = 32 / P;
      e = launch_q4<T, ST, Conf<4, 2, 4, 8, 4>, 32>(a, m0, rows * P, s);
    }
    if (e != cudaSuccess) return e;
    m0 += rows;
  }
  return cudaSuccess;
}

}  // namespace

gdn_status run_q4_matvec(const void* x, int64_t ldx, const uint8_t* qweight, const void* scales, gdn_dtype sdt,
                         const uint8_t* zeros, const float* bias, int M, int N, int K, int group, gdn_dtype dt,
                         void* y, cudaStream_t s) {
  const int es = dt == GDN_F32 ? 4 : 2, g32 = group / 32;
  const bool vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && (ldx * es) % 16 == 0;
  const Q4Args a = {x, qweight, scales, zeros, bias, y, ldx, M, N, K, K / group,
                    g32 == 1 ? 0u : (unsigned)(((1ull << 32) + g32 - 1) / g32), vec};
  using B = __nv_bfloat16;
  cudaError_t e;
  if (dt == GDN_F32) e = sdt == GDN_F32 ? run_rows<float, float>(a, s) : run_rows<float, B>(a, s);
  else e = sdt == GDN_F32 ? run_rows<B, float>(a, s) : run_rows<B, B>(a, s);
  return e == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
}

}  // namespace gdn
