// gdn_linear_tc.cuh -- shared by the tensor-core kernels of decayed linear attention: their parameters, the copies and
// the walk that forms states (gdn_linear_tc.cu), used by the forward pass and by the backward pass
// (gdn_linear_tc_bwd.cu).
#pragma once

#include <string.h>

#include "gdn_linear_sums.cuh"
#include "gdn_solve64.cuh"

namespace gdn {
namespace lin {

using namespace sm100;
using solve64::dsw;

struct TcParams {
  const float* decays;   // [slots of chunks][Hv][kDecays], decays_kernel
  const float* h0;       // [N][Hv][K][V]
  const float* start;    // [segments][Hv][K][V] states before the segments, or null (one segment a sequence)
  float* ht;             // final states (or a pool), or null
  const int32_t* idx;
  float* own;            // kOwn: the segments' own contributions
  Two* total;            // kOwn: their decays
  __nv_bfloat16* o;
  int32_t* status;
  Pieces pc;
  const int32_t* cu;
  float* emit;           // kEmit: [slots of chunks][Hv][K / 8][V][8]
  int slots, Hqk, Hv, V, varlen, T;
  float scale;
};

// The two bf16 values of a word.
__device__ __forceinline__ float2 halves(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// a and b as sums of two bf16 values each, packed.
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
  hi = pack_bf16(a, b);
  const float2 r = __ffma2_rn(halves(hi), make_float2(-1.f, -1.f), make_float2(a, b));
  lo = pack_bf16(r.x, r.y);
}

// Four values as sums of three bf16 values each, packed.
__device__ __forceinline__ void split3(const float4& v, uint32_t (&a)[2], uint32_t (&b)[2], uint32_t (&c)[2]) {
  const float2 minus = make_float2(-1.f, -1.f);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    float2 x = i ? make_float2(v.z, v.w) : make_float2(v.x, v.y);
    a[i] = pack_bf16(x.x, x.y);
    x = __ffma2_rn(halves(a[i]), minus, x);
    b[i] = pack_bf16(x.x, x.y);
    x = __ffma2_rn(halves(b[i]), minus, x);
    c[i] = pack_bf16(x.x, x.y);
  }
}

// 16-byte aligned block of a multiple of 16 bytes, global -> shared.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
               : "memory");
}

// Zeros in rows [from, 64) of a tile of 64-column atom columns `stride` bytes apart.
__device__ __forceinline__ void zero_rows(uint8_t* tile, int columns, uint32_t stride, int from, int tid, int threads) {
  const int n = (64 - from) * columns * 8;
  for (int u = tid; u < n; u += threads) {
    const int c = u % (columns * 8), r = from + u / (columns * 8);
    *reinterpret_cast<uint4*>(tile + (c >> 3) * stride + r * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
}

// Slot of a piece's first chunk among all chunks' decays: one more for every sequence before, whose last chunk may be
// short, so that no two chunks share one.
__device__ __forceinline__ int64_t chunk_slot(const Piece& p) { return p.tok0 / 64 + p.seq; }

// A chunk's decays: log2(e) b_i, e^{b_last - b_j}, scale e^{b_i} (64 each); e^{b_last} in two floats, and two unused;
// what the first 64 lack to 48 bits.  The walk reads all but the last.
constexpr int kDecays = 260, kWalkDecays = 196;

// What a launch of the walk does: the segments' own contributions and decays; outputs and final states; the state
// before every chunk, for the backward pass.
constexpr int kOwn = 0, kFull = 1, kEmit = 2;

int segment_tokens(const gdn_linear_problem& p);
size_t decays_bytes(const gdn_linear_problem& p);   // [slots of chunks][Hv][kDecays] fp32
gdn_status launch_decays(const gdn_linear_problem& p, const Pieces& pc, int size, const float* g, float scale,
                         float* decays, cudaStream_t s);
// One launch over the segments (size tokens each).  adj: the adjoint's walk, from the sequences' ends to their starts,
// with q and do in the places of k and v (and their row strides ld_x, ld_y).
gdn_status launch_walk(const gdn_linear_problem& p, int mode, bool adj, const void* q, const void* x, int64_t ld_x,
                       const void* y, int64_t ld_y, void* o, TcParams prm, int size, cudaStream_t s);
// Final states of sequences without tokens: the initial ones.
gdn_status launch_empty(const gdn_linear_problem& p, const Pieces& pc, const int32_t* cu, const float* h0, float* ht,
                        const int32_t* idx, int slots, cudaStream_t s);
// Parameters that do not depend on the launch.
TcParams tc_params(const gdn_linear_problem& p, const Pieces& pc, const int32_t* cu, float scale, const float* decays,
                   int32_t* status);

}  // namespace lin
}  // namespace gdn
