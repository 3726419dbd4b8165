// gdn_api.cu -- the C ABI of libgdn.so (declared in include/gdn.h): host-side
// validation, workspace sizing, path selection and the device status word.
#include <string.h>

#include "gdn_internal.h"

using namespace gdn;

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool dim_ok(int d) { return d == 64 || d == 128 || d == 256; }

// Shape checks that need no pointer.  Also normalises N for fixed length.
bool problem_ok(const gdn_problem* pp, gdn_problem* out) {
  if (!pp) return false;
  gdn_problem p = *pp;
  if (p.dt != GDN_F32 && p.dt != GDN_BF16) return false;
  if (p.Hqk <= 0 || p.Hv <= 0 || p.Hv % p.Hqk != 0 || p.Hv > 1024) return false;
  if (!dim_ok(p.K) || !dim_ok(p.V)) return false;
  if (p.C != 64 && p.C != 128) return false;
  if (p.varlen) {
    if (p.B != 1 || p.N <= 0 || p.T < 0) return false;
  } else {
    if (p.B <= 0 || p.T <= 0) return false;
    p.N = p.B;
  }
  // Token indices are int32 inside the kernels; element offsets are int64.
  if ((int64_t)p.B * p.T >= ((int64_t)1 << 31)) return false;
  if ((int64_t)p.N * p.Hv >= ((int64_t)1 << 31)) return false;
  *out = p;
  return true;
}

// Shape checks of a scan problem; normalises N for equal lengths and the flag.
gdn_status scan_problem_ok(const gdn_scan_problem* pp, gdn_scan_problem* out) {
  if (!pp) return GDN_ERR_INVALID_ARG;
  gdn_scan_problem p = *pp;
  if (p.dt != GDN_F32 && p.dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (p.D <= 0 || p.S <= 0 || p.G <= 0 || p.D % p.G != 0) return GDN_ERR_INVALID_ARG;
  if (p.varlen) {
    if (p.B != 1 || p.N <= 0 || p.T < 0) return GDN_ERR_INVALID_ARG;
  } else {
    if (p.B <= 0 || p.T <= 0) return GDN_ERR_INVALID_ARG;
    p.N = p.B;
  }
  if ((int64_t)p.B * p.T >= ((int64_t)1 << 31) - 1024) return GDN_ERR_INVALID_ARG;
  const int64_t gs = (int64_t)p.G * p.S;
  const int64_t ld[5] = {p.ld_x, p.ld_delta, p.ld_z, p.ld_b, p.ld_c}, row[5] = {p.D, p.D, p.D, gs, gs};
  for (int i = 0; i < 5; ++i)
    if (ld[i] != 0 && ld[i] < row[i]) return GDN_ERR_INVALID_ARG;
  for (int64_t l : ld)
    if (l > (1 << 28)) return GDN_ERR_UNSUPPORTED;   // the kernels keep row strides as 32-bit byte counts
  if (p.S > kScanMaxS || p.D > kScanMaxD || gs > (1 << 28)) return GDN_ERR_UNSUPPORTED;
  p.softplus = p.softplus != 0;
  *out = p;
  return GDN_OK;
}

// Pointers of a scan's inputs.
bool scan_inputs_ok(const gdn_scan_problem& p, const void* x, const void* delta, const float* A, const void* Bm,
                    const void* Cm, const float* Dskip, const void* z, const float* dt_bias, const int32_t* cu) {
  if (!A || (p.varlen ? !cu : cu != nullptr)) return false;
  if ((int64_t)p.B * p.T > 0 && (!x || !delta || !Bm || !Cm)) return false;
  const size_t es = p.dt == GDN_F32 ? 4 : 2;
  if (!aligned(x, es) || !aligned(delta, es) || !aligned(z, es) || !aligned(Bm, es) || !aligned(Cm, es)) return false;
  return aligned(A, p.S % 4 == 0 ? 16 : 4) && aligned(Dskip, 4) && aligned(dt_bias, 4) && aligned(cu, 4);
}

// Shape checks of a linear attention problem; fills in N, the row strides and the flags.
gdn_status linear_problem_ok(const gdn_linear_problem* pp, gdn_linear_problem* out) {
  if (!pp) return GDN_ERR_INVALID_ARG;
  gdn_linear_problem p = *pp;
  if (p.dt != GDN_F32 && p.dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (p.Hqk <= 0 || p.Hv <= 0 || p.Hv % p.Hqk != 0 || !dim_ok(p.K) || !dim_ok(p.V)) return GDN_ERR_INVALID_ARG;
  if (p.varlen) {
    if (p.B != 1 || p.N <= 0 || p.T < 0) return GDN_ERR_INVALID_ARG;
  } else {
    if (p.B <= 0 || p.T <= 0) return GDN_ERR_INVALID_ARG;
    p.N = p.B;
  }
  if (p.Hv > 1024) return GDN_ERR_UNSUPPORTED;
  // tokens are int32 in the kernels (room for the last chunk's end), element offsets int64; the grids are one-dimensional
  const int64_t tokens = (int64_t)p.B * p.T, blocks = (int64_t)(p.K / 64) * (p.V / 64) * p.Hv;
  if (tokens >= ((int64_t)1 << 31) - 1024) return GDN_ERR_INVALID_ARG;
  const int64_t chunks = p.varlen ? tokens / 64 + p.N : p.B * ceil_div(p.T, 64);
  if (chunks * blocks >= ((int64_t)1 << 31) || p.N * blocks * 4 >= ((int64_t)1 << 31)) return GDN_ERR_UNSUPPORTED;
  int64_t* ld[3] = {&p.ld_q, &p.ld_k, &p.ld_v};
  const int64_t row[3] = {(int64_t)p.Hqk * p.K, (int64_t)p.Hqk * p.K, (int64_t)p.Hv * p.V};
  for (int i = 0; i < 3; ++i) {
    if (*ld[i] == 0) *ld[i] = row[i];
    if (*ld[i] < row[i] || *ld[i] % (p.dt == GDN_F32 ? 4 : 8) != 0) return GDN_ERR_INVALID_ARG;
    if (*ld[i] > (1 << 28)) return GDN_ERR_UNSUPPORTED;
  }
  p.varlen = p.varlen != 0;
  p.g_per_head = p.g_per_head != 0;
  *out = p;
  return GDN_OK;
}

bool linear_inputs_ok(const gdn_linear_problem& p, const void* q, const void* k, const void* v, const float* g,
                      const int32_t* cu) {
  if (p.varlen ? !cu : cu != nullptr) return false;
  if ((int64_t)p.B * p.T > 0 && (!q || !k || !v || !g)) return false;
  return aligned(q, 16) && aligned(k, 16) && aligned(v, 16) && aligned(g, 4) && aligned(cu, 4);
}

gdn_path resolve(const gdn_problem& p, gdn_path path) {
  if (path == GDN_PATH_AUTO) {
    if (!fused_supported(p) && !fused1_supported(p)) return GDN_PATH_STAGED;
    if (!fused128_supported(p)) return GDN_PATH_FUSED1;
    if (cp_preferred(p)) return GDN_PATH_CP;
    return fused1_preferred(p) ? GDN_PATH_FUSED1 : GDN_PATH_FUSED;
  }
  return path;
}

bool path_ok(gdn_path path) {
  return path == GDN_PATH_AUTO || path == GDN_PATH_STAGED || path == GDN_PATH_FUSED || path == GDN_PATH_CP ||
         path == GDN_PATH_FUSED1;
}

bool path_supported(const gdn_problem& p, gdn_path path) {
  if (path == GDN_PATH_FUSED) return fused_supported(p);
  if (path == GDN_PATH_FUSED1) return fused1_supported(p);
  if (path == GDN_PATH_CP) return fused128_supported(p);
  return true;
}

size_t workspace_for(const gdn_problem& p, gdn_path path) {
  if (path == GDN_PATH_FUSED1) return fused1_workspace_bytes(p);
  if (path == GDN_PATH_FUSED) return fused_workspace_bytes(p);
  if (path == GDN_PATH_CP) return cp_workspace_bytes(p);
  gdn_staged_layout_t L;
  staged_layout(p, &L);
  return L.total;
}

size_t status_offset(const gdn_problem& p, gdn_path path) {
  if (path == GDN_PATH_FUSED || path == GDN_PATH_FUSED1) return fused_status_offset(p);
  if (path == GDN_PATH_CP) return 0;
  gdn_staged_layout_t L;
  staged_layout(p, &L);
  return L.status;
}

gdn_status check_call(const gdn_problem& p, const void* q, const void* k, const void* v, const float* g,
                      const float* beta, const float* h0, const int32_t* cu, const void* o, const float* ht,
                      const void* ws, size_t ws_bytes, size_t need) {
  const bool any_tokens = (int64_t)p.B * p.T > 0;
  if (any_tokens && (!q || !k || !v || !g || !beta || !o)) return GDN_ERR_INVALID_ARG;
  if (p.varlen && !cu) return GDN_ERR_INVALID_ARG;
  if (!p.varlen && cu) return GDN_ERR_INVALID_ARG;
  if (!ws || ws_bytes < need || !aligned(ws, kAlign)) return GDN_ERR_INVALID_ARG;
  const void* a16[] = {q, k, v, o};
  for (const void* x : a16)
    if (x && !aligned(x, 16)) return GDN_ERR_INVALID_ARG;
  const void* a4[] = {g, beta, h0, ht, cu};
  for (const void* x : a4)
    if (x && !aligned(x, 4)) return GDN_ERR_INVALID_ARG;
  return GDN_OK;
}

}  // namespace

size_t gdn::fwd_status_offset(const gdn_problem& p, gdn_path path) { return status_offset(p, resolve(p, path)); }

extern "C" {

size_t gdn_chunk_fwd_workspace_size(const gdn_problem* pp, gdn_path path) {
  gdn_problem p;
  if (!problem_ok(pp, &p)) return 0;
  if (!path_ok(path)) return 0;
  path = resolve(p, path);
  if (!path_supported(p, path)) return 0;
  return workspace_for(p, path);
}

gdn_path gdn_resolve_path(const gdn_problem* pp) {
  gdn_problem p;
  if (!problem_ok(pp, &p)) return GDN_PATH_STAGED;
  return resolve(p, GDN_PATH_AUTO);
}

gdn_status gdn_chunk_fwd(const gdn_problem* pp, gdn_path path, const void* q, const void* k, const void* v,
                         const float* g, const float* beta, float scale, const float* h0,
                         const int32_t* cu_seqlens, void* o, float* ht, void* workspace, size_t workspace_bytes,
                         void* stream) {
  gdn_problem p;
  if (!problem_ok(pp, &p)) return GDN_ERR_INVALID_ARG;
  if (!path_ok(path)) return GDN_ERR_INVALID_ARG;
  path = resolve(p, path);
  if (!path_supported(p, path)) return GDN_ERR_UNSUPPORTED;
  gdn_status st = check_call(p, q, k, v, g, beta, h0, cu_seqlens, o, ht, workspace, workspace_bytes,
                             workspace_for(p, path));
  if (st != GDN_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (path == GDN_PATH_FUSED) return run_fused(p, q, k, v, g, beta, scale, h0, cu_seqlens, o, ht, workspace, s);
  if (path == GDN_PATH_FUSED1) return run_fused1(p, q, k, v, g, beta, scale, h0, cu_seqlens, o, ht, workspace, s);
  if (path == GDN_PATH_CP)
    return run_cp(p, q, k, v, g, beta, scale, h0, cu_seqlens, o, ht, workspace, workspace_bytes, s);
  return run_staged(p, 6, q, k, v, g, beta, scale, h0, cu_seqlens, o, ht, workspace, s);
}

gdn_status gdn_chunk_fwd_staged(const gdn_problem* pp, int stop_after, const void* q, const void* k, const void* v,
                                const float* g, const float* beta, float scale, const float* h0,
                                const int32_t* cu_seqlens, void* o, float* ht, void* workspace,
                                size_t workspace_bytes, void* stream) {
  gdn_problem p;
  if (!problem_ok(pp, &p)) return GDN_ERR_INVALID_ARG;
  if (stop_after < 0 || stop_after > 6) return GDN_ERR_INVALID_ARG;
  gdn_status st = check_call(p, q, k, v, g, beta, h0, cu_seqlens, o, ht, workspace, workspace_bytes,
                             workspace_for(p, GDN_PATH_STAGED));
  if (st != GDN_OK) return st;
  return run_staged(p, stop_after, q, k, v, g, beta, scale, h0, cu_seqlens, o, ht, workspace,
                    static_cast<cudaStream_t>(stream));
}

gdn_status gdn_staged_layout(const gdn_problem* pp, gdn_staged_layout_t* out) {
  gdn_problem p;
  if (!problem_ok(pp, &p) || !out) return GDN_ERR_INVALID_ARG;
  return staged_layout(p, out);
}

gdn_status gdn_get_device_status(const gdn_problem* pp, gdn_path path, void* workspace, void* stream,
                                 int* dev_status) {
  gdn_problem p;
  if (!problem_ok(pp, &p) || !workspace || !dev_status) return GDN_ERR_INVALID_ARG;
  if (!path_ok(path)) return GDN_ERR_INVALID_ARG;
  path = resolve(p, path);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int32_t* word = reinterpret_cast<int32_t*>(static_cast<char*>(workspace) + status_offset(p, path));
  int32_t host = 0;
  if (cudaStreamSynchronize(s) != cudaSuccess) return GDN_ERR_CUDA;
  if (cudaMemcpy(&host, word, sizeof(host), cudaMemcpyDeviceToHost) != cudaSuccess) return GDN_ERR_CUDA;
  if (cudaMemset(word, 0, sizeof(int32_t)) != cudaSuccess) return GDN_ERR_CUDA;
  *dev_status = host;
  return GDN_OK;
}

gdn_status gdn_selftest_handover_timeout(const gdn_problem* pp, gdn_path path, const void* q, const void* k,
                                         const void* v,
                                         const float* g, const float* beta, float scale, const float* h0, void* o,
                                         float* ht, void* workspace, size_t workspace_bytes, int drop_window,
                                         long long wait_ns, void* stream) {
  gdn_problem p;
  if (!problem_ok(pp, &p) || p.varlen || wait_ns <= 0) return GDN_ERR_INVALID_ARG;
  if (path != GDN_PATH_FUSED && path != GDN_PATH_FUSED1) return GDN_ERR_INVALID_ARG;
  const bool one = path == GDN_PATH_FUSED1;
  if (!(one ? fused1_supported(p) && fused1_handover_window(p, drop_window) : fused_handover_window(p, drop_window)))
    return GDN_ERR_UNSUPPORTED;
  gdn_status st = check_call(p, q, k, v, g, beta, h0, nullptr, o, ht, workspace, workspace_bytes,
                             workspace_for(p, path));
  if (st != GDN_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const unsigned long long lim = static_cast<unsigned long long>(wait_ns);
  return one ? run_fused1(p, q, k, v, g, beta, scale, h0, nullptr, o, ht, workspace, s, drop_window, lim)
             : run_fused(p, q, k, v, g, beta, scale, h0, nullptr, o, ht, workspace, s, drop_window, lim);
}

gdn_status gdn_recurrent_fwd(const gdn_problem* pp, const void* q, const void* k, const void* v, const float* a,
                             const float* b, const float* A_log, const float* dt_bias, float scale, float* state,
                             const int32_t* state_indices, int state_slots, const int32_t* cu_seqlens, void* o,
                             void* stream) {
  gdn_problem p;
  if (!problem_ok(pp, &p)) return GDN_ERR_INVALID_ARG;
  if (p.V % 64 != 0 || state_slots <= 0 || !state || !A_log) return GDN_ERR_INVALID_ARG;
  if (!state_indices && state_slots < p.N) return GDN_ERR_INVALID_ARG;
  const bool any_tokens = (int64_t)p.B * p.T > 0;
  if (any_tokens && (!q || !k || !v || !a || !b || !o)) return GDN_ERR_INVALID_ARG;
  if (p.varlen != (cu_seqlens != nullptr)) return GDN_ERR_INVALID_ARG;
  const void* a16[] = {q, k, v, o, state};
  for (const void* x : a16)
    if (x && !aligned(x, 16)) return GDN_ERR_INVALID_ARG;
  const void* a4[] = {a, b, A_log, dt_bias, state_indices, cu_seqlens};
  for (const void* x : a4)
    if (x && !aligned(x, 4)) return GDN_ERR_INVALID_ARG;
  return run_recurrent(p, q, k, v, a, b, A_log, dt_bias, scale, state, state_indices, state_slots, cu_seqlens, o,
                       static_cast<cudaStream_t>(stream));
}

gdn_status gdn_causal_conv1d_fwd(const void* x, const float* weight, const float* bias, int W, void* conv_state,
                                 int state_slots, const int32_t* cache_indices, const int32_t* has_initial_state,
                                 const int32_t* cu_seqlens, int N, int B, int T, int D, gdn_dtype dt,
                                 gdn_activation act, void* y, void* stream) {
  if (W < 1 || W > 4 || D <= 0 || D % 8 != 0 || B < 0 || T < 0 || N < 0) return GDN_ERR_INVALID_ARG;
  if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (act != GDN_ACT_NONE && act != GDN_ACT_SILU) return GDN_ERR_INVALID_ARG;
  if (cu_seqlens ? B != 1 : N != B) return GDN_ERR_INVALID_ARG;
  if ((int64_t)B * T > 0 && (!x || !y)) return GDN_ERR_INVALID_ARG;
  if (!weight) return GDN_ERR_INVALID_ARG;
  if (W > 1 && conv_state && (state_slots <= 0 || (!cache_indices && state_slots < N))) return GDN_ERR_INVALID_ARG;
  const void* a16[] = {x, y, W > 1 ? conv_state : nullptr};
  for (const void* p : a16)
    if (p && !aligned(p, 16)) return GDN_ERR_INVALID_ARG;
  const void* a4[] = {weight, bias, cache_indices, has_initial_state, cu_seqlens};
  for (const void* p : a4)
    if (p && !aligned(p, 4)) return GDN_ERR_INVALID_ARG;
  return run_causal_conv1d(x, weight, bias, W, conv_state, state_slots, cache_indices, has_initial_state, cu_seqlens,
                           N, B, T, D, dt, act == GDN_ACT_SILU, y, static_cast<cudaStream_t>(stream));
}

size_t gdn_chunk_bwd_workspace_size(const gdn_problem* pp) {
  gdn_problem p;
  if (!problem_ok(pp, &p) || !bwd_supported(p)) return 0;
  // the chunked form also needs 16-byte aligned q, k, v and dout, which the
  // query cannot see: size for whichever form the call takes
  const size_t token = bwd_workspace_bytes(p);
  if (!bwdc_supported(p)) return token;
  const size_t chunked = bwdc_workspace_bytes(p);
  return chunked > token ? chunked : token;
}

gdn_status gdn_chunk_bwd(const gdn_problem* pp, const void* q, const void* k, const void* v, const float* g,
                         const float* beta, float scale, const float* h0, const int32_t* cu_seqlens,
                         const void* dout, const float* dht, float* dq, float* dk, float* dv, float* dg,
                         float* dbeta, float* dh0, void* workspace, size_t workspace_bytes, void* stream) {
  gdn_problem p;
  if (!problem_ok(pp, &p)) return GDN_ERR_INVALID_ARG;
  if (!bwd_supported(p)) return GDN_ERR_UNSUPPORTED;
  const bool any_tokens = (int64_t)p.B * p.T > 0;
  if (any_tokens && (!q || !k || !v || !g || !beta || !dout || !dq || !dk || !dv || !dg || !dbeta))
    return GDN_ERR_INVALID_ARG;
  if (p.varlen != (cu_seqlens != nullptr)) return GDN_ERR_INVALID_ARG;
  // the chunked backward reads q, k, v and dout in 16-byte vectors
  const bool chunked = bwdc_supported(p) && (int64_t)p.N * p.Hv > 0 && aligned(q, 16) && aligned(k, 16) &&
                       aligned(v, 16) && aligned(dout, 16);
  const size_t need = chunked ? bwdc_workspace_bytes(p) : bwd_workspace_bytes(p);
  if (!workspace || workspace_bytes < need || !aligned(workspace, kAlign)) return GDN_ERR_INVALID_ARG;
  const void* a16[] = {dh0, dht, h0};
  for (const void* x : a16)
    if (x && !aligned(x, 16)) return GDN_ERR_INVALID_ARG;
  const void* a4[] = {q, k, v, g, beta, cu_seqlens, dout, dq, dk, dv, dg, dbeta};
  for (const void* x : a4)
    if (x && !aligned(x, 4)) return GDN_ERR_INVALID_ARG;
  if (chunked)
    return run_bwdc(p, q, k, v, g, beta, scale, h0, cu_seqlens, dout, dht, dq, dk, dv, dg, dbeta, dh0, workspace,
                    static_cast<cudaStream_t>(stream));
  return run_bwd(p, q, k, v, g, beta, scale, h0, cu_seqlens, dout, dht, dq, dk, dv, dg, dbeta, dh0, workspace,
                 static_cast<cudaStream_t>(stream));
}

gdn_status gdn_chunk_bwd_get_device_status(void* workspace, void* stream, int* dev_status) {
  if (!workspace || !dev_status) return GDN_ERR_INVALID_ARG;
  int32_t* word = static_cast<int32_t*>(workspace);
  int32_t host = 0;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return GDN_ERR_CUDA;
  if (cudaMemcpy(&host, word, sizeof(host), cudaMemcpyDeviceToHost) != cudaSuccess) return GDN_ERR_CUDA;
  if (cudaMemset(word, 0, sizeof(int32_t)) != cudaSuccess) return GDN_ERR_CUDA;
  *dev_status = host;
  return GDN_OK;
}

size_t gdn_selective_scan_fwd_workspace_size(const gdn_scan_problem* pp) {
  gdn_scan_problem p;
  return scan_problem_ok(pp, &p) == GDN_OK ? scan_fwd_workspace_bytes(p) : 0;
}

namespace {
// The scan forward, its final states to rows of ht in order or by a slot map.
gdn_status scan_fwd(const gdn_scan_problem* pp, const void* x, const void* delta, const float* A, const void* Bm,
                    const void* Cm, const float* Dskip, const void* z, const float* dt_bias, const float* h0,
                    const int32_t* cu_seqlens, void* y, float* ht, const int32_t* state_indices, int state_slots,
                    void* workspace, size_t workspace_bytes, void* stream) {
  gdn_scan_problem p;
  const gdn_status ok = scan_problem_ok(pp, &p);
  if (ok != GDN_OK) return ok;
  if (!scan_inputs_ok(p, x, delta, A, Bm, Cm, Dskip, z, dt_bias, cu_seqlens)) return GDN_ERR_INVALID_ARG;
  const size_t sa = p.S % 4 == 0 ? 16 : 4, es = p.dt == GDN_F32 ? 4 : 2;
  if (!aligned(h0, sa) || !aligned(ht, sa) || !aligned(y, es)) return GDN_ERR_INVALID_ARG;
  if ((int64_t)p.B * p.T > 0 && !y) return GDN_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, kAlign) || workspace_bytes < scan_fwd_workspace_bytes(p))
    return GDN_ERR_INVALID_ARG;
  return run_scan_fwd(p, x, delta, A, Bm, Cm, Dskip, z, dt_bias, h0, cu_seqlens, y, ht, state_indices, state_slots,
                      workspace, static_cast<cudaStream_t>(stream));
}
}  // namespace

gdn_status gdn_selective_scan_fwd(const gdn_scan_problem* pp, const void* x, const void* delta, const float* A,
                                  const void* Bm, const void* Cm, const float* Dskip, const void* z,
                                  const float* dt_bias, const float* h0, const int32_t* cu_seqlens, void* y,
                                  float* ht, void* workspace, size_t workspace_bytes, void* stream) {
  return scan_fwd(pp, x, delta, A, Bm, Cm, Dskip, z, dt_bias, h0, cu_seqlens, y, ht, nullptr, 0, workspace,
                  workspace_bytes, stream);
}

gdn_status gdn_selective_scan_fwd_pool(const gdn_scan_problem* pp, const void* x, const void* delta, const float* A,
                                       const void* Bm, const void* Cm, const float* Dskip, const void* z,
                                       const float* dt_bias, const float* h0, const int32_t* cu_seqlens, void* y,
                                       float* state, const int32_t* state_indices, int state_slots, void* workspace,
                                       size_t workspace_bytes, void* stream) {
  if (!state || !state_indices || !aligned(state_indices, 4) || state_slots <= 0) return GDN_ERR_INVALID_ARG;
  return scan_fwd(pp, x, delta, A, Bm, Cm, Dskip, z, dt_bias, h0, cu_seqlens, y, state, state_indices, state_slots,
                  workspace, workspace_bytes, stream);
}

gdn_status gdn_selective_scan_get_device_status(const gdn_scan_problem* pp, void* workspace, void* stream,
                                                int* dev_status) {
  gdn_scan_problem p;
  if (!dev_status || scan_problem_ok(pp, &p) != GDN_OK) return GDN_ERR_INVALID_ARG;
  if (p.varlen) return gdn_chunk_bwd_get_device_status(workspace, stream, dev_status);   // the word is at the front
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return GDN_ERR_CUDA;
  *dev_status = GDN_DEV_OK;
  return GDN_OK;
}

gdn_status gdn_selective_scan_step(const gdn_scan_problem* pp, const void* x, const void* delta, const float* A,
                                   const void* Bm, const void* Cm, const float* Dskip, const void* z,
                                   const float* dt_bias, float* state, const int32_t* state_indices,
                                   int state_slots, const int32_t* cu_seqlens, void* y, void* stream) {
  gdn_scan_problem p;
  const gdn_status ok = scan_problem_ok(pp, &p);
  if (ok != GDN_OK) return ok;
  if (!scan_inputs_ok(p, x, delta, A, Bm, Cm, Dskip, z, dt_bias, cu_seqlens)) return GDN_ERR_INVALID_ARG;
  const size_t sa = p.S % 4 == 0 ? 16 : 4, es = p.dt == GDN_F32 ? 4 : 2;
  if (!state || state_slots <= 0 || !aligned(state, sa) || !aligned(state_indices, 4) || !aligned(y, es))
    return GDN_ERR_INVALID_ARG;
  if (!state_indices && state_slots < p.N) return GDN_ERR_INVALID_ARG;
  if ((int64_t)p.B * p.T > 0 && !y) return GDN_ERR_INVALID_ARG;
  return run_scan_step(p, x, delta, A, Bm, Cm, Dskip, z, dt_bias, state, state_indices, state_slots, cu_seqlens, y,
                       static_cast<cudaStream_t>(stream));
}

size_t gdn_selective_scan_bwd_workspace_size(const gdn_scan_problem* pp) {
  gdn_scan_problem p;
  return scan_problem_ok(pp, &p) == GDN_OK && p.G <= kScanBwdMaxG ? scan_bwd_workspace_bytes(p) : 0;
}

gdn_status gdn_selective_scan_bwd(const gdn_scan_problem* pp, const void* x, const void* delta, const float* A,
                                  const void* Bm, const void* Cm, const float* Dskip, const void* z,
                                  const float* dt_bias, const float* h0, const int32_t* cu_seqlens,
                                  const void* dout, const float* dht, void* dx, void* ddelta, float* dA, void* dB,
                                  void* dC, float* dD, void* dz, float* ddt_bias, float* dh0, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  gdn_scan_problem p;
  const gdn_status ok = scan_problem_ok(pp, &p);
  if (ok != GDN_OK) return ok;
  if (p.G > kScanBwdMaxG) return GDN_ERR_UNSUPPORTED;
  if (!scan_inputs_ok(p, x, delta, A, Bm, Cm, Dskip, z, dt_bias, cu_seqlens)) return GDN_ERR_INVALID_ARG;
  const size_t sa = p.S % 4 == 0 ? 16 : 4, es = p.dt == GDN_F32 ? 4 : 2;
  const void* states[] = {h0, dht, dA, dh0};
  for (const void* q : states)
    if (!aligned(q, sa)) return GDN_ERR_INVALID_ARG;
  const void* rows[] = {dout, dx, ddelta, dB, dC, dz};
  for (const void* q : rows)
    if (!aligned(q, es)) return GDN_ERR_INVALID_ARG;
  if (!dA || !aligned(dD, 4) || !aligned(ddt_bias, 4) || !z != !dz) return GDN_ERR_INVALID_ARG;
  if ((int64_t)p.B * p.T > 0 && (!dout || !dx || !ddelta || !dB || !dC)) return GDN_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, kAlign) || workspace_bytes < scan_bwd_workspace_bytes(p))
    return GDN_ERR_INVALID_ARG;
  return run_scan_bwd(p, x, delta, A, Bm, Cm, Dskip, z, dt_bias, h0, cu_seqlens, dout, dht, dx, ddelta, dA, dB, dC,
                      dD, dz, ddt_bias, dh0, workspace, static_cast<cudaStream_t>(stream));
}

size_t gdn_causal_conv1d_bwd_workspace_size(int B, int T, int D, int W) {
  if (W < 1 || W > 4 || D <= 0 || D % 8 != 0 || B < 0 || T < 0) return 0;
  return conv1d_bwd_workspace_bytes((int64_t)B * T, D, W);
}

gdn_status gdn_causal_conv1d_bwd(const void* x, const float* weight, const float* bias, int W,
                                 const void* initial_state, const int32_t* cu_seqlens, int N, int B, int T, int D,
                                 gdn_dtype dt, gdn_activation act, const void* dout, const void* dfinal_state,
                                 void* dx, float* dweight, float* dbias, void* dinitial_state, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  if (W < 1 || W > 4 || D <= 0 || D % 8 != 0 || B < 0 || T < 0 || N < 0) return GDN_ERR_INVALID_ARG;
  if (dt != GDN_F32 && dt != GDN_BF16) return GDN_ERR_INVALID_ARG;
  if (act != GDN_ACT_NONE && act != GDN_ACT_SILU) return GDN_ERR_INVALID_ARG;
  if (cu_seqlens ? B != 1 : N != B) return GDN_ERR_INVALID_ARG;
  if ((int64_t)B * T > 0 && (!x || !dout || !dx)) return GDN_ERR_INVALID_ARG;
  if (!weight || !dweight) return GDN_ERR_INVALID_ARG;
  const void* a16[] = {x, dout, dx, initial_state, dfinal_state, dinitial_state};
  for (const void* p : a16)
    if (!aligned(p, 16)) return GDN_ERR_INVALID_ARG;
  const void* a4[] = {weight, bias, cu_seqlens, dweight, dbias};
  for (const void* p : a4)
    if (!aligned(p, 4)) return GDN_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, kAlign) ||
      workspace_bytes < conv1d_bwd_workspace_bytes((int64_t)B * T, D, W))
    return GDN_ERR_INVALID_ARG;
  return run_causal_conv1d_bwd(x, weight, bias, W, initial_state, cu_seqlens, N, B, T, D, dt, act == GDN_ACT_SILU,
                               dout, dfinal_state, dx, dweight, dbias, dinitial_state, workspace,
                               static_cast<cudaStream_t>(stream));
}

gdn_status gdn_q4_matvec(const void* x, int64_t ld_x, const uint8_t* qweight, const void* scales, gdn_dtype sdt,
                         const uint8_t* zeros, const float* bias, int M, int N, int K, int group, gdn_dtype dt,
                         void* y, void* stream) {
  if ((dt != GDN_F32 && dt != GDN_BF16) || (sdt != GDN_F32 && sdt != GDN_BF16)) return GDN_ERR_INVALID_ARG;
  if (M < 0 || N <= 0 || K <= 0 || group <= 0 || group % 32 != 0 || K % group != 0) return GDN_ERR_INVALID_ARG;
  if (K > (1 << 20)) return GDN_ERR_UNSUPPORTED;
  if (ld_x == 0) ld_x = K;
  if (ld_x < K || !qweight || !aligned(qweight, 16) || !scales) return GDN_ERR_INVALID_ARG;
  const size_t es = dt == GDN_F32 ? 4 : 2;
  if (!aligned(x, es) || !aligned(y, es) || !aligned(scales, sdt == GDN_F32 ? 4 : 2) || !aligned(bias, 4))
    return GDN_ERR_INVALID_ARG;
  if (M == 0) return GDN_OK;
  if (!x || !y) return GDN_ERR_INVALID_ARG;
  return run_q4_matvec(x, ld_x, qweight, scales, sdt, zeros, bias, M, N, K, group, dt, y,
                       static_cast<cudaStream_t>(stream));
}

size_t gdn_linear_attn_fwd_workspace_size(const gdn_linear_problem* pp) {
  gdn_linear_problem p;
  return linear_problem_ok(pp, &p) == GDN_OK ? linear_fwd_workspace_bytes(p) : 0;
}

gdn_status gdn_linear_attn_fwd(const gdn_linear_problem* pp, const void* q, const void* k, const void* v,
                               const float* g, float scale, const float* h0, const int32_t* cu_seqlens, void* o,
                               float* ht, const int32_t* state_indices, int state_slots, void* workspace,
                               size_t workspace_bytes, void* stream) {
  gdn_linear_problem p;
  const gdn_status st = linear_problem_ok(pp, &p);
  if (st != GDN_OK) return st;
  if (!linear_inputs_ok(p, q, k, v, g, cu_seqlens) || !aligned(h0, 16) || !aligned(ht, 16) || !aligned(o, 16))
    return GDN_ERR_INVALID_ARG;
  if ((int64_t)p.B * p.T > 0 && !o) return GDN_ERR_INVALID_ARG;
  if (state_indices && (!ht || state_slots <= 0 || !aligned(state_indices, 4))) return GDN_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, kAlign) || workspace_bytes < linear_fwd_workspace_bytes(p))
    return GDN_ERR_INVALID_ARG;
  return run_linear_fwd(p, q, k, v, g, scale, h0, cu_seqlens, o, ht, state_indices, state_slots, workspace,
                        static_cast<cudaStream_t>(stream));
}

size_t gdn_linear_attn_bwd_workspace_size(const gdn_linear_problem* pp) {
  gdn_linear_problem p;
  return linear_problem_ok(pp, &p) == GDN_OK ? linear_bwd_workspace_bytes(p) : 0;
}

gdn_status gdn_linear_attn_bwd(const gdn_linear_problem* pp, const void* q, const void* k, const void* v,
                               const float* g, float scale, const float* h0, const int32_t* cu_seqlens,
                               const void* dout, const float* dht, void* dq, void* dk, void* dv, float* dg,
                               float* dh0, void* workspace, size_t workspace_bytes, void* stream) {
  gdn_linear_problem p;
  const gdn_status st = linear_problem_ok(pp, &p);
  if (st != GDN_OK) return st;
  if (!linear_inputs_ok(p, q, k, v, g, cu_seqlens)) return GDN_ERR_INVALID_ARG;
  const void* a16[] = {h0, dht, dh0, dout, dq, dk, dv};
  for (const void* x : a16)
    if (!aligned(x, 16)) return GDN_ERR_INVALID_ARG;
  if ((int64_t)p.B * p.T > 0 && (!dout || !dq || !dk || !dv || !dg)) return GDN_ERR_INVALID_ARG;
  if (p.g_per_head && !dg) return GDN_ERR_INVALID_ARG;
  if (!aligned(dg, 4) || !workspace || !aligned(workspace, kAlign) ||
      workspace_bytes < linear_bwd_workspace_bytes(p))
    return GDN_ERR_INVALID_ARG;
  return run_linear_bwd(p, q, k, v, g, scale, h0, cu_seqlens, dout, dht, dq, dk, dv, dg, dh0, workspace,
                        static_cast<cudaStream_t>(stream));
}

gdn_status gdn_selftest_linear_grads_timeout(const gdn_linear_problem* pp, const void* q, const void* k, const void* v,
                                             const float* g, float scale, const void* dout, void* dq, void* dk, void* dv,
                                             float* dg, void* workspace, size_t workspace_bytes, int batch,
                                             unsigned warps, void* stream) {
  gdn_linear_problem p;
  const gdn_status st = linear_problem_ok(pp, &p);
  if (st != GDN_OK) return st;
  if (p.dt != GDN_F32 || p.varlen || p.g_per_head || p.Hqk != p.Hv || p.K < 128 || p.V < 128 || batch < 0 || !warps)
    return GDN_ERR_UNSUPPORTED;
  if (!linear_inputs_ok(p, q, k, v, g, nullptr) || !dout || !dq || !dk || !dv || !dg) return GDN_ERR_INVALID_ARG;
  const void* a16[] = {dout, dq, dk, dv};
  for (const void* x : a16)
    if (!aligned(x, 16)) return GDN_ERR_INVALID_ARG;
  if (!aligned(dg, 4) || !workspace || !aligned(workspace, kAlign) || workspace_bytes < linear_bwd_workspace_bytes(p))
    return GDN_ERR_INVALID_ARG;
  return run_linear_bwd_drop(p, q, k, v, g, scale, dout, dq, dk, dv, dg, workspace, batch, warps,
                             static_cast<cudaStream_t>(stream));
}

gdn_status gdn_linear_attn_get_device_status(void* workspace, void* stream, int* dev_status) {
  if (!workspace || !dev_status) return GDN_ERR_INVALID_ARG;
  int32_t host = 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (cudaStreamSynchronize(s) != cudaSuccess) return GDN_ERR_CUDA;
  if (cudaMemcpy(&host, workspace, sizeof(host), cudaMemcpyDeviceToHost) != cudaSuccess) return GDN_ERR_CUDA;
  // on the call's stream and waited for: cudaMemset may still be under way on the default stream, which non-blocking
  // streams do not wait for, when the next call has left its word
  if (cudaMemsetAsync(workspace, 0, sizeof(host), s) != cudaSuccess) return GDN_ERR_CUDA;
  if (cudaStreamSynchronize(s) != cudaSuccess) return GDN_ERR_CUDA;
  *dev_status = host;
  return GDN_OK;
}

gdn_status gdn_linear_attn_step(const gdn_linear_problem* pp, const void* q, const void* k, const void* v,
                                const float* g, float scale, float* state, const int32_t* state_indices,
                                int state_slots, const int32_t* cu_seqlens, void* o, void* stream) {
  gdn_linear_problem p;
  const gdn_status st = linear_problem_ok(pp, &p);
  if (st != GDN_OK) return st;
  if (!linear_inputs_ok(p, q, k, v, g, cu_seqlens) || !aligned(o, 16)) return GDN_ERR_INVALID_ARG;
  if ((int64_t)p.B * p.T > 0 && !o) return GDN_ERR_INVALID_ARG;
  if (!state || !aligned(state, 16) || state_slots <= 0 || !aligned(state_indices, 4)) return GDN_ERR_INVALID_ARG;
  if (!state_indices && state_slots < p.N) return GDN_ERR_INVALID_ARG;
  return run_linear_step(p, q, k, v, g, scale, state, state_indices, state_slots, cu_seqlens, o,
                         static_cast<cudaStream_t>(stream));
}

namespace {

bool dtype_ok(gdn_dtype d) { return d == GDN_F32 || d == GDN_BF16; }
size_t size_of(gdn_dtype d) { return d == GDN_F32 ? 4 : 2; }

gdn_status gated_norm_ok(int64_t* ld_x, int64_t* ld_z, const void* x, const void* z, const float* weight, int rows,
                         int H, int V, gdn_dtype dt) {
  if (!dtype_ok(dt) || rows < 0 || H <= 0 || V <= 0) return GDN_ERR_INVALID_ARG;
  if (V > kNormMaxWidth || (int64_t)H * V >= ((int64_t)1 << 31) || (int64_t)rows * H >= ((int64_t)1 << 31) - 1024)
    return GDN_ERR_UNSUPPORTED;
  if (*ld_x == 0) *ld_x = (int64_t)H * V;
  if (*ld_z == 0) *ld_z = (int64_t)H * V;
  if (*ld_x < (int64_t)H * V || *ld_z < (int64_t)H * V) return GDN_ERR_INVALID_ARG;
  const size_t es = size_of(dt);
  if (!aligned(x, es) || !aligned(z, es) || !weight || !aligned(weight, 4)) return GDN_ERR_INVALID_ARG;
  return rows > 0 && !x ? GDN_ERR_INVALID_ARG : GDN_OK;
}

gdn_status residual_norm_ok(int64_t* ld_y, const void* y, const void* residual, const float* post_weight,
                            const void* gate, gdn_gate kind, const float* weight, int rows, int D, gdn_dtype dt,
                            gdn_dtype rdt) {
  if (!dtype_ok(dt) || !dtype_ok(rdt) || rows < 0 || D <= 0) return GDN_ERR_INVALID_ARG;
  if (dt == GDN_F32 && rdt != GDN_F32) return GDN_ERR_INVALID_ARG;
  if (kind != GDN_GATE_NONE && kind != GDN_GATE_CHANNEL && kind != GDN_GATE_ELEMENT) return GDN_ERR_INVALID_ARG;
  if (D > kNormMaxWidth || rows >= 0x7fffffff - 1024) return GDN_ERR_UNSUPPORTED;
  if (*ld_y == 0) *ld_y = D;
  if (*ld_y < D) return GDN_ERR_INVALID_ARG;
  if ((kind == GDN_GATE_NONE) != (gate == nullptr)) return GDN_ERR_INVALID_ARG;
  if (!aligned(y, size_of(dt)) || !aligned(residual, size_of(rdt)) || !aligned(post_weight, 4) ||
      !aligned(weight, 4) || !aligned(gate, kind == GDN_GATE_CHANNEL ? 4 : size_of(dt)))
    return GDN_ERR_INVALID_ARG;
  return rows > 0 && (!y || !residual) ? GDN_ERR_INVALID_ARG : GDN_OK;
}

}  // namespace

gdn_status gdn_gated_norm_fwd(const void* x, int64_t ld_x, const void* z, int64_t ld_z, const float* weight, int rows,
                              int H, int V, gdn_dtype dt, float eps, void* y, float* rstd, void* stream) {
  const gdn_status st = gated_norm_ok(&ld_x, &ld_z, x, z, weight, rows, H, V, dt);
  if (st != GDN_OK) return st;
  if ((rows > 0 && !y) || !aligned(y, size_of(dt)) || !aligned(rstd, 4)) return GDN_ERR_INVALID_ARG;
  if (rows == 0) return GDN_OK;
  return run_gated_norm_fwd(x, ld_x, z, ld_z, weight, rows, H, V, dt, eps, y, rstd, static_cast<cudaStream_t>(stream));
}

size_t gdn_gated_norm_bwd_workspace_size(int V) {
  return V > 0 && V <= kNormMaxWidth ? gated_norm_bwd_workspace_bytes(V) : 0;
}

gdn_status gdn_gated_norm_bwd(const void* x, int64_t ld_x, const void* z, int64_t ld_z, const float* weight,
                              const float* rstd, const void* dy, int rows, int H, int V, gdn_dtype dt, void* dx,
                              void* dz, float* dweight, void* workspace, size_t workspace_bytes, void* stream) {
  const gdn_status st = gated_norm_ok(&ld_x, &ld_z, x, z, weight, rows, H, V, dt);
  if (st != GDN_OK) return st;
  const size_t es = size_of(dt);
  if ((z == nullptr) != (dz == nullptr) || (rows > 0 && (!rstd || !dy || !dx)) || !dweight) return GDN_ERR_INVALID_ARG;
  if (!aligned(rstd, 4) || !aligned(dweight, 4) || !aligned(dy, es) || !aligned(dx, es) || !aligned(dz, es))
    return GDN_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, kAlign) || workspace_bytes < gated_norm_bwd_workspace_bytes(V))
    return GDN_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) return cudaMemsetAsync(dweight, 0, sizeof(float) * V, s) == cudaSuccess ? GDN_OK : GDN_ERR_CUDA;
  return run_gated_norm_bwd(x, ld_x, z, ld_z, weight, rstd, dy, rows, H, V, dt, dx, dz, dweight, workspace, s);
}

gdn_status gdn_residual_norm_fwd(const void* y, int64_t ld_y, const void* residual, const float* post_weight,
                                 const void* gate, gdn_gate gate_kind, float residual_scale, const float* weight,
                                 int rows, int D, gdn_dtype dt, gdn_dtype rdt, float eps, void* h, void* n,
                                 float* rstd, void* stream) {
  const gdn_status st = residual_norm_ok(&ld_y, y, residual, post_weight, gate, gate_kind, weight, rows, D, dt, rdt);
  if (st != GDN_OK) return st;
  if (rows == 0) return GDN_OK;
  if (!h || (weight == nullptr) != (n == nullptr)) return GDN_ERR_INVALID_ARG;
  if (!aligned(h, size_of(rdt)) || !aligned(n, size_of(dt)) || !aligned(rstd, 4)) return GDN_ERR_INVALID_ARG;
  return run_residual_norm_fwd(y, ld_y, residual, post_weight, gate, gate_kind, residual_scale, weight, rows, D, dt, rdt,
                               eps, h, n, rstd, static_cast<cudaStream_t>(stream));
}

size_t gdn_residual_norm_bwd_workspace_size(int D) {
  return D > 0 && D <= kNormMaxWidth ? residual_norm_bwd_workspace_bytes(D) : 0;
}

gdn_status gdn_residual_norm_bwd(const void* y, int64_t ld_y, const void* residual, const float* rstd, const void* dh,
                                 const void* dn, const float* post_weight, const void* gate, gdn_gate gate_kind,
                                 float residual_scale, const float* weight, int rows, int D, gdn_dtype dt,
                                 gdn_dtype rdt, void* dy, void* dresidual, float* dpost_weight, void* dgate,
                                 float* dweight, void* workspace, size_t workspace_bytes, void* stream) {
  const gdn_status st = residual_norm_ok(&ld_y, y, residual, post_weight, gate, gate_kind, weight, rows, D, dt, rdt);
  if (st != GDN_OK) return st;
  const size_t es = size_of(dt), er = size_of(rdt);
  if ((post_weight == nullptr) != (dpost_weight == nullptr) || (weight == nullptr) != (dweight == nullptr))
    return GDN_ERR_INVALID_ARG;
  if (!aligned(rstd, 4) || !aligned(dh, er) || !aligned(dn, es) || !aligned(dy, es) || !aligned(dresidual, er) ||
      !aligned(dpost_weight, 4) || !aligned(dweight, 4) || !aligned(dgate, gate_kind == GDN_GATE_CHANNEL ? 4 : es))
    return GDN_ERR_INVALID_ARG;
  if (!workspace || !aligned(workspace, kAlign) || workspace_bytes < residual_norm_bwd_workspace_bytes(D))
    return GDN_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {   // the sums over no rows
    float* sums[3] = {dpost_weight, dweight, gate_kind == GDN_GATE_CHANNEL ? static_cast<float*>(dgate) : nullptr};
    for (float* x : sums)
      if (x && cudaMemsetAsync(x, 0, sizeof(float) * D, s) != cudaSuccess) return GDN_ERR_CUDA;
    return GDN_OK;
  }
  if (!rstd || !dy || !dresidual || (weight == nullptr) != (dn == nullptr) || (gate == nullptr) != (dgate == nullptr))
    return GDN_ERR_INVALID_ARG;
  return run_residual_norm_bwd(y, ld_y, residual, rstd, dh, dn, post_weight, gate, gate_kind, residual_scale, weight,
                               rows, D, dt, rdt, dy, dresidual, dpost_weight, dgate, dweight, workspace, s);
}

const char* gdn_status_string(gdn_status s) {
  switch (s) {
    case GDN_OK: return "ok";
    case GDN_ERR_INVALID_ARG: return "invalid argument";
    case GDN_ERR_UNSUPPORTED: return "unsupported problem for this path";
    case GDN_ERR_CUDA: return "CUDA runtime error";
    case GDN_ERR_DEVICE: return "device reported an error";
    case GDN_ERR_SCRATCH_LIMIT: return "problem needs more than the built-in 32 MiB static scratch";
  }
  return "unknown status";
}

const char* gdn_version(void) { return "gdn 0.1 sm_103a"; }

}  // extern "C"

// ---------------------------------------------------------------------------
// Forward pass without any caller-provided or library-allocated device memory
// beyond the caller's inputs and outputs.
//
// Some callers cannot allocate device memory in the call path: an op embedded
// in a host framework that owns every device buffer and hands the op only its
// inputs and outputs (no workspace), or a caller that cannot afford the
// implicit device-wide synchronisation of cudaMalloc/cudaFree between its
// launches.  For them the forward pass runs with its workspace in one
// file-scope device array, kStaticScratchBytes (32 MiB) per GPU, which every
// GPU that loads this library holds until the process exits: the fused
// kernels whenever their workspace fits (a status word, the order table of a
// packed batch, or the window schedule's hand-over states: about 20 MB on 152
// SMs), else the staged path when its intermediates fit.  The first kAlign
// bytes of the array hold the status word of the last call (copied there from
// the workspace, which starts right after it), so that
// gdn_chunk_fwd_noalloc_get_device_status can read it without the problem.
#include <cudaTypedefs.h>
#include <mutex>

namespace {

constexpr size_t kStaticScratchBytes = size_t(32) << 20;
constexpr size_t kStaticStagedBytes = kStaticScratchBytes - kAlign;   // after the status slot
constexpr int kMaxDevices = 64;

static __device__ __align__(256) uint8_t g_static_scratch[kStaticScratchBytes];

std::mutex g_static_mu;
void* g_static_ptr[kMaxDevices] = {};
unsigned long long g_static_ctx[kMaxDevices] = {};   // context the cached address belongs to

// Unique id of the current CUDA context (0 when the driver cannot tell), through
// the driver entry points that the runtime hands out.
unsigned long long current_context_id() {
  static PFN_cuCtxGetCurrent_v4000 get_cur = nullptr;
  static PFN_cuCtxGetId_v12000 get_id = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &p, 4000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_cur = reinterpret_cast<PFN_cuCtxGetCurrent_v4000>(p);
    if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      get_id = reinterpret_cast<PFN_cuCtxGetId_v12000>(p);
  });
  if (!get_cur || !get_id) return 0;
  CUcontext ctx = nullptr;
  unsigned long long id = 0;
  if (get_cur(&ctx) != CUDA_SUCCESS || !ctx || get_id(ctx, &id) != CUDA_SUCCESS) return 0;
  return id;
}

// Device address of g_static_scratch on the current device.  The host-side
// name of the array is only a stand-in, so the address is fetched with
// cudaGetSymbolAddress (with that device current) once per device and
// context, and cached: a device reset that replaces the context makes the
// next call look the address up again.
gdn_status static_scratch(void** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return GDN_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return GDN_ERR_UNSUPPORTED;
  // 0 before the runtime has made the device's context current: then the
  // look-up below creates it, and the id is read again afterwards
  const unsigned long long ctx = current_context_id();
  std::lock_guard<std::mutex> lock(g_static_mu);
  if (!g_static_ptr[dev] || ctx == 0 || g_static_ctx[dev] != ctx) {
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_static_scratch) != cudaSuccess || !p) return GDN_ERR_CUDA;
    g_static_ptr[dev] = p;
    g_static_ctx[dev] = current_context_id();
  }
  *out = g_static_ptr[dev];
  return GDN_OK;
}

// The path of a gdn_chunk_fwd_noalloc call: AUTO's choice, with the fused
// kernel in place of the chunk-parallel path (whose per-segment states do
// not fit the array), when its workspace fits; else the staged path when its
// intermediates fit; GDN_PATH_AUTO when neither does.
gdn_path noalloc_path(const gdn_problem& p) {
  gdn_path path = resolve(p, GDN_PATH_AUTO);
  if (path == GDN_PATH_CP) path = GDN_PATH_FUSED;
  if (path != GDN_PATH_STAGED && workspace_for(p, path) <= kStaticStagedBytes) return path;
  if (workspace_for(p, GDN_PATH_STAGED) <= kStaticStagedBytes) return GDN_PATH_STAGED;
  return GDN_PATH_AUTO;
}

}  // namespace

extern "C" gdn_status gdn_chunk_fwd_noalloc(const gdn_problem* pp, const void* q, const void* k, const void* v,
                                            const float* g, const float* beta, float scale, const float* h0,
                                            const int32_t* cu_seqlens, void* o, float* ht, void* stream) {
  gdn_problem p;
  if (!problem_ok(pp, &p)) return GDN_ERR_INVALID_ARG;
  const gdn_path path = noalloc_path(p);
  if (path == GDN_PATH_AUTO) return GDN_ERR_SCRATCH_LIMIT;
  const size_t need = workspace_for(p, path);
  void* scratch = nullptr;
  gdn_status st = static_scratch(&scratch);
  if (st != GDN_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(scratch) + kAlign;
  st = check_call(p, q, k, v, g, beta, h0, cu_seqlens, o, ht, ws, kStaticStagedBytes, need);
  if (st != GDN_OK) return st;
  // each path clears the status word (and the window flags) it uses; every
  // other intermediate is rewritten before it is read, so stale contents of
  // earlier calls are harmless.
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (path == GDN_PATH_FUSED) st = run_fused(p, q, k, v, g, beta, scale, h0, cu_seqlens, o, ht, ws, s);
  else if (path == GDN_PATH_FUSED1) st = run_fused1(p, q, k, v, g, beta, scale, h0, cu_seqlens, o, ht, ws, s);
  else st = run_staged(p, 6, q, k, v, g, beta, scale, h0, cu_seqlens, o, ht, ws, s);
  if (st != GDN_OK) return st;
  // the call's status word goes to the fixed slot at the array's start
  if (cudaMemcpyAsync(scratch, ws + status_offset(p, path), sizeof(int32_t), cudaMemcpyDeviceToDevice, s) !=
      cudaSuccess)
    return GDN_ERR_CUDA;
  return GDN_OK;
}

extern "C" gdn_status gdn_chunk_fwd_noalloc_get_device_status(void* stream, int* dev_status) {
  if (!dev_status) return GDN_ERR_INVALID_ARG;
  void* scratch = nullptr;
  gdn_status st = static_scratch(&scratch);
  if (st != GDN_OK) return st;
  int32_t host = 0;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return GDN_ERR_CUDA;
  if (cudaMemcpy(&host, scratch, sizeof(host), cudaMemcpyDeviceToHost) != cudaSuccess) return GDN_ERR_CUDA;
  if (cudaMemset(scratch, 0, sizeof(int32_t)) != cudaSuccess) return GDN_ERR_CUDA;
  *dev_status = host;
  return GDN_OK;
}
