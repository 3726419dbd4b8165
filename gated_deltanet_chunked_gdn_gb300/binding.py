"""Thin ctypes binding over libgdn.so (include/gdn.h).

Argument marshalling only: tensors are checked for device, dtype, shape and
contiguity, outputs and the workspace are allocated with torch when the caller
does not pass them, and everything else runs in the library's CUDA kernels.
There is no CPU fallback: a missing library or a CPU tensor raises.
"""
from __future__ import annotations

import ctypes
import os
import threading
from dataclasses import dataclass
from typing import Optional

import torch

GDN_OK, GDN_ERR_INVALID_ARG, GDN_ERR_UNSUPPORTED, GDN_ERR_CUDA, GDN_ERR_DEVICE = range(5)
GDN_F32, GDN_BF16 = 0, 1
PATHS = {"auto": 0, "staged": 1, "fused": 2, "cp": 3, "fused1": 4}
PATH_NAMES = {v: k for k, v in PATHS.items()}
DEV_OK, DEV_BAD_CU_SEQLENS, DEV_WAIT_TIMEOUT = 0, 1, 2
STAGES = {"prepare": 0, "cumsum": 1, "kkt": 2, "solve_tril": 3, "wy_fast": 4, "chunk_h": 5, "chunk_o": 6}

EXPORTED = ["gdn_chunk_fwd_workspace_size", "gdn_chunk_fwd", "gdn_chunk_fwd_staged", "gdn_staged_layout",
            "gdn_get_device_status", "gdn_resolve_path", "gdn_status_string", "gdn_version", "gdn_recurrent_fwd",
            "gdn_causal_conv1d_fwd", "gdn_chunk_bwd_workspace_size", "gdn_chunk_bwd",
            "gdn_chunk_bwd_get_device_status", "gdn_chunk_fwd_host_workspace_size", "gdn_chunk_fwd_host",
            "gdn_chunk_fwd_host_get_device_status", "gdn_selective_scan_fwd_workspace_size",
            "gdn_selective_scan_fwd", "gdn_selective_scan_fwd_pool", "gdn_selective_scan_get_device_status", "gdn_selective_scan_step",
            "gdn_selective_scan_bwd_workspace_size", "gdn_selective_scan_bwd",
            "gdn_causal_conv1d_bwd_workspace_size", "gdn_causal_conv1d_bwd", "gdn_q4_matvec",
            "gdn_linear_attn_fwd_workspace_size", "gdn_linear_attn_fwd", "gdn_linear_attn_bwd_workspace_size",
            "gdn_linear_attn_bwd", "gdn_linear_attn_get_device_status", "gdn_linear_attn_step", "gdn_gated_norm_fwd",
            "gdn_gated_norm_bwd_workspace_size", "gdn_gated_norm_bwd", "gdn_residual_norm_fwd",
            "gdn_residual_norm_bwd_workspace_size", "gdn_residual_norm_bwd"]


class Problem(ctypes.Structure):
    _fields_ = [("B", ctypes.c_int), ("T", ctypes.c_int), ("N", ctypes.c_int), ("Hqk", ctypes.c_int),
                ("Hv", ctypes.c_int), ("K", ctypes.c_int), ("V", ctypes.c_int), ("C", ctypes.c_int),
                ("dt", ctypes.c_int), ("varlen", ctypes.c_int)]


class ScanProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "T", "N", "D", "S", "G", "dt", "varlen", "softplus")] + \
        [(n, ctypes.c_int64) for n in ("ld_x", "ld_delta", "ld_z", "ld_b", "ld_c")]


class LinearProblem(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("B", "T", "N", "Hqk", "Hv", "K", "V", "dt", "varlen", "g_per_head")] + \
        [(n, ctypes.c_int64) for n in ("ld_q", "ld_k", "ld_v")]


class StagedLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("tables", "status", "gamma", "A", "Tinv", "W", "U", "S0", "Vn",
                                               "total")] + [("nc_max", ctypes.c_int)]


class GDNError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_string(status)} ({status})")
        self.status = status


_lib = None
_lock = threading.Lock()


def library_path() -> str:
    return os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build", "libgdn.so")


def load(build_if_missing: bool = True) -> ctypes.CDLL:
    """Load libgdn.so (building it first if it is missing and nvcc exists)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = library_path()
        if not os.path.exists(path):
            if not build_if_missing:
                raise RuntimeError(f"libgdn.so not built ({path}); run __graft_entry__.build()")
            from . import build as _build
            _build.build()
        lib = ctypes.CDLL(path)
        P = ctypes.POINTER(Problem)
        vp, fp, i32p = ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p
        lib.gdn_chunk_fwd_workspace_size.argtypes = [P, ctypes.c_int]
        lib.gdn_chunk_fwd_workspace_size.restype = ctypes.c_size_t
        call = [P, ctypes.c_int, vp, vp, vp, fp, fp, ctypes.c_float, fp, i32p, vp, fp, vp, ctypes.c_size_t, vp]
        lib.gdn_chunk_fwd.argtypes = call
        lib.gdn_chunk_fwd.restype = ctypes.c_int
        lib.gdn_chunk_fwd_staged.argtypes = call
        lib.gdn_chunk_fwd_staged.restype = ctypes.c_int
        lib.gdn_staged_layout.argtypes = [P, ctypes.POINTER(StagedLayout)]
        lib.gdn_staged_layout.restype = ctypes.c_int
        lib.gdn_get_device_status.argtypes = [P, ctypes.c_int, vp, vp, ctypes.POINTER(ctypes.c_int)]
        lib.gdn_get_device_status.restype = ctypes.c_int
        lib.gdn_resolve_path.argtypes = [P]
        lib.gdn_resolve_path.restype = ctypes.c_int
        lib.gdn_status_string.argtypes = [ctypes.c_int]
        lib.gdn_status_string.restype = ctypes.c_char_p
        lib.gdn_recurrent_fwd.argtypes = [P, vp, vp, vp, fp, fp, fp, fp, ctypes.c_float, fp, i32p, ctypes.c_int,
                                          i32p, vp, vp]
        lib.gdn_recurrent_fwd.restype = ctypes.c_int
        lib.gdn_causal_conv1d_fwd.argtypes = [vp, fp, fp, ctypes.c_int, vp, ctypes.c_int, i32p, i32p, i32p,
                                              ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                              ctypes.c_int, vp, vp]
        lib.gdn_causal_conv1d_fwd.restype = ctypes.c_int
        lib.gdn_chunk_bwd_workspace_size.argtypes = [P]
        lib.gdn_chunk_bwd_workspace_size.restype = ctypes.c_size_t
        lib.gdn_chunk_bwd.argtypes = [P, vp, vp, vp, fp, fp, ctypes.c_float, fp, i32p, vp, fp, fp, fp, fp, fp, fp, fp,
                                      vp, ctypes.c_size_t, vp]
        lib.gdn_chunk_bwd.restype = ctypes.c_int
        lib.gdn_chunk_bwd_get_device_status.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_int)]
        lib.gdn_chunk_bwd_get_device_status.restype = ctypes.c_int
        lib.gdn_chunk_fwd_host_workspace_size.argtypes = [P, i32p, ctypes.c_int, ctypes.c_int]
        lib.gdn_chunk_fwd_host_workspace_size.restype = ctypes.c_size_t
        lib.gdn_chunk_fwd_host.argtypes = [P, ctypes.c_int, ctypes.c_int, vp, vp, vp, fp, fp, ctypes.c_float, fp, i32p,
                                           vp, fp, vp, ctypes.c_size_t, vp]
        lib.gdn_chunk_fwd_host.restype = ctypes.c_int
        lib.gdn_chunk_fwd_host_get_device_status.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_int)]
        lib.gdn_chunk_fwd_host_get_device_status.restype = ctypes.c_int
        SP = ctypes.POINTER(ScanProblem)
        lib.gdn_selective_scan_fwd_workspace_size.argtypes = [SP]
        lib.gdn_selective_scan_fwd_workspace_size.restype = ctypes.c_size_t
        lib.gdn_selective_scan_fwd.argtypes = [SP] + [vp] * 13 + [ctypes.c_size_t, vp]
        lib.gdn_selective_scan_fwd.restype = ctypes.c_int
        lib.gdn_selective_scan_fwd_pool.argtypes = [SP] + [vp] * 13 + [ctypes.c_int, vp, ctypes.c_size_t, vp]
        lib.gdn_selective_scan_fwd_pool.restype = ctypes.c_int
        lib.gdn_selective_scan_get_device_status.argtypes = [SP, vp, vp, ctypes.POINTER(ctypes.c_int)]
        lib.gdn_selective_scan_get_device_status.restype = ctypes.c_int
        lib.gdn_selective_scan_step.argtypes = [SP] + [vp] * 10 + [ctypes.c_int, vp, vp, vp]
        lib.gdn_selective_scan_step.restype = ctypes.c_int
        lib.gdn_selective_scan_bwd_workspace_size.argtypes = [SP]
        lib.gdn_selective_scan_bwd_workspace_size.restype = ctypes.c_size_t
        lib.gdn_selective_scan_bwd.argtypes = [SP] + [vp] * 22 + [ctypes.c_size_t, vp]
        lib.gdn_selective_scan_bwd.restype = ctypes.c_int
        lib.gdn_causal_conv1d_bwd_workspace_size.argtypes = [ctypes.c_int] * 4
        lib.gdn_causal_conv1d_bwd_workspace_size.restype = ctypes.c_size_t
        lib.gdn_causal_conv1d_bwd.argtypes = [vp, fp, fp, ctypes.c_int, vp, i32p] + [ctypes.c_int] * 6 + \
            [vp] * 7 + [ctypes.c_size_t, vp]
        lib.gdn_causal_conv1d_bwd.restype = ctypes.c_int
        lib.gdn_q4_matvec.argtypes = [vp, ctypes.c_int64, vp, vp, ctypes.c_int, vp, fp] + [ctypes.c_int] * 5 + [vp, vp]
        lib.gdn_q4_matvec.restype = ctypes.c_int
        LP, sz, i64, ci, cf = ctypes.POINTER(LinearProblem), ctypes.c_size_t, ctypes.c_int64, ctypes.c_int, ctypes.c_float
        for name, args in (("gdn_linear_attn_fwd", [LP, vp, vp, vp, vp, cf, vp, vp, vp, vp, vp, ci, vp, sz, vp]),
                           ("gdn_linear_attn_bwd", [LP, vp, vp, vp, vp, cf] + [vp] * 10 + [sz, vp]),
                           ("gdn_linear_attn_get_device_status", [vp, vp, ctypes.POINTER(ci)]),
                           ("gdn_linear_attn_step", [LP, vp, vp, vp, vp, cf, vp, vp, ci, vp, vp, vp]),
                           ("gdn_gated_norm_fwd", [vp, i64, vp, i64, vp, ci, ci, ci, ci, cf, vp, vp, vp]),
                           ("gdn_gated_norm_bwd", [vp, i64, vp, i64, vp, vp, vp] + [ci] * 4 + [vp] * 4 + [sz, vp]),
                           ("gdn_residual_norm_fwd", [vp, i64, vp, vp, vp, ci, cf, vp] + [ci] * 4 + [cf] + [vp] * 4),
                           ("gdn_residual_norm_bwd", [vp, i64, vp, vp, vp, vp, vp, vp, ci, cf, vp] + [ci] * 4 +
                            [vp] * 6 + [sz, vp])):
            getattr(lib, name).argtypes = args
            getattr(lib, name).restype = ci
        for name, args in (("gdn_linear_attn_fwd_workspace_size", [LP]), ("gdn_linear_attn_bwd_workspace_size", [LP]),
                           ("gdn_gated_norm_bwd_workspace_size", [ci]), ("gdn_residual_norm_bwd_workspace_size", [ci])):
            getattr(lib, name).argtypes = args
            getattr(lib, name).restype = sz
        lib.gdn_version.argtypes = []
        lib.gdn_version.restype = ctypes.c_char_p
        _lib = lib
        return lib


def status_string(s: int) -> str:
    return load().gdn_status_string(int(s)).decode()


def gdn_version() -> str:
    return load().gdn_version().decode()


@dataclass
class Shapes:
    B: int
    T: int
    N: int
    Hqk: int
    Hv: int
    K: int
    V: int


def problem(B, T, N, Hqk, Hv, K, V, C, dtype, varlen) -> Problem:
    dt = GDN_F32 if dtype in (torch.float32, "f32", GDN_F32) else GDN_BF16
    return Problem(int(B), int(T), int(N), int(Hqk), int(Hv), int(K), int(V), int(C), dt, int(bool(varlen)))


def problem_of(q, v, C, cu_seqlens=None) -> Problem:
    B, T, Hqk, K = q.shape
    Hv, V = v.shape[2], v.shape[3]
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else B
    return problem(B, T, N, Hqk, Hv, K, V, C, q.dtype, cu_seqlens is not None)


def gdn_chunk_fwd_workspace_size(p: Problem, path: str = "auto") -> int:
    return int(load().gdn_chunk_fwd_workspace_size(ctypes.byref(p), PATHS[path]))


def gdn_resolve_path(p: Problem) -> str:
    return PATH_NAMES[int(load().gdn_resolve_path(ctypes.byref(p)))]


def gdn_staged_layout(p: Problem) -> StagedLayout:
    out = StagedLayout()
    st = load().gdn_staged_layout(ctypes.byref(p), ctypes.byref(out))
    if st:
        raise GDNError(st, "gdn_staged_layout")
    return out


def _ptr(t: Optional[torch.Tensor]):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else ctypes.c_void_p()


def _check_inputs(q, k, v, g, beta, h0, cu_seqlens):
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("h0", h0), ("cu_seqlens", cu_seqlens)):
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor (the library has no CPU path)")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    if q.dtype not in (torch.float32, torch.bfloat16) or k.dtype != q.dtype or v.dtype != q.dtype:
        raise ValueError("q, k, v must share one dtype, float32 or bfloat16")
    for name, t in (("g", g), ("beta", beta), ("h0", h0)):
        if t is not None and t.dtype != torch.float32:
            raise ValueError(f"{name} must be float32")
    if cu_seqlens is not None and cu_seqlens.dtype != torch.int32:
        raise ValueError("cu_seqlens must be int32")
    B, T, Hqk, K = q.shape
    Hv, V = v.shape[2], v.shape[3]
    if k.shape != q.shape or v.shape[:2] != (B, T) or g.shape != (B, T, Hv) or beta.shape != (B, T, Hv):
        raise ValueError("shape mismatch among q, k, v, g, beta")
    N = (cu_seqlens.numel() - 1) if cu_seqlens is not None else B
    if h0 is not None and h0.shape != (N, Hv, K, V):
        raise ValueError(f"h0 must be [N, Hv, K, V] = {(N, Hv, K, V)}")


def _alloc_ws(nbytes: int, device) -> torch.Tensor:
    # torch's caching allocator returns 512-byte aligned blocks.
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def gdn_chunk_fwd(q, k, v, g, beta, scale: Optional[float] = None, h0=None, cu_seqlens=None, C: int = 64,
                  path: str = "auto", o=None, ht=None, output_final_state: bool = True, workspace=None,
                  stream=None):
    """Chunked Gated DeltaNet forward.  Returns (o, ht); ht is None when
    ``output_final_state`` is False.  ``scale`` defaults to K ** -0.5."""
    lib = load()
    _check_inputs(q, k, v, g, beta, h0, cu_seqlens)
    p = problem_of(q, v, C, cu_seqlens)
    if scale is None:
        scale = q.shape[-1] ** -0.5
    given = o, ht, workspace
    if o is None:
        o = torch.empty_like(v)
    if ht is None and output_final_state:
        ht = torch.empty((p.N, p.Hv, p.K, p.V), dtype=torch.float32, device=q.device)
    need = gdn_chunk_fwd_workspace_size(p, path)
    if need == 0:
        raise GDNError(GDN_ERR_UNSUPPORTED if path in ("fused", "cp", "fused1") else GDN_ERR_INVALID_ARG, "gdn_chunk_fwd_workspace_size")
    if workspace is None:
        workspace = _alloc_ws(need, q.device)
    if stream is not None:
        _lend(stream, q.device, [t for t, g in zip((o, ht, workspace), given) if g is None])
    s = stream if stream is not None else torch.cuda.current_stream(q.device).cuda_stream
    st = lib.gdn_chunk_fwd(ctypes.byref(p), PATHS[path], _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                           ctypes.c_float(scale), _ptr(h0), _ptr(cu_seqlens), _ptr(o), _ptr(ht), _ptr(workspace),
                           ctypes.c_size_t(workspace.numel()), ctypes.c_void_p(s))
    if st:
        raise GDNError(st, "gdn_chunk_fwd")
    return o, ht


def gdn_chunk_fwd_host_workspace_size(p: Problem, cu_seqlens=None, nsplit: int = 4, path: str = "auto") -> int:
    return int(load().gdn_chunk_fwd_host_workspace_size(ctypes.byref(p), _ptr(cu_seqlens), int(nsplit), PATHS[path]))


def gdn_chunk_fwd_host(q, k, v, g, beta, scale: Optional[float] = None, h0=None, cu_seqlens=None, C: int = 64,
                       path: str = "auto", nsplit: int = 4, o=None, ht=None, output_final_state: bool = True,
                       workspace=None, device=None, stream=None):
    """The forward pass on host (CPU) tensors, streamed through the GPU in
    ``nsplit`` sub-batches (pin the tensors for the copies to overlap the
    compute).  Returns host (o, ht) after the call has finished; ht is None
    when ``output_final_state`` is False."""
    lib = load()
    for name, t in (("q", q), ("k", k), ("v", v), ("g", g), ("beta", beta), ("h0", h0), ("cu_seqlens", cu_seqlens)):
        if t is not None and (t.device.type != "cpu" or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous host tensor")
    p = problem_of(q, v, C, cu_seqlens)
    if scale is None:
        scale = q.shape[-1] ** -0.5
    pin = q.is_pinned()
    if o is None:
        o = torch.empty(v.shape, dtype=v.dtype, pin_memory=pin)
    if ht is None and output_final_state:
        ht = torch.empty((p.N, p.Hv, p.K, p.V), dtype=torch.float32, pin_memory=pin)
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    need = gdn_chunk_fwd_host_workspace_size(p, cu_seqlens, nsplit, path)
    if need == 0:
        raise GDNError(GDN_ERR_INVALID_ARG, "gdn_chunk_fwd_host_workspace_size")
    if workspace is None:
        workspace = _alloc_ws(need, dev)
        if stream is not None:
            _lend(stream, dev, (workspace,))
    s = stream if stream is not None else torch.cuda.current_stream(dev).cuda_stream
    st = lib.gdn_chunk_fwd_host(ctypes.byref(p), PATHS[path], int(nsplit), _ptr(q), _ptr(k), _ptr(v), _ptr(g),
                                _ptr(beta), ctypes.c_float(scale), _ptr(h0), _ptr(cu_seqlens), _ptr(o), _ptr(ht),
                                _ptr(workspace), ctypes.c_size_t(workspace.numel()), ctypes.c_void_p(s))
    if st:
        raise GDNError(st, "gdn_chunk_fwd_host")
    torch.cuda.synchronize(dev)
    return o, ht


def gdn_chunk_fwd_host_get_device_status(workspace, stream=None) -> int:
    out = ctypes.c_int(0)
    s = stream if stream is not None else torch.cuda.current_stream(workspace.device).cuda_stream
    st = load().gdn_chunk_fwd_host_get_device_status(_ptr(workspace), ctypes.c_void_p(s), ctypes.byref(out))
    if st:
        raise GDNError(st, "gdn_chunk_fwd_host_get_device_status")
    return out.value


def gdn_chunk_fwd_staged(q, k, v, g, beta, scale: Optional[float] = None, h0=None, cu_seqlens=None, C: int = 64,
                         stop_after: int | str = 6, workspace=None, stream=None):
    """Staged path up to ``stop_after``; returns (o, ht, workspace, layout)."""
    lib = load()
    _check_inputs(q, k, v, g, beta, h0, cu_seqlens)
    p = problem_of(q, v, C, cu_seqlens)
    if scale is None:
        scale = q.shape[-1] ** -0.5
    stop = STAGES[stop_after] if isinstance(stop_after, str) else int(stop_after)
    layout = gdn_staged_layout(p)
    given = workspace
    o = torch.zeros_like(v)
    ht = torch.zeros((p.N, p.Hv, p.K, p.V), dtype=torch.float32, device=q.device)
    if workspace is None:
        workspace = _alloc_ws(layout.total, q.device)
    if stream is not None:
        _lend(stream, q.device, (o, ht, workspace if given is None else None))
    s = stream if stream is not None else torch.cuda.current_stream(q.device).cuda_stream
    st = lib.gdn_chunk_fwd_staged(ctypes.byref(p), stop, _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta),
                                  ctypes.c_float(scale), _ptr(h0), _ptr(cu_seqlens), _ptr(o), _ptr(ht),
                                  _ptr(workspace), ctypes.c_size_t(workspace.numel()), ctypes.c_void_p(s))
    if st:
        raise GDNError(st, "gdn_chunk_fwd_staged")
    return o, ht, workspace, layout


def staged_view(workspace: torch.Tensor, layout: StagedLayout, p: Problem, name: str) -> torch.Tensor:
    """A typed view of one staged intermediate inside ``workspace``."""
    nc, H, C, K, V = layout.nc_max, p.Hv, p.C, p.K, p.V
    shapes = {"gamma": (nc, H, C), "A": (nc, H, C, C), "Tinv": (nc, H, C, C), "W": (nc, H, C, K),
              "U": (nc, H, C, V), "S0": (nc, H, K, V), "Vn": (nc, H, C, V)}
    if name == "tables":
        n = p.N + 1 + 3 * nc + 1
        t = workspace[layout.tables: layout.tables + 4 * n].view(torch.int32)
        return {"seq_chunk0": t[: p.N + 1], "chunk_seq": t[p.N + 1: p.N + 1 + nc],
                "chunk_tok0": t[p.N + 1 + nc: p.N + 1 + 2 * nc], "chunk_len": t[p.N + 1 + 2 * nc: p.N + 1 + 3 * nc],
                "nc": t[-1:]}
    shape = shapes[name]
    off = getattr(layout, name)
    numel = 1
    for d in shape:
        numel *= d
    return workspace[off: off + 4 * numel].view(torch.float32).view(shape)


def gdn_get_device_status(p: Problem, path: str, workspace: torch.Tensor, stream=None) -> int:
    out = ctypes.c_int(0)
    s = stream if stream is not None else torch.cuda.current_stream(workspace.device).cuda_stream
    st = load().gdn_get_device_status(ctypes.byref(p), PATHS[path], _ptr(workspace), ctypes.c_void_p(s),
                                      ctypes.byref(out))
    if st:
        raise GDNError(st, "gdn_get_device_status")
    return int(out.value)


def chunk_gated_delta_rule(q, k, v, g, beta, scale=None, initial_state=None, output_final_state=True,
                           cu_seqlens=None, chunk_size: int = 64):
    """Framework-style entry: (o, final_state) like the pages' integration call."""
    return gdn_chunk_fwd(q, k, v, g, beta, scale=scale, h0=initial_state, cu_seqlens=cu_seqlens, C=chunk_size,
                         output_final_state=output_final_state)


def gdn_recurrent_fwd(q, k, v, a, b, A_log, state, dt_bias=None, scale: Optional[float] = None,
                      state_indices=None, cu_seqlens=None, o=None, stream=None):
    """Fused gated recurrent (decode) step.  ``state`` [slots, Hv, K, V] fp32 is
    updated in place; returns o.  g = -exp(A_log) softplus(a + dt_bias),
    beta = sigmoid(b), then the gated delta rule token by token."""
    lib = load()
    for name, t in (("q", q), ("k", k), ("v", v), ("a", a), ("b", b), ("A_log", A_log), ("state", state),
                    ("dt_bias", dt_bias), ("state_indices", state_indices), ("cu_seqlens", cu_seqlens)):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    for name, t in (("a", a), ("b", b), ("A_log", A_log), ("state", state), ("dt_bias", dt_bias)):
        if t is not None and t.dtype != torch.float32:
            raise ValueError(f"{name} must be float32")
    p = problem_of(q, v, 64, cu_seqlens)
    if scale is None:
        scale = q.shape[-1] ** -0.5
    if o is None:
        o = torch.empty_like(v)
        if stream is not None:
            _lend(stream, q.device, (o,))
    s = stream if stream is not None else torch.cuda.current_stream(q.device).cuda_stream
    st = lib.gdn_recurrent_fwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(a), _ptr(b), _ptr(A_log),
                               _ptr(dt_bias), ctypes.c_float(scale), _ptr(state), _ptr(state_indices),
                               int(state.shape[0]), _ptr(cu_seqlens), _ptr(o), ctypes.c_void_p(s))
    if st:
        raise GDNError(st, "gdn_recurrent_fwd")
    return o


ACTIVATIONS = {None: 0, "none": 0, "silu": 1}
DTYPES = {torch.float32: GDN_F32, torch.bfloat16: GDN_BF16}


def gdn_causal_conv1d_fwd(x, weight, bias=None, activation="silu", conv_state=None, cache_indices=None,
                          has_initial_state=None, cu_seqlens=None, y=None, stream=None):
    """Causal depthwise convolution with a carried state.  x [B, T, D] (bf16
    or fp32; packed with cu_seqlens when B == 1), weight [D, W] fp32, bias [D]
    fp32.  ``conv_state`` [slots, W-1, D] (dtype of x) is read and then
    updated in place; returns y (shape and dtype of x)."""
    lib = load()
    for name, t in (("x", x), ("weight", weight), ("bias", bias), ("conv_state", conv_state),
                    ("cache_indices", cache_indices), ("has_initial_state", has_initial_state),
                    ("cu_seqlens", cu_seqlens)):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None and t.dtype != torch.float32:
            raise ValueError(f"{name} must be float32")
    for name, t in (("cache_indices", cache_indices), ("has_initial_state", has_initial_state),
                    ("cu_seqlens", cu_seqlens)):
        if t is not None and t.dtype != torch.int32:
            raise ValueError(f"{name} must be int32")
    if x.dtype not in DTYPES:
        raise ValueError("x must be float32 or bfloat16")
    if conv_state is not None and conv_state.dtype != x.dtype:
        raise ValueError("conv_state must have the dtype of x")
    B, T, D = x.shape
    W = int(weight.shape[1])
    N = int(cu_seqlens.numel()) - 1 if cu_seqlens is not None else B
    if y is None:
        y = torch.empty_like(x)
        if stream is not None:
            _lend(stream, x.device, (y,))
    slots = int(conv_state.shape[0]) if conv_state is not None else 0
    s = stream if stream is not None else torch.cuda.current_stream(x.device).cuda_stream
    st = lib.gdn_causal_conv1d_fwd(_ptr(x), _ptr(weight), _ptr(bias), W, _ptr(conv_state), slots,
                                   _ptr(cache_indices), _ptr(has_initial_state), _ptr(cu_seqlens), N, B, T, D,
                                   DTYPES[x.dtype], ACTIVATIONS[activation], _ptr(y), ctypes.c_void_p(s))
    if st:
        raise GDNError(st, "gdn_causal_conv1d_fwd")
    return y


def gdn_chunk_bwd_workspace_size(p: Problem) -> int:
    return int(load().gdn_chunk_bwd_workspace_size(ctypes.byref(p)))


def gdn_chunk_bwd(q, k, v, g, beta, dout, scale: Optional[float] = None, h0=None, dht=None, cu_seqlens=None,
                  want_dh0: bool = True, workspace=None, stream=None) -> dict:
    """Backward of gdn_chunk_fwd for upstream gradients ``dout`` (dL/do, dtype of v)
    and ``dht`` (dL/dht, fp32 or None).  Returns fp32 gradients dq, dk
    [B,T,Hqk,K], dv [B,T,Hv,V], dg, dbeta [B,T,Hv] and dh0 [N,Hv,K,V] (None
    unless ``want_dh0``), plus the workspace under "workspace"."""
    lib = load()
    _check_inputs(q, k, v, g, beta, h0, cu_seqlens)
    for name, t in (("dout", dout), ("dht", dht)):
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous CUDA tensor")
    if dout.dtype != v.dtype or dout.shape != v.shape:
        raise ValueError("dout must match v in shape and dtype")
    if dht is not None and dht.dtype != torch.float32:
        raise ValueError("dht must be float32")
    p = problem_of(q, v, 64, cu_seqlens)
    if scale is None:
        scale = q.shape[-1] ** -0.5
    need = gdn_chunk_bwd_workspace_size(p)
    if need == 0:
        raise GDNError(GDN_ERR_UNSUPPORTED, "gdn_chunk_bwd_workspace_size")
    given = workspace
    if workspace is None:
        workspace = _alloc_ws(need, q.device)
    f32 = dict(dtype=torch.float32, device=q.device)
    out = {"dq": torch.empty(q.shape, **f32), "dk": torch.empty(k.shape, **f32), "dv": torch.empty(v.shape, **f32),
           "dg": torch.empty(g.shape, **f32), "dbeta": torch.empty(beta.shape, **f32),
           "dh0": torch.empty((p.N, p.Hv, p.K, p.V), **f32) if want_dh0 else None}
    if stream is not None:
        _lend(stream, q.device, (*out.values(), workspace if given is None else None))
    s = stream if stream is not None else torch.cuda.current_stream(q.device).cuda_stream
    st = lib.gdn_chunk_bwd(ctypes.byref(p), _ptr(q), _ptr(k), _ptr(v), _ptr(g), _ptr(beta), ctypes.c_float(scale),
                           _ptr(h0), _ptr(cu_seqlens), _ptr(dout), _ptr(dht), _ptr(out["dq"]), _ptr(out["dk"]),
                           _ptr(out["dv"]), _ptr(out["dg"]), _ptr(out["dbeta"]), _ptr(out["dh0"]),
                           _ptr(workspace), ctypes.c_size_t(workspace.numel()), ctypes.c_void_p(s))
    if st:
        raise GDNError(st, "gdn_chunk_bwd")
    out["workspace"] = workspace
    return out


def gdn_chunk_bwd_get_device_status(workspace, stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream(workspace.device).cuda_stream
    v = ctypes.c_int(0)
    st = load().gdn_chunk_bwd_get_device_status(_ptr(workspace), ctypes.c_void_p(s), ctypes.byref(v))
    if st:
        raise GDNError(st, "gdn_chunk_bwd_get_device_status")
    return int(v.value)


def _address(t: Optional[torch.Tensor]) -> int:
    return t.data_ptr() if t is not None else 0


try:   # the current stream's handle without a Stream object around it
    _current_stream = torch._C._cuda_getCurrentRawStream
except AttributeError:
    def _current_stream(index: int) -> int:
        return torch.cuda.current_stream(index).cuda_stream


try:
    _current_device = torch._C._cuda_getDevice
except AttributeError:
    def _current_device() -> int:
        return torch.cuda.current_device()


def _call(dev: int, fn, *args):
    """fn(*args) with the device current that it launches on."""
    if _current_device() == dev:
        return fn(*args)
    with torch.cuda.device(dev):
        return fn(*args)


def _check_ws(workspace, x) -> None:
    if workspace is not None and workspace.device != x.device:
        raise ValueError("workspace must be on the device of x")


def _lend(stream: int, device, blocks) -> None:
    """Hands blocks that a call has allocated (None among them) to the stream that it runs on.  They come from the
    current stream's pool, where work queued earlier may still use their memory and where they return when they are
    dropped: another stream waits for that work, and the memory is not given out again before it is done."""
    blocks = [b for b in blocks if b is not None]
    if not blocks or stream == _current_stream(blocks[0].get_device()):
        return
    other = torch.cuda.ExternalStream(stream, device=device)
    other.wait_stream(torch.cuda.current_stream(device))
    for b in blocks:
        b.record_stream(other)


def _row_stride(name: str, t: torch.Tensor, row: int) -> int:
    """Elements from one token's row of t [B, T, ...] to the next; the rows themselves contiguous, the
    sequences of a batch one after the other at the same stride."""
    if t.is_contiguous():
        return row
    B, T = t.shape[:2]
    ld = t.stride(1) if T > 1 else t.stride(0) if B > 1 else row
    inner, ok = 1, True
    for i in range(t.dim() - 1, 1, -1):
        ok = ok and (t.shape[i] == 1 or t.stride(i) == inner)
        inner *= t.shape[i]
    if not ok or ld < row or (B > 1 and T > 1 and t.stride(0) != T * ld):
        raise ValueError(f"{name} must have contiguous rows, one token after the other at one stride")
    return ld


def _scan_problem(x, delta, A, B, C, D, z, dt_bias, softplus, cu_seqlens, fp32=(), others=()):
    """Checks of a scan's tensors and its problem.  fp32: (name, tensor, shape) that must be contiguous float32;
    others: (name, tensor) that must be like x and contiguous."""
    # the usual call, all rows contiguous, in one expression: a decode step's launch is shorter than its checks
    dtype, shape, dev = x.dtype, x.shape, x.get_device()
    if len(shape) == 3 and B.dim() == 4 and dev >= 0 and dtype in DTYPES:
        nb, T, d = shape
        _, _, G, S = bshape = B.shape
        f32 = torch.float32
        if (x.is_contiguous() and delta.is_contiguous() and B.is_contiguous() and C.is_contiguous()
                and A.is_contiguous() and delta.shape == shape and C.shape == bshape and bshape[0] == nb
                and bshape[1] == T and A.shape == (d, S) and delta.dtype is dtype and B.dtype is dtype
                and C.dtype is dtype and A.dtype is f32 and delta.get_device() == dev and B.get_device() == dev
                and C.get_device() == dev and A.get_device() == dev
                and (z is None or (z.shape == shape and z.dtype is dtype and z.get_device() == dev
                                   and z.is_contiguous()))
                and (D is None or (D.shape == (d,) and D.dtype is f32 and D.get_device() == dev
                                   and D.is_contiguous()))
                and (dt_bias is None or (dt_bias.shape == (d,) and dt_bias.dtype is f32
                                         and dt_bias.get_device() == dev and dt_bias.is_contiguous()))):
            for _, t, want in fp32:
                if t is not None and (t.dtype is not f32 or t.get_device() != dev or t.shape != want
                                      or not t.is_contiguous()):
                    break
            else:
                if cu_seqlens is None and not others:
                    return ScanProblem(nb, T, nb, d, S, G, DTYPES[dtype], 0, 1 if softplus else 0)
    return _scan_problem_checked(x, delta, A, B, C, D, z, dt_bias, softplus, cu_seqlens, fp32, others)


def _scan_problem_checked(x, delta, A, B, C, D, z, dt_bias, softplus, cu_seqlens, fp32, others):
    dtype, shape = x.dtype, x.shape
    if dtype not in DTYPES:
        raise ValueError("x must be float32 or bfloat16")
    if len(shape) != 3 or B.dim() != 4:
        raise ValueError("x must be [B, T, D] and B [B, T, G, S]")
    nb, T, d = shape
    G, S = B.shape[2], B.shape[3]
    if delta.shape != shape or (z is not None and z.shape != shape):
        raise ValueError("delta and z must have the shape of x")
    if C.shape != B.shape or B.shape[:2] != shape[:2] or A.shape != (d, S):
        raise ValueError("B and C must be [B, T, G, S] and A [D, S]")
    for name, t in (("x", x), ("delta", delta), ("B", B), ("C", C), ("z", z), *others):
        if t is not None and (t.dtype != dtype or not t.is_cuda or t.device != x.device):
            raise ValueError(f"{name} must be a CUDA tensor with the dtype and device of x")
    for name, t in others:
        if t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous with the shape of x")
    for name, t, want in (("A", A, (d, S)), ("D", D, (d,)), ("dt_bias", dt_bias, (d,)), *fp32):
        if t is not None and (t.dtype != torch.float32 or t.shape != want or t.device != x.device
                              or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous float32 CUDA tensor of shape {tuple(want)}")
    N = nb
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.device != x.device or not cu_seqlens.is_contiguous():
            raise ValueError("cu_seqlens must be a contiguous int32 CUDA tensor")
        N = cu_seqlens.numel() - 1
    gs = G * S
    return ScanProblem(nb, T, N, d, S, G, DTYPES[dtype], int(cu_seqlens is not None), int(bool(softplus)),
                       _row_stride("x", x, d), _row_stride("delta", delta, d),
                       _row_stride("z", z, d) if z is not None else 0, _row_stride("B", B, gs),
                       _row_stride("C", C, gs))


def _scan_sequences(x, cu_seqlens) -> int:
    return cu_seqlens.numel() - 1 if cu_seqlens is not None else x.shape[0]


def gdn_selective_scan_fwd(x, delta, A, B, C, D=None, z=None, dt_bias=None, softplus: bool = True, h0=None,
                           cu_seqlens=None, y=None, ht=None, output_final_state: bool = True, workspace=None,
                           stream=None, state_indices=None):
    """Selective state space scan.  x, delta, z [B, T, D], B and C [B, T, G, S] (one dtype, bf16 or fp32; rows
    may be slices of wider rows), A [D, S], D and dt_bias [D], h0 [N, D, S] fp32.  Returns (y, ht); ht is None
    when ``output_final_state`` is False.  With ``state_indices`` [N] int32, ht is a pool [slots, D, S] whose rows
    they are (outside the pool: the sequence keeps no state)."""
    lib = _lib or load()
    _check_ws(workspace, x)
    state = (_scan_sequences(x, cu_seqlens), x.shape[-1], A.shape[-1])
    rows = state
    if state_indices is not None:
        if (ht is None or ht.dim() != 3 or ht.shape[0] == 0 or state_indices.dtype is not torch.int32
                or state_indices.device != x.device or not state_indices.is_contiguous()
                or state_indices.numel() != state[0]):
            raise ValueError("state_indices must be a contiguous int32 CUDA tensor, one row of the pool ht "
                             "[slots, D, S] a sequence")
        rows = (ht.shape[0], *state[1:])
    p = _scan_problem(x, delta, A, B, C, D, z, dt_bias, softplus, cu_seqlens, (("h0", h0, state), ("ht", ht, rows)),
                      (("y", y),) if y is not None else ())
    given = y, ht, workspace
    if y is None:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
    if ht is None and output_final_state:
        ht = torch.empty(state, dtype=torch.float32, device=x.device)
    if workspace is None:
        need = lib.gdn_selective_scan_fwd_workspace_size(p)
        if need == 0:
            raise GDNError(GDN_ERR_UNSUPPORTED, "gdn_selective_scan_fwd_workspace_size")
        workspace = _alloc_ws(need, x.device)
    if stream is not None:
        _lend(stream, x.device, [t for t, g in zip((y, ht, workspace), given) if g is None])
    s = stream if stream is not None else _current_stream(x.get_device())
    call = (p, x.data_ptr(), delta.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(), _address(D), _address(z),
            _address(dt_bias), _address(h0), _address(cu_seqlens), y.data_ptr(), _address(ht))
    if state_indices is None:
        st = lib.gdn_selective_scan_fwd(*call, workspace.data_ptr(), workspace.numel(), s)
    else:
        st = lib.gdn_selective_scan_fwd_pool(*call, state_indices.data_ptr(), rows[0], workspace.data_ptr(),
                                             workspace.numel(), s)
    if st:
        raise GDNError(st, "gdn_selective_scan_fwd")
    return y, ht


def gdn_selective_scan_fwd_workspace_size(p: ScanProblem) -> int:
    return int(load().gdn_selective_scan_fwd_workspace_size(ctypes.byref(p)))


def gdn_selective_scan_get_device_status(p: ScanProblem, workspace, stream=None) -> int:
    s = stream if stream is not None else torch.cuda.current_stream(workspace.device).cuda_stream
    v = ctypes.c_int(0)
    st = load().gdn_selective_scan_get_device_status(ctypes.byref(p), workspace.data_ptr(), s, ctypes.byref(v))
    if st:
        raise GDNError(st, "gdn_selective_scan_get_device_status")
    return int(v.value)


def gdn_selective_scan_step(x, delta, A, B, C, state, D=None, z=None, dt_bias=None, softplus: bool = True,
                            state_indices=None, cu_seqlens=None, y=None, stream=None):
    """The scan's tokens on a state pool (decode).  ``state`` [slots, D, S] fp32 is updated in place; returns y."""
    lib = _lib or load()
    slots, d, S = state.shape
    p = _scan_problem(x, delta, A, B, C, D, z, dt_bias, softplus, cu_seqlens, (),
                      (("y", y),) if y is not None else ())
    dev = x.get_device()
    if (state.dtype is not torch.float32 or d != x.shape[-1] or S != A.shape[-1] or state.get_device() != dev
            or not state.is_contiguous()):
        raise ValueError("state must be a contiguous float32 CUDA tensor [slots, D, S]")
    idx = 0
    if state_indices is not None:
        if (state_indices.dtype is not torch.int32 or state_indices.get_device() != dev
                or not state_indices.is_contiguous() or state_indices.numel() != p.N):
            raise ValueError("state_indices must be a contiguous int32 CUDA tensor, one slot a sequence")
        idx = state_indices.data_ptr()
    if y is None:
        y = torch.empty_like(x) if x.is_contiguous() else torch.empty(x.shape, dtype=x.dtype, device=x.device)
        if stream is not None:
            _lend(stream, x.device, (y,))
    st = lib.gdn_selective_scan_step(p, x.data_ptr(), delta.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(),
                                     0 if D is None else D.data_ptr(), 0 if z is None else z.data_ptr(),
                                     0 if dt_bias is None else dt_bias.data_ptr(), state.data_ptr(), idx, slots,
                                     0 if cu_seqlens is None else cu_seqlens.data_ptr(), y.data_ptr(),
                                     _current_stream(dev) if stream is None else stream)
    if st:
        raise GDNError(st, "gdn_selective_scan_step")
    return y


def gdn_selective_scan_bwd_workspace_size(p: ScanProblem) -> int:
    return int(load().gdn_selective_scan_bwd_workspace_size(ctypes.byref(p)))


def gdn_selective_scan_bwd(x, delta, A, B, C, dout, D=None, z=None, dt_bias=None, softplus: bool = True, h0=None,
                           dht=None, cu_seqlens=None, want_dh0: Optional[bool] = None, workspace=None,
                           stream=None) -> dict:
    """Backward of gdn_selective_scan_fwd for upstream gradients ``dout`` (dL/dy, dtype of x) and ``dht`` (dL/dht,
    fp32 or None).  Returns dx, ddelta, dB, dC, dz (dtype of x), dA, dD, ddt_bias, dh0 (fp32) and the workspace
    under "workspace"; dD, dz and ddt_bias are None where the input is, dh0 unless ``want_dh0`` (by default: h0 is
    given)."""
    lib = _lib or load()
    _check_ws(workspace, x)
    state = (_scan_sequences(x, cu_seqlens), x.shape[-1], A.shape[-1])
    p = _scan_problem(x, delta, A, B, C, D, z, dt_bias, softplus, cu_seqlens,
                      (("h0", h0, state), ("dht", dht, state)), (("dout", dout),))
    given = workspace
    if workspace is None:
        need = lib.gdn_selective_scan_bwd_workspace_size(p)
        if need == 0:
            raise GDNError(GDN_ERR_UNSUPPORTED, "gdn_selective_scan_bwd_workspace_size")
        workspace = _alloc_ws(need, x.device)
    like = dict(dtype=x.dtype, device=x.device)
    f32 = dict(dtype=torch.float32, device=x.device)
    if want_dh0 is None:
        want_dh0 = h0 is not None
    out = {"dx": torch.empty(x.shape, **like), "ddelta": torch.empty(x.shape, **like),
           "dA": torch.empty(A.shape, **f32), "dB": torch.empty(B.shape, **like), "dC": torch.empty(C.shape, **like),
           "dD": torch.empty(D.shape, **f32) if D is not None else None,
           "dz": torch.empty(x.shape, **like) if z is not None else None,
           "ddt_bias": torch.empty(dt_bias.shape, **f32) if dt_bias is not None else None,
           "dh0": torch.empty(state, **f32) if want_dh0 else None}
    if stream is not None:
        _lend(stream, x.device, (*out.values(), workspace if given is None else None))
    s = stream if stream is not None else _current_stream(x.get_device())
    st = lib.gdn_selective_scan_bwd(p, x.data_ptr(), delta.data_ptr(), A.data_ptr(), B.data_ptr(), C.data_ptr(),
                                    _address(D), _address(z), _address(dt_bias), _address(h0), _address(cu_seqlens),
                                    dout.data_ptr(), _address(dht), *(_address(t) for t in out.values()),
                                    workspace.data_ptr(), workspace.numel(), s)
    if st:
        raise GDNError(st, "gdn_selective_scan_bwd")
    out["workspace"] = workspace
    return out


def gdn_causal_conv1d_bwd(x, weight, dout, bias=None, activation="silu", initial_state=None, dfinal_state=None,
                          cu_seqlens=None, want_dinitial_state: Optional[bool] = None, workspace=None,
                          stream=None) -> dict:
    """Backward of gdn_causal_conv1d_fwd for ``dout`` (dL/dy) and ``dfinal_state`` (dL/d new state, [N, W-1, D], or
    None).  x, dout [B, T, D] and initial_state [N, W-1, D] share a dtype; weight [D, W], bias [D] fp32.  Returns
    dx, dweight, dbias, dinitial_state and the workspace under "workspace"; dbias is None without bias,
    dinitial_state unless ``want_dinitial_state`` (by default: initial_state is given)."""
    lib = _lib or load()
    if x.dtype not in DTYPES or x.dim() != 3 or weight.dim() != 2 or weight.shape[0] != x.shape[2]:
        raise ValueError("x must be float32 or bfloat16 [B, T, D] and weight [D, W]")
    _check_ws(workspace, x)
    B, T, D = x.shape
    W = weight.shape[1]
    if cu_seqlens is not None and cu_seqlens.dtype != torch.int32:
        raise ValueError("cu_seqlens must be int32")
    N = cu_seqlens.numel() - 1 if cu_seqlens is not None else B
    state = (N, W - 1, D)
    for name, t, dtype, shape in (("x", x, x.dtype, x.shape), ("dout", dout, x.dtype, x.shape),
                                  ("weight", weight, torch.float32, (D, W)), ("bias", bias, torch.float32, (D,)),
                                  ("initial_state", initial_state, x.dtype, state),
                                  ("dfinal_state", dfinal_state, x.dtype, state),
                                  ("cu_seqlens", cu_seqlens, torch.int32, (N + 1,))):
        if t is not None and (not t.is_cuda or t.device != x.device or not t.is_contiguous() or t.dtype != dtype
                              or t.shape != shape):
            raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of shape {tuple(shape)} on the device "
                             "of x")
    given = workspace
    if workspace is None:
        need = lib.gdn_causal_conv1d_bwd_workspace_size(B, T, D, W)
        if need == 0:
            raise GDNError(GDN_ERR_INVALID_ARG, "gdn_causal_conv1d_bwd_workspace_size")
        workspace = _alloc_ws(need, x.device)
    if want_dinitial_state is None:
        want_dinitial_state = initial_state is not None
    f32 = dict(dtype=torch.float32, device=x.device)
    out = {"dx": torch.empty_like(x), "dweight": torch.empty((D, W), **f32),
           "dbias": torch.empty((D,), **f32) if bias is not None else None,
           "dinitial_state": torch.empty(state, dtype=x.dtype, device=x.device) if want_dinitial_state else None}
    if stream is not None:
        _lend(stream, x.device, (*out.values(), workspace if given is None else None))
    s = stream if stream is not None else _current_stream(x.get_device())
    st = lib.gdn_causal_conv1d_bwd(x.data_ptr(), weight.data_ptr(), _address(bias), W, _address(initial_state),
                                   _address(cu_seqlens), N, B, T, D, DTYPES[x.dtype], ACTIVATIONS[activation],
                                   dout.data_ptr(), _address(dfinal_state), *(_address(t) for t in out.values()),
                                   workspace.data_ptr(), workspace.numel(), s)
    if st:
        raise GDNError(st, "gdn_causal_conv1d_bwd")
    out["workspace"] = workspace
    return out


def gdn_q4_matvec(x, qweight, scales, zeros=None, bias=None, y=None, stream=None):
    """y = x W^T + bias for 4-bit weights W [N, K] = (code - zero) * scale.  x [..., K] (bf16 or fp32; two
    dimensions may have any row stride), qweight [N, K / 2] uint8 (code 2j in byte j's low half), scales
    [N, K / group] (bf16 or fp32), zeros [N, K / group] uint8 or None (8), bias [N] fp32.  Returns y [..., N]."""
    lib = _lib or load()
    N, half = qshape = qweight.shape
    K, groups = 2 * half, scales.shape[1]
    dtype, sdt, dev = x.dtype, scales.dtype, x.get_device()
    if dtype not in DTYPES or sdt not in DTYPES:
        raise ValueError("x and scales must be float32 or bfloat16")
    if x.shape[-1] != K or dev < 0 or groups == 0 or K % groups != 0:
        raise ValueError("x must be a CUDA tensor of shape [..., K] and scales [N, K / group]")
    if not (qweight.dtype is torch.uint8 and qweight.get_device() == dev and qweight.is_contiguous()
            and scales.shape[0] == N and scales.get_device() == dev and scales.is_contiguous()
            and (zeros is None or (zeros.dtype is torch.uint8 and zeros.shape == scales.shape
                                   and zeros.get_device() == dev and zeros.is_contiguous()))
            and (bias is None or (bias.dtype is torch.float32 and bias.shape == (N,) and bias.get_device() == dev
                                  and bias.is_contiguous()))):
        raise ValueError(f"qweight (uint8 {tuple(qshape)}), scales and zeros (uint8) [N, K / group] and bias (float32 "
                         "[N]) must be contiguous and on the device of x")
    if x.is_contiguous():
        M, ld = x.numel() // K, K
    elif x.dim() == 2 and x.stride(1) == 1 and x.stride(0) >= K:
        M, ld = x.shape[0], x.stride(0)
    else:
        raise ValueError("x must be contiguous, or two-dimensional with contiguous rows")
    if y is None:
        y = torch.empty((*x.shape[:-1], N), dtype=dtype, device=x.device)
        if stream is not None:
            _lend(stream, x.device, (y,))
    elif y.shape != (*x.shape[:-1], N) or y.dtype != dtype or y.get_device() != dev or not y.is_contiguous():
        raise ValueError("y must be a contiguous CUDA tensor [..., N] with the dtype of x")
    s = stream if stream is not None else _current_stream(dev)
    st = lib.gdn_q4_matvec(x.data_ptr(), ld, qweight.data_ptr(), scales.data_ptr(), DTYPES[scales.dtype],
                           _address(zeros), _address(bias), M, N, K, K // groups, DTYPES[x.dtype], y.data_ptr(), s)
    if st:
        raise GDNError(st, "gdn_q4_matvec")
    return y


def _check_ints(what: str, *sizes) -> None:
    """Sizes that the C interface takes as ints (ctypes would pass their low 32 bits)."""
    if any(n >> 31 for n in sizes):
        raise GDNError(GDN_ERR_UNSUPPORTED, what)


def _linear_problem(q, k, v, g, cu_seqlens, fp32=(), others=()):
    """Checks of a linear attention's tensors and its problem.  fp32: (name, tensor, shape) that must be contiguous
    float32; others: (name, tensor) that must be like v and contiguous."""
    dtype, dev = v.dtype, v.get_device()
    # the usual call, all rows contiguous, in one expression: a decode step's launch is shorter than its checks
    if cu_seqlens is None and not others and dtype in DTYPES and dev >= 0 and q.dim() == 4 and v.dim() == 4:
        B, T, Hqk, K = qshape = q.shape
        b, t, Hv, V = v.shape
        f32 = torch.float32
        if (k.shape == qshape and b == B and t == T and q.dtype is dtype and k.dtype is dtype and g.dtype is f32
                and q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and g.is_contiguous()
                and q.get_device() == dev and k.get_device() == dev and g.get_device() == dev
                and (g.shape == (B, T, Hv) or g.shape == (Hv,)) and not (B | T | Hqk | Hv | K | V) >> 31):
            for _, x, want in fp32:
                if x is not None and (x.dtype is not f32 or x.get_device() != dev or x.shape != want
                                      or not x.is_contiguous()):
                    break
            else:
                return LinearProblem(B, T, B, Hqk, Hv, K, V, DTYPES[dtype], 0, 1 if g.dim() == 1 else 0)
    return _linear_problem_checked(q, k, v, g, cu_seqlens, fp32, others)


def _linear_problem_checked(q, k, v, g, cu_seqlens, fp32, others):
    dtype, dev = v.dtype, v.get_device()
    if dtype not in DTYPES or dev < 0 or q.dim() != 4 or v.dim() != 4:
        raise ValueError("q, k [B, T, Hqk, K] and v [B, T, Hv, V] must be float32 or bfloat16 CUDA tensors")
    B, T, Hqk, K = qshape = q.shape
    _, _, Hv, V = vshape = v.shape
    if k.shape != qshape or vshape[0] != B or vshape[1] != T:
        raise ValueError("q and k must have one shape, and v their batch and tokens")
    _check_ints("gdn_linear_attn", B, T, Hqk, K, Hv, V)
    for name, t in (("q", q), ("k", k), *others):
        if t.dtype is not dtype or t.get_device() != dev:
            raise ValueError(f"{name} must have the dtype and device of v")
    for name, t in others:
        if t.shape != vshape or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous with the shape of v")
    per_head = g.dim() == 1
    if (g.dtype is not torch.float32 or g.get_device() != dev or not g.is_contiguous()
            or g.shape != ((Hv,) if per_head else (B, T, Hv))):
        raise ValueError("g must be a contiguous float32 CUDA tensor [B, T, Hv], or [Hv] for one decay a head")
    for name, t, want in fp32:
        if t is not None and (t.dtype is not torch.float32 or t.get_device() != dev or t.shape != want
                              or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous float32 CUDA tensor of shape {tuple(want)}")
    N = B
    if cu_seqlens is not None:
        if (cu_seqlens.dtype is not torch.int32 or cu_seqlens.get_device() != dev or not cu_seqlens.is_contiguous()
                or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1):
            raise ValueError("cu_seqlens must be a contiguous int32 CUDA tensor [N + 1]")
        N = cu_seqlens.numel() - 1
        _check_ints("gdn_linear_attn", N)
    return LinearProblem(B, T, N, Hqk, Hv, K, V, DTYPES[dtype], int(cu_seqlens is not None), int(per_head),
                         _row_stride("q", q, Hqk * K), _row_stride("k", k, Hqk * K), _row_stride("v", v, Hv * V))


def _linear_state(q, v, cu_seqlens):
    return _scan_sequences(q, cu_seqlens), v.shape[-2], q.shape[-1], v.shape[-1]


def _slot_map(state_indices, n, dev, what):
    if (state_indices.dtype is not torch.int32 or state_indices.get_device() != dev
            or not state_indices.is_contiguous() or state_indices.numel() != n):
        raise ValueError(f"state_indices must be a contiguous int32 CUDA tensor, one {what} a sequence")
    return state_indices.data_ptr()


def gdn_linear_attn_fwd(q, k, v, g, scale: Optional[float] = None, h0=None, cu_seqlens=None, o=None, ht=None,
                        output_final_state: bool = True, state_indices=None, workspace=None, stream=None):
    """Linear attention with a decay for each head: S_t = e^{g_t} S_{t-1} + k_t v_t^T, o_t = scale S_t^T q_t.  q, k
    [B, T, Hqk, K] and v [B, T, Hv, V] (one dtype, bf16 or fp32; rows may be slices of wider rows), g fp32 [B, T, Hv]
    or [Hv], h0 [N, Hv, K, V] fp32.  Returns (o, ht); ht is None when ``output_final_state`` is False.  With
    ``state_indices`` [N] int32, ht is a pool [slots, Hv, K, V] whose rows they are (outside the pool: the sequence
    keeps no state).  ``scale`` defaults to K ** -0.5."""
    lib = _lib or load()
    _check_ws(workspace, q)
    state = _linear_state(q, v, cu_seqlens)
    rows, idx, dev = state, 0, v.get_device()
    if state_indices is not None:
        if ht is None or ht.dim() != 4 or ht.shape[0] == 0:
            raise ValueError("state_indices needs a pool ht [slots, Hv, K, V]")
        idx = _slot_map(state_indices, state[0], dev, "row of the pool")
        rows = (ht.shape[0], *state[1:])
    p = _linear_problem(q, k, v, g, cu_seqlens, (("h0", h0, state), ("ht", ht, rows)),
                        (("o", o),) if o is not None else ())
    given = o, ht, workspace
    if o is None:
        o = torch.empty_like(v, memory_format=torch.contiguous_format)
    if ht is None and output_final_state:
        ht = torch.empty(state, dtype=torch.float32, device=v.device)
    if workspace is None:
        need = _call(dev, lib.gdn_linear_attn_fwd_workspace_size, p)
        if need == 0:
            raise GDNError(GDN_ERR_UNSUPPORTED, "gdn_linear_attn_fwd_workspace_size")
        workspace = _alloc_ws(need, v.device)
    if stream is not None:
        _lend(stream, v.device, [t for t, x in zip((o, ht, workspace), given) if x is None])
    st = _call(dev, lib.gdn_linear_attn_fwd, p, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
               state[2] ** -0.5 if scale is None else scale, _address(h0), _address(cu_seqlens), o.data_ptr(),
               _address(ht), idx, rows[0], workspace.data_ptr(), workspace.numel(),
               stream if stream is not None else _current_stream(dev))
    if st:
        raise GDNError(st, "gdn_linear_attn_fwd")
    return o, ht


def gdn_linear_attn_fwd_workspace_size(p: LinearProblem) -> int:
    return int(load().gdn_linear_attn_fwd_workspace_size(ctypes.byref(p)))


def gdn_linear_attn_bwd_workspace_size(p: LinearProblem) -> int:
    return int(load().gdn_linear_attn_bwd_workspace_size(ctypes.byref(p)))


def gdn_linear_attn_get_device_status(workspace, stream=None) -> int:
    s = stream if stream is not None else _current_stream(workspace.get_device())
    v = ctypes.c_int(0)
    st = load().gdn_linear_attn_get_device_status(workspace.data_ptr(), s, ctypes.byref(v))
    if st:
        raise GDNError(st, "gdn_linear_attn_get_device_status")
    return int(v.value)


def gdn_linear_attn_bwd(q, k, v, g, dout, scale: Optional[float] = None, h0=None, dht=None, cu_seqlens=None,
                        want_dh0: Optional[bool] = None, workspace=None, stream=None) -> dict:
    """Backward of gdn_linear_attn_fwd for upstream gradients ``dout`` (dL/do, like v) and ``dht`` (dL/dht, fp32 or
    None).  Returns dq, dk, dv (dtype of v), dg, dh0 (fp32) and the workspace under "workspace"; dh0 is None unless
    ``want_dh0`` (by default: h0 is given)."""
    lib = _lib or load()
    _check_ws(workspace, q)
    state, dev = _linear_state(q, v, cu_seqlens), v.get_device()
    p = _linear_problem(q, k, v, g, cu_seqlens, (("h0", h0, state), ("dht", dht, state)), (("dout", dout),))
    given = workspace
    if workspace is None:
        need = _call(dev, lib.gdn_linear_attn_bwd_workspace_size, p)
        if need == 0:
            raise GDNError(GDN_ERR_UNSUPPORTED, "gdn_linear_attn_bwd_workspace_size")
        workspace = _alloc_ws(need, v.device)
    if want_dh0 is None:
        want_dh0 = h0 is not None
    like, f32 = dict(dtype=v.dtype, device=v.device), dict(dtype=torch.float32, device=v.device)
    out = {"dq": torch.empty(q.shape, **like), "dk": torch.empty(k.shape, **like), "dv": torch.empty(v.shape, **like),
           "dg": torch.empty(g.shape, **f32), "dh0": torch.empty(state, **f32) if want_dh0 else None}
    if stream is not None:
        _lend(stream, v.device, (*out.values(), workspace if given is None else None))
    st = _call(dev, lib.gdn_linear_attn_bwd, p, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
               state[2] ** -0.5 if scale is None else scale, _address(h0), _address(cu_seqlens), dout.data_ptr(),
               _address(dht), *(_address(t) for t in out.values()), workspace.data_ptr(), workspace.numel(),
               stream if stream is not None else _current_stream(dev))
    if st:
        raise GDNError(st, "gdn_linear_attn_bwd")
    out["workspace"] = workspace
    return out


def gdn_linear_attn_step(q, k, v, g, state, scale: Optional[float] = None, state_indices=None, cu_seqlens=None, o=None,
                         stream=None):
    """The recurrence's tokens on a state pool (decode).  ``state`` [slots, Hv, K, V] fp32 is updated in place;
    returns o.  Other arguments as for gdn_linear_attn_fwd."""
    lib = _lib or load()
    dev = v.get_device()
    slots = state.shape[0]
    p = _linear_problem(q, k, v, g, cu_seqlens, (("state", state, (slots, v.shape[-2], q.shape[-1], v.shape[-1])),),
                        (("o", o),) if o is not None else ())
    idx = 0 if state_indices is None else _slot_map(state_indices, p.N, dev, "slot")
    if o is None:
        o = torch.empty_like(v, memory_format=torch.contiguous_format)
        if stream is not None:
            _lend(stream, v.device, (o,))
    st = _call(dev, lib.gdn_linear_attn_step, p, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(),
               p.K ** -0.5 if scale is None else scale, state.data_ptr(), idx, slots, _address(cu_seqlens),
               o.data_ptr(), stream if stream is not None else _current_stream(dev))
    if st:
        raise GDNError(st, "gdn_linear_attn_step")
    return o


def _norm_rows(name: str, t, inner: int, width: int):
    """(rows, elements from one row to the next) of t, whose last ``inner`` dimensions are a row of ``width``."""
    if t.is_contiguous():
        return t.numel() // width if width else 0, width
    lead, want = t.dim() - inner, 1
    for i in range(t.dim() - 1, lead - 1, -1):
        if t.shape[i] != 1 and t.stride(i) != want:
            raise ValueError(f"{name} must have contiguous rows, one after the other at one stride")
        want *= t.shape[i]
    rows, ld = 1, None
    for i in range(lead - 1, -1, -1):
        if t.shape[i] != 1:
            if ld is None:
                ld = t.stride(i)
            elif t.stride(i) != ld * rows:
                raise ValueError(f"{name} must have contiguous rows, one after the other at one stride")
            rows *= t.shape[i]
    if ld is not None and ld < width:
        raise ValueError(f"{name} must have contiguous rows, one after the other at one stride")
    return rows, width if ld is None else ld


def _check_like(dev, *tensors):
    """(name, tensor, dtype, shape): contiguous CUDA tensors of the device."""
    for name, t, dtype, shape in tensors:
        if t is not None and (t.dtype is not dtype or t.get_device() != dev or t.shape != shape
                              or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on the device of x")


def _gated_norm(x, z, weight, others=()):
    dtype, dev, shape = x.dtype, x.get_device(), x.shape
    if weight is None:
        raise ValueError("weight must be a contiguous float32 tensor [V] (z alone may be None)")
    if (not others and dtype in DTYPES and dev >= 0 and len(shape) >= 2 and x.is_contiguous()
            and weight.dtype is torch.float32 and weight.shape == shape[-1:] and weight.get_device() == dev
            and weight.is_contiguous()
            and (z is None or (z.shape == shape and z.dtype is dtype and z.get_device() == dev and z.is_contiguous()))):
        H, V = shape[-2:]   # the usual call
        rows = x.numel() // (H * V) if H * V else 0
        if (rows | H | V) >> 31:
            _check_ints("gdn_gated_norm", rows, H, V)
        return rows, H, V, 0, 0, DTYPES[dtype], dev
    if dtype not in DTYPES or dev < 0 or x.dim() < 2:
        raise ValueError("x must be a float32 or bfloat16 CUDA tensor [..., H, V]")
    H, V = x.shape[-2:]
    if z is not None and (z.shape != x.shape or z.dtype is not dtype or z.get_device() != dev):
        raise ValueError("z must have the shape, dtype and device of x")
    _check_like(dev, ("weight", weight, torch.float32, (V,)), *others)
    rows, ld_x = _norm_rows("x", x, 2, H * V)
    _check_ints("gdn_gated_norm", rows, H, V)
    return rows, H, V, ld_x, _norm_rows("z", z, 2, H * V)[1] if z is not None else 0, DTYPES[dtype], dev


def gdn_gated_norm_fwd(x, z, weight, eps: float = 1e-6, y=None, save_rstd: bool = False, stream=None):
    """y = silu(z) * weight * x / rms(x) for every head: x, z [..., H, V] (bf16 or fp32; rows of H * V may be slices of
    wider rows; z None: no gate), weight [V] fp32.  Returns (y, rstd); rstd [..., H] fp32 is None unless
    ``save_rstd`` (for the backward)."""
    lib = _lib or load()
    rows, H, V, ld_x, ld_z, dt, dev = _gated_norm(x, z, weight, (("y", y, x.dtype, x.shape),) if y is not None else ())
    fresh = []
    if y is None:
        y = torch.empty_like(x, memory_format=torch.contiguous_format)
        fresh.append(y)
    rstd = None
    if save_rstd:
        rstd = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device)
        fresh.append(rstd)
    if stream is not None:
        _lend(stream, x.device, fresh)
    st = _call(dev, lib.gdn_gated_norm_fwd, x.data_ptr(), ld_x, _address(z), ld_z, weight.data_ptr(), rows, H, V, dt,
               eps, y.data_ptr(), _address(rstd), stream if stream is not None else _current_stream(dev))
    if st:
        raise GDNError(st, "gdn_gated_norm_fwd")
    return y, rstd


def gdn_gated_norm_bwd(x, z, weight, rstd, dy, workspace=None, stream=None) -> dict:
    """Backward of gdn_gated_norm_fwd for ``dy`` (like y), with the rstd that it saved.  Returns dx, dz (None without
    z), dweight (fp32) and the workspace under "workspace"."""
    lib = _lib or load()
    _check_ws(workspace, x)
    if rstd is None or dy is None:
        raise ValueError("rstd, which the forward saves with save_rstd, and dy are needed")
    rows, H, V, ld_x, ld_z, dt, dev = _gated_norm(x, z, weight, (("dy", dy, x.dtype, x.shape),
                                                                 ("rstd", rstd, torch.float32, x.shape[:-1])))
    given = workspace
    if workspace is None:
        need = _call(dev, lib.gdn_gated_norm_bwd_workspace_size, V)
        if need == 0:
            raise GDNError(GDN_ERR_UNSUPPORTED, "gdn_gated_norm_bwd_workspace_size")
        workspace = _alloc_ws(need, x.device)
    out = {"dx": torch.empty(x.shape, dtype=x.dtype, device=x.device),
           "dz": torch.empty(x.shape, dtype=x.dtype, device=x.device) if z is not None else None,
           "dweight": torch.empty((V,), dtype=torch.float32, device=x.device)}
    if stream is not None:
        _lend(stream, x.device, (*out.values(), workspace if given is None else None))
    st = _call(dev, lib.gdn_gated_norm_bwd, x.data_ptr(), ld_x, _address(z), ld_z, weight.data_ptr(), rstd.data_ptr(),
               dy.data_ptr(), rows, H, V, dt, *(_address(t) for t in out.values()), workspace.data_ptr(),
               workspace.numel(), stream if stream is not None else _current_stream(dev))
    if st:
        raise GDNError(st, "gdn_gated_norm_bwd")
    out["workspace"] = workspace
    return out


def _residual_norm(y, residual, post_weight, gate, weight, others):
    dtype, dev = y.dtype, y.get_device()
    if dtype not in DTYPES or dev < 0 or y.dim() < 1:
        raise ValueError("y must be a float32 or bfloat16 CUDA tensor [..., D]")
    shape, D = y.shape, y.shape[-1]
    f32 = torch.float32
    if (not others and y.is_contiguous() and residual.is_contiguous() and residual.shape == shape
            and residual.get_device() == dev and (residual.dtype is dtype or residual.dtype is f32)):
        vec, kind = shape[-1:], 0
        if gate is not None:   # 1: a vector, 2: like y
            kind = 2 if gate.shape == shape and gate.dtype is dtype else 1
        for t in (post_weight, weight, gate if kind == 1 else None):
            if t is not None and (t.dtype is not f32 or t.shape != vec or t.get_device() != dev
                                  or not t.is_contiguous()):
                break
        else:   # the usual call
            if kind < 2 or (gate.get_device() == dev and gate.is_contiguous()):
                rows = y.numel() // D if D else 0
                if (rows | D) >> 31:
                    _check_ints("gdn_residual_norm", rows, D)
                return rows, D, 0, kind, DTYPES[dtype], DTYPES[residual.dtype], dev
    if residual.dtype not in (dtype, torch.float32):
        raise ValueError("residual must have the dtype of y, or float32")
    kind = 0 if gate is None else 2 if gate.shape == shape and gate.dtype is dtype else 1
    _check_like(dev, ("residual", residual, residual.dtype, shape), ("post_weight", post_weight, f32, (D,)),
                ("gate", gate, *((f32, (D,)) if kind < 2 else (dtype, shape))), ("weight", weight, f32, (D,)),
                *others)
    rows, ld = _norm_rows("y", y, 1, D)
    _check_ints("gdn_residual_norm", rows, D)
    return rows, D, ld, kind, DTYPES[dtype], DTYPES[residual.dtype], dev


def gdn_residual_norm_fwd(y, residual, post_weight=None, gate=None, residual_scale: float = 1.0, weight=None,
                          eps: float = 1e-6, h=None, n=None, save_rstd: bool = False, stream=None):
    """Between two blocks: h = residual + residual_scale * gate * (post_weight * y / rms(y)), n = weight * h / rms(h).
    y [..., D] (bf16 or fp32; rows may be slices of wider rows), residual [..., D] (the dtype of y, or fp32), gate None,
    [D] fp32 or [..., D] like y, post_weight (None: y as it is) and weight (None: no n) [D] fp32.  Returns
    (h, n, rstd); h may be the residual itself, n is None without weight, rstd [..., 2] fp32 unless ``save_rstd``."""
    lib = _lib or load()
    given = (("h", h, residual.dtype, y.shape), ("n", n, y.dtype, y.shape)) if h is not None or n is not None else ()
    rows, D, ld, kind, dt, rdt, dev = _residual_norm(y, residual, post_weight, gate, weight, given)
    if n is not None and weight is None:
        raise ValueError("n needs weight")
    fresh = []
    if h is None:
        h = torch.empty_like(residual)
        fresh.append(h)
    if n is None and weight is not None:
        n = torch.empty_like(y, memory_format=torch.contiguous_format)
        fresh.append(n)
    rstd = None
    if save_rstd:
        rstd = torch.empty((*y.shape[:-1], 2), dtype=torch.float32, device=y.device)
        fresh.append(rstd)
    if stream is not None:
        _lend(stream, y.device, fresh)
    st = _call(dev, lib.gdn_residual_norm_fwd, y.data_ptr(), ld, residual.data_ptr(), _address(post_weight),
               _address(gate), kind, residual_scale, _address(weight), rows, D, dt, rdt, eps, h.data_ptr(),
               _address(n), _address(rstd), stream if stream is not None else _current_stream(dev))
    if st:
        raise GDNError(st, "gdn_residual_norm_fwd")
    return h, n, rstd


def gdn_residual_norm_bwd(y, residual, rstd, dh, dn=None, post_weight=None, gate=None, residual_scale: float = 1.0,
                          weight=None, workspace=None, stream=None) -> dict:
    """Backward of gdn_residual_norm_fwd for ``dh`` (like h, or None) and ``dn`` (like n; with weight), from its inputs
    (the residual as it was before the call) and the rstd that it saved.  Returns dy, dresidual, dpost_weight, dgate,
    dweight (None where the input is) and the workspace under "workspace"."""
    lib = _lib or load()
    if workspace is not None and workspace.device != y.device:
        raise ValueError("workspace must be on the device of y")
    if rstd is None:
        raise ValueError("rstd, which the forward saves with save_rstd, is needed")
    rows, D, ld, kind, dt, rdt, dev = _residual_norm(
        y, residual, post_weight, gate, weight,
        (("rstd", rstd, torch.float32, (*y.shape[:-1], 2)), ("dh", dh, residual.dtype, y.shape),
         ("dn", dn, y.dtype, y.shape)))
    if (dn is None) != (weight is None):
        raise ValueError("dn and weight come together")
    given = workspace
    if workspace is None:
        need = _call(dev, lib.gdn_residual_norm_bwd_workspace_size, D)
        if need == 0:
            raise GDNError(GDN_ERR_UNSUPPORTED, "gdn_residual_norm_bwd_workspace_size")
        workspace = _alloc_ws(need, y.device)
    f32 = dict(dtype=torch.float32, device=y.device)
    out = {"dy": torch.empty(y.shape, dtype=y.dtype, device=y.device),
           "dresidual": torch.empty(y.shape, dtype=residual.dtype, device=y.device),
           "dpost_weight": torch.empty((D,), **f32) if post_weight is not None else None,
           "dgate": torch.empty(gate.shape, dtype=gate.dtype, device=y.device) if gate is not None else None,
           "dweight": torch.empty((D,), **f32) if weight is not None else None}
    if stream is not None:
        _lend(stream, y.device, (*out.values(), workspace if given is None else None))
    st = _call(dev, lib.gdn_residual_norm_bwd, y.data_ptr(), ld, residual.data_ptr(), rstd.data_ptr(), _address(dh),
               _address(dn), _address(post_weight), _address(gate), kind, residual_scale, _address(weight), rows, D,
               dt, rdt, *(_address(t) for t in out.values()), workspace.data_ptr(), workspace.numel(),
               stream if stream is not None else _current_stream(dev))
    if st:
        raise GDNError(st, "gdn_residual_norm_bwd")
    out["workspace"] = workspace
    return out
