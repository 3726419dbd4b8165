"""Host-side checks of linear attention's and the norms' C entry points, and of their binding (no GPU): every call below
has fake, never dereferenced device addresses and must be refused before any CUDA call."""
import ctypes

import pytest
import torch

from gated_deltanet_chunked_gdn_gb300 import binding as b

BAD, UNSUPPORTED = b.GDN_ERR_INVALID_ARG, b.GDN_ERR_UNSUPPORTED
A4K = [i << 12 for i in range(1, 40)]


def P(**kw):
    base = dict(B=2, T=300, N=2, Hqk=2, Hv=4, K=128, V=64, dt=b.GDN_BF16, varlen=0, g_per_head=0, ld_q=0, ld_k=0, ld_v=0)
    return b.LinearProblem(*(base | kw).values())


def fwd(p, ws_bytes=1 << 40, slots=4, **kw):
    v = dict(q=A4K[0], k=A4K[1], v=A4K[2], g=A4K[3], scale=1.0, h0=0, cu=0, o=A4K[4], ht=0, idx=0) | kw
    ws = v.pop("ws", A4K[5])
    return b.load().gdn_linear_attn_fwd(p, *v.values(), slots, ws, ws_bytes, 0)


def bwd(p, ws_bytes=1 << 40, **kw):
    v = dict(q=A4K[0], k=A4K[1], v=A4K[2], g=A4K[3], scale=1.0, h0=0, cu=0, dout=A4K[6], dht=0, dq=A4K[7], dk=A4K[8],
             dv=A4K[9], dg=A4K[10], dh0=0, ws=A4K[5]) | kw
    return b.load().gdn_linear_attn_bwd(p, *v.values(), ws_bytes, 0)


def step(p, slots=4, **kw):
    v = dict(q=A4K[0], k=A4K[1], v=A4K[2], g=A4K[3], scale=1.0, state=A4K[11], idx=A4K[12]) | kw
    cu, o = v.pop("cu", 0), v.pop("o", A4K[4])
    return b.load().gdn_linear_attn_step(p, *v.values(), slots, cu, o, 0)


@pytest.mark.parametrize("bad,want", [
    (dict(Hv=3), BAD), (dict(Hqk=0), BAD), (dict(K=96), BAD), (dict(V=32), BAD), (dict(B=0), BAD), (dict(T=0), BAD),
    (dict(dt=7), BAD), (dict(varlen=1), BAD), (dict(varlen=1, B=1, N=0), BAD), (dict(ld_q=255), BAD),
    (dict(ld_k=260), BAD), (dict(ld_v=-8), BAD), (dict(B=1 << 16, T=1 << 15), BAD), (dict(Hv=2048), UNSUPPORTED),
    (dict(ld_v=1 << 29), UNSUPPORTED), (dict(B=1 << 20, T=64, Hv=1024, Hqk=1024, K=256, V=256), UNSUPPORTED)])
def test_problems(bad, want):
    p = P(**bad)
    assert fwd(p) == want and bwd(p) == want and step(p) == want
    assert b.gdn_linear_attn_fwd_workspace_size(p) == 0 and b.gdn_linear_attn_bwd_workspace_size(p) == 0


@pytest.mark.parametrize("p", [P(), P(dt=b.GDN_F32), P(K=256, V=256)])
def test_pointers(p):
    for k in ("q", "k", "v", "g", "o", "ws"):
        assert fwd(p, **{k: 0}) == BAD
    for k, v in (("q", 8), ("k", 2), ("v", 4), ("g", 2), ("o", 8), ("h0", 4), ("ht", 8), ("ws", 64)):
        assert fwd(p, **{k: A4K[21] + v}) == BAD, k
    assert fwd(p, cu=A4K[20]) == BAD and fwd(P(varlen=1, B=1, N=3)) == BAD
    assert fwd(p, idx=A4K[20]) == BAD and fwd(p, idx=A4K[20], ht=A4K[22], slots=0) == BAD    # rows of no pool
    assert fwd(p, ws_bytes=b.gdn_linear_attn_fwd_workspace_size(p) - 1) == BAD
    for k in ("dout", "dq", "dk", "dv", "dg", "ws"):
        assert bwd(p, **{k: 0}) == BAD
    for k in ("dout", "dq", "dk", "dv", "dht", "dh0"):
        assert bwd(p, **{k: A4K[21] + 8}) == BAD
    assert bwd(p, dg=A4K[21] + 2) == BAD
    assert bwd(p, ws_bytes=b.gdn_linear_attn_bwd_workspace_size(p) - 1) == BAD
    assert step(p, state=0) == BAD and step(p, slots=0) == BAD and step(p, state=A4K[13] + 4) == BAD
    assert step(p, idx=0, slots=1) == BAD
    out = ctypes.c_int(5)
    assert b.load().gdn_linear_attn_get_device_status(0, 0, ctypes.byref(out)) == BAD
    assert b.load().gdn_linear_attn_get_device_status(A4K[0], 0, None) == BAD


def test_workspaces_grow_with_the_problem():
    for kw in (dict(), dict(dt=b.GDN_F32), dict(varlen=1, B=1, N=5)):
        small, large = P(**kw), P(**{**kw, "T": 30000})
        assert 0 < b.gdn_linear_attn_fwd_workspace_size(small) < b.gdn_linear_attn_fwd_workspace_size(large)
        assert 0 < b.gdn_linear_attn_bwd_workspace_size(small) < b.gdn_linear_attn_bwd_workspace_size(large)
    assert b.gdn_linear_attn_fwd_workspace_size(P(varlen=1, B=1, N=1, T=0)) > 0


def gated_fwd(**kw):
    v = dict(x=A4K[0], ldx=0, z=A4K[1], ldz=0, w=A4K[2], rows=3, H=2, V=64, dt=1, eps=1e-6, y=A4K[3], rstd=0) | kw
    return b.load().gdn_gated_norm_fwd(*v.values(), 0)


def gated_bwd(ws_bytes=1 << 40, **kw):
    v = dict(x=A4K[0], ldx=0, z=A4K[1], ldz=0, w=A4K[2], rstd=A4K[4], dy=A4K[5], rows=3, H=2, V=64, dt=1, dx=A4K[6],
             dz=A4K[7], dw=A4K[8], ws=A4K[9]) | kw
    return b.load().gdn_gated_norm_bwd(*v.values(), ws_bytes, 0)


def test_gated_norm_refusals():
    for kw in (dict(x=0), dict(w=0), dict(rows=-1), dict(H=0), dict(V=0), dict(dt=5), dict(ldx=127), dict(ldz=1),
               dict(x=A4K[0] + 1), dict(z=A4K[1] + 1), dict(w=A4K[2] + 2)):
        assert gated_fwd(**kw) == BAD and gated_bwd(**kw) == BAD, kw
    assert gated_fwd(y=0) == BAD and gated_fwd(y=A4K[3] + 1) == BAD and gated_fwd(rstd=A4K[3] + 2) == BAD
    for kw in (dict(dx=0), dict(dw=0), dict(dy=0), dict(rstd=0), dict(dz=0), dict(z=0), dict(ws=0), dict(ws=A4K[9] + 64)):
        assert gated_bwd(**kw) == BAD, kw
    size = b.load().gdn_gated_norm_bwd_workspace_size
    assert gated_bwd(ws_bytes=size(64) - 1) == BAD and size(0) == 0 and size(16385) == 0
    assert gated_fwd(V=16385) == UNSUPPORTED and gated_fwd(rows=1 << 30, H=8) == UNSUPPORTED
    assert gated_fwd(rows=0, x=0, y=0) == b.GDN_OK     # nothing to do, nothing launched


def residual_fwd(**kw):
    v = dict(y=A4K[0], ld=0, r=A4K[1], pw=A4K[2], gate=A4K[3], kind=1, scale=1.0, w=A4K[4], rows=3, D=64, dt=1, rdt=0,
             eps=1e-6, h=A4K[5], n=A4K[6], rstd=0) | kw
    return b.load().gdn_residual_norm_fwd(*v.values(), 0)


def residual_bwd(ws_bytes=1 << 40, **kw):
    v = dict(y=A4K[0], ld=0, r=A4K[1], rstd=A4K[7], dh=0, dn=A4K[8], pw=A4K[2], gate=A4K[3], kind=1, scale=1.0, w=A4K[4],
             rows=3, D=64, dt=1, rdt=0, dy=A4K[9], dr=A4K[10], dpw=A4K[11], dgate=A4K[12], dw=A4K[13], ws=A4K[14]) | kw
    return b.load().gdn_residual_norm_bwd(*v.values(), ws_bytes, 0)


def test_residual_norm_refusals():
    for kw in (dict(y=0), dict(r=0), dict(rows=-1), dict(D=0), dict(dt=2), dict(rdt=2), dict(dt=0, rdt=1), dict(kind=3),
               dict(kind=0), dict(gate=0), dict(ld=63), dict(y=A4K[0] + 1), dict(r=A4K[1] + 2), dict(gate=A4K[3] + 2)):
        assert residual_fwd(**kw) == BAD and residual_bwd(**kw) == BAD, kw
    for kw in (dict(h=0), dict(n=0), dict(w=0), dict(h=A4K[5] + 2), dict(rstd=2)):
        assert residual_fwd(**kw) == BAD, kw
    for kw in (dict(dy=0), dict(dr=0), dict(dpw=0), dict(pw=0), dict(dgate=0), dict(dw=0), dict(w=0), dict(dn=0),
               dict(rstd=0), dict(ws=0), dict(dh=A4K[15] + 2)):
        assert residual_bwd(**kw) == BAD, kw
    size = b.load().gdn_residual_norm_bwd_workspace_size
    assert residual_bwd(ws_bytes=size(64) - 1) == BAD and size(0) == 0 and size(16385) == 0
    assert residual_fwd(D=16385) == UNSUPPORTED and residual_fwd(rows=0, h=0, n=0) == b.GDN_OK


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    q, v, g = torch.zeros(1, 4, 1, 64), torch.zeros(1, 4, 2, 64), torch.zeros(1, 4, 2)
    for call in (lambda: b.gdn_linear_attn_fwd(q, q, v, g), lambda: b.gdn_linear_attn_bwd(q, q, v, g, v),
                 lambda: b.gdn_linear_attn_step(q, q, v, g, torch.zeros(1, 2, 64, 64)),
                 lambda: b.gdn_gated_norm_fwd(v, v, torch.ones(64)),
                 lambda: b.gdn_residual_norm_fwd(v, v, weight=torch.ones(64))):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("t,ok", [
    (torch.zeros(6, 10)[:, :8], (6, 10)), (torch.zeros(2, 3, 10)[..., :8], (6, 10)), (torch.zeros(3, 8), (3, 8)),
    (torch.zeros(2, 3, 8)[:, :2], None), (torch.zeros(8, 6).t(), None), (torch.zeros(1, 16)[:, ::2], None),
    (torch.zeros(1, 10)[:, :8], (1, 8)), (torch.zeros(1, 8).expand(4, 8), None)])
def test_rows_at_one_stride(t, ok):
    if ok is None:
        with pytest.raises(ValueError):
            b._norm_rows("x", t, 1, 8)
    else:
        assert b._norm_rows("x", t, 1, 8) == ok
