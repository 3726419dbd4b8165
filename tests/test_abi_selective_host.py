"""Host-side checks of the selective layer's C entry points (no GPU): every call
below has fake, never dereferenced device addresses and must be refused before any
CUDA call; workspaces are sized without one."""
import ctypes

import pytest

from gated_deltanet_chunked_gdn_gb300 import binding as b

BAD, UNSUPPORTED = b.GDN_ERR_INVALID_ARG, b.GDN_ERR_UNSUPPORTED


def P(**kw):
    base = dict(B=2, T=300, N=2, D=48, S=16, G=2, dt=b.GDN_BF16, varlen=0, softplus=1, ld_x=0, ld_delta=0, ld_z=0,
                ld_b=0, ld_c=0)
    return b.ScanProblem(*(base | kw).values())


A4K = [i << 12 for i in range(1, 40)]


def fwd(p, ws_bytes=1 << 40, **kw):
    v = dict(x=A4K[0], delta=A4K[1], A=A4K[2], B=A4K[3], C=A4K[4], D=0, z=0, bias=0, h0=0, cu=0, y=A4K[5], ht=0,
             ws=A4K[6]) | kw
    return b.load().gdn_selective_scan_fwd(p, *v.values(), ws_bytes, 0)


def bwd(p, ws_bytes=1 << 40, **kw):
    v = dict(x=A4K[0], delta=A4K[1], A=A4K[2], B=A4K[3], C=A4K[4], D=0, z=0, bias=0, h0=0, cu=0, dout=A4K[7], dht=0,
             dx=A4K[8], ddelta=A4K[9], dA=A4K[10], dB=A4K[11], dC=A4K[12], dD=0, dz=0, dbias=0, dh0=0, ws=A4K[6]) | kw
    return b.load().gdn_selective_scan_bwd(p, *v.values(), ws_bytes, 0)


def step(p, slots=4, **kw):
    v = dict(x=A4K[0], delta=A4K[1], A=A4K[2], B=A4K[3], C=A4K[4], D=0, z=0, bias=0, state=A4K[13], idx=A4K[14]) | kw
    cu, y = v.pop("cu", 0), v.pop("y", A4K[5])
    return b.load().gdn_selective_scan_step(p, *v.values(), slots, cu, y, 0)


@pytest.mark.parametrize("bad,want", [(dict(D=0), BAD), (dict(G=5), BAD), (dict(S=0), BAD), (dict(B=0), BAD),
                                      (dict(T=0), BAD), (dict(dt=7), BAD), (dict(varlen=1), BAD),
                                      (dict(varlen=1, B=1, N=0), BAD), (dict(ld_x=47), BAD), (dict(ld_b=31), BAD),
                                      (dict(ld_z=-1), BAD), (dict(S=65), UNSUPPORTED),
                                      (dict(D=65538), UNSUPPORTED), (dict(ld_c=1 << 29), UNSUPPORTED)])
def test_scan_problems(bad, want):
    p = P(**bad)
    assert fwd(p) == want and bwd(p) == want and step(p) == want
    assert b.gdn_selective_scan_fwd_workspace_size(p) == 0 and b.gdn_selective_scan_bwd_workspace_size(p) == 0


def test_scan_bwd_group_limit():
    p = P(D=65536, G=65536, S=4)
    assert b.gdn_selective_scan_fwd_workspace_size(p) > 0 and b.gdn_selective_scan_bwd_workspace_size(p) == 0
    assert bwd(p) == UNSUPPORTED


def test_scan_pointers():
    p = P()
    for k in ("x", "delta", "A", "B", "C", "y", "ws"):
        assert fwd(p, **{k: 0}) == BAD
    for k, v in (("x", 1), ("A", 8), ("h0", 8), ("ht", 4), ("bias", 2), ("ws", 64), ("cu", A4K[20]), ("y", 1)):
        assert fwd(p, **{k: (v if k == "cu" else A4K[21] + v)}) == BAD
    assert fwd(p, ws_bytes=b.gdn_selective_scan_fwd_workspace_size(p) - 1) == BAD
    assert fwd(P(varlen=1, B=1, N=3)) == BAD                        # packed without offsets
    for k in ("dout", "dx", "ddelta", "dA", "dB", "dC", "ws"):
        assert bwd(p, **{k: 0}) == BAD
    assert bwd(p, z=A4K[22]) == BAD and bwd(p, dz=A4K[22]) == BAD    # a gate and its gradient come together
    assert bwd(p, dh0=A4K[23] + 4) == BAD
    assert bwd(p, ws_bytes=b.gdn_selective_scan_bwd_workspace_size(p) - 1) == BAD
    assert step(p, state=0) == BAD and step(p, slots=0) == BAD and step(p, state=A4K[13] + 4) == BAD
    assert step(p, idx=0, slots=1) == BAD                           # a slot for every sequence without a map


def test_scan_device_status_refusals():
    out = ctypes.c_int(5)
    assert b.load().gdn_selective_scan_get_device_status(P(S=65), 0, 0, ctypes.byref(out)) == BAD
    assert b.load().gdn_selective_scan_get_device_status(P(), 0, 0, None) == BAD


def conv(ws_bytes=1 << 40, **kw):
    v = dict(x=A4K[0], w=A4K[1], bias=0, W=4, init=0, cu=0, N=2, B=2, T=16, D=64, dt=1, act=1, dout=A4K[2], dfinal=0,
             dx=A4K[3], dw=A4K[4], db=0, dinit=0, ws=A4K[5]) | kw
    return b.load().gdn_causal_conv1d_bwd(*v.values(), ws_bytes, 0)


def test_conv_bwd_refusals():
    size = b.load().gdn_causal_conv1d_bwd_workspace_size
    assert size(2, 16, 64, 4) > 0 and size(2, 16, 60, 4) == 0 and size(2, 16, 64, 5) == 0
    for kw in (dict(D=12), dict(W=0), dict(W=5), dict(x=0), dict(w=0), dict(dout=0), dict(dx=0), dict(dw=0), dict(N=3),
               dict(cu=A4K[9]), dict(dt=3), dict(act=2), dict(x=A4K[0] + 8), dict(dinit=A4K[8] + 4),
               dict(db=A4K[8] + 2), dict(ws=0), dict(ws=A4K[5] + 16), dict(ws_bytes=size(2, 16, 64, 4) - 1)):
        assert conv(**kw) == BAD, kw


def q4(**kw):
    v = dict(x=A4K[0], ld=0, w=A4K[1], sc=A4K[2], sdt=1, zero=0, bias=0, M=2, N=8, K=256, group=64, dt=1, y=A4K[3]) | kw
    return b.load().gdn_q4_matvec(*v.values(), 0)


def test_q4_refusals():
    for kw in (dict(x=0), dict(w=0), dict(sc=0), dict(y=0), dict(M=-1), dict(N=0), dict(K=0), dict(group=16),
               dict(group=96), dict(K=250), dict(dt=2), dict(sdt=2), dict(ld=255), dict(w=A4K[1] + 8),
               dict(x=A4K[0] + 1), dict(bias=A4K[4] + 2)):
        assert q4(**kw) == BAD, kw
    assert q4(K=(1 << 20) + 64) == UNSUPPORTED
    assert q4(M=0, x=0, y=0) == b.GDN_OK                            # nothing to do, nothing launched
