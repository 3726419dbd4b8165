"""Host-side refusals of the scan forward that writes its final states to a pool (no
GPU: fake addresses, refused before any CUDA call)."""
import pytest
import torch

from gated_deltanet_chunked_gdn_gb300 import binding as b

AT = [i << 12 for i in range(1, 20)]


def call(ws_bytes=1 << 40, slots=4, **kw):
    p = kw.pop("p", None) or b.ScanProblem(2, 300, 2, 48, 16, 2, b.GDN_BF16, 0, 1, 0, 0, 0, 0, 0)
    v = dict(x=AT[0], delta=AT[1], A=AT[2], B=AT[3], C=AT[4], D=0, z=0, bias=0, h0=0, cu=0, y=AT[5], state=AT[6],
             idx=AT[7]) | kw
    return b.load().gdn_selective_scan_fwd_pool(p, *v.values(), slots, AT[8], ws_bytes, 0)


def test_refusals():
    for kw in (dict(state=0), dict(idx=0), dict(slots=0), dict(slots=-3), dict(idx=AT[7] + 2), dict(state=AT[6] + 4),
               dict(x=0), dict(y=0), dict(A=AT[2] + 8), dict(cu=AT[9]), dict(ws_bytes=16),
               dict(p=b.ScanProblem(2, 300, 2, 48, 0, 2, b.GDN_BF16, 0, 1, 0, 0, 0, 0, 0))):
        assert call(**kw) == b.GDN_ERR_INVALID_ARG, kw
    p = b.ScanProblem(2, 300, 2, 48, 65, 2, b.GDN_BF16, 0, 1, 0, 0, 0, 0, 0)
    assert call(p=p) == b.GDN_ERR_UNSUPPORTED


@pytest.mark.parametrize("bad", ["no pool", "count", "dtype", "device", "shape", "empty"])
def test_binding_refusals(bad):
    FakeTensorMode = pytest.importorskip("torch._subclasses.fake_tensor").FakeTensorMode
    with FakeTensorMode():
        at = lambda *s, **kw: torch.empty(*s, **(dict(device="cuda:0") | kw))
        i32 = dict(dtype=torch.int32)
        ht = None if bad == "no pool" else at(0 if bad == "empty" else 5, 32, 8 if bad == "shape" else 4)
        idx = at(3 if bad == "count" else 2, **(dict(dtype=torch.int64) if bad == "dtype" else
                                                dict(i32, device="cuda:1") if bad == "device" else i32))
        with pytest.raises(ValueError):
            b.gdn_selective_scan_fwd(at(2, 16, 32), at(2, 16, 32), at(32, 4), at(2, 16, 1, 4), at(2, 16, 1, 4), ht=ht,
                                     state_indices=idx)
