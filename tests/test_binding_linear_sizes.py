"""Sizes that the C interface's ints do not hold are refused by linear attention's and the norms' binding, not cut to
their low 32 bits (no GPU: tensors without storage, refused before any address is taken)."""
import pytest
import torch

from gated_deltanet_chunked_gdn_gb300 import binding as gdn

FakeTensorMode = pytest.importorskip("torch._subclasses.fake_tensor").FakeTensorMode
BIG = (1 << 32) + 64   # 64 in its low 32 bits
BF, F32 = torch.bfloat16, torch.float32


def at(*s, dtype=BF):
    return torch.empty(*s, dtype=dtype, device="cuda:0")


def refused(call, *args, **kw):
    with pytest.raises(gdn.GDNError) as e:
        call(*args, **kw)
    assert e.value.status == gdn.GDN_ERR_UNSUPPORTED


@pytest.mark.parametrize("shape", [(BIG, 1, 1), (BIG, 2, 8), (2, BIG, 1), (1, 1, BIG)])
@pytest.mark.parametrize("sliced", [False, True])
def test_gated_norm(shape, sliced):
    with FakeTensorMode():
        x = at(shape[0], shape[1] * shape[2] + sliced)[:, :shape[1] * shape[2]].unflatten(1, shape[1:])
        y, w, rstd = at(*shape), at(shape[2], dtype=F32), at(*shape[:2], dtype=F32)
        refused(gdn.gdn_gated_norm_fwd, x, None, w)
        refused(gdn.gdn_gated_norm_bwd, x, None, w, rstd, y)


@pytest.mark.parametrize("shape", [(BIG, 1), (1 << 31, 3), (2, BIG)])
def test_residual_norm(shape):
    with FakeTensorMode():
        y, w, rstd = at(*shape), at(shape[1], dtype=F32), at(shape[0], 2, dtype=F32)
        refused(gdn.gdn_residual_norm_fwd, y, y, weight=w)
        refused(gdn.gdn_residual_norm_bwd, y, y, rstd, y, dn=y, weight=w)


@pytest.mark.parametrize("B,T,Hqk,Hv,K,V", [(1, 1, 1, 1, BIG, 64), (1, 1, 1, 1, 64, BIG), (1, 1, BIG, BIG, 64, 64),
                                            (BIG, 1, 1, 1, 64, 64), (1, BIG, 1, 1, 64, 64)])
def test_linear_attention(B, T, Hqk, Hv, K, V):
    with FakeTensorMode():
        q, v, g = at(B, T, Hqk, K), at(B, T, Hv, V), at(B, T, Hv, dtype=F32)
        refused(gdn.gdn_linear_attn_fwd, q, q, v, g, output_final_state=False)
        refused(gdn.gdn_linear_attn_fwd, q, q, v, g, o=at(B, T, Hv, V), output_final_state=False)
        refused(gdn.gdn_linear_attn_bwd, q, q, v, g, v)
        refused(gdn.gdn_linear_attn_step, q, q, v, g, at(B, Hv, K, V, dtype=F32))


def test_no_offsets_at_all():
    with FakeTensorMode():
        q, v, g = at(1, 8, 1, 64), at(1, 8, 1, 64), at(1, 8, 1, dtype=F32)
        with pytest.raises(ValueError, match="cu_seqlens"):
            gdn.gdn_linear_attn_fwd(q, q, v, g, cu_seqlens=at(0, dtype=torch.int32))
