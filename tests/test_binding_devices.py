"""The binding's checks of tensors on several devices (no GPU: tensors without
storage stand for those of two GPUs, and every call must be refused before any
address is taken)."""
import pytest
import torch

from gated_deltanet_chunked_gdn_gb300 import binding as gdn

FakeTensorMode = pytest.importorskip("torch._subclasses.fake_tensor").FakeTensorMode


@pytest.mark.parametrize("other", ["weight", "dout", "bias", "initial_state", "dfinal_state", "cu_seqlens"])
def test_conv_bwd_tensors_share_a_device(other):
    with FakeTensorMode():
        at = lambda name, *s, **kw: torch.empty(*s, device="cuda:1" if name == other else "cuda:0", **kw)
        args = dict(x=at("x", 1, 16, 32), weight=at("weight", 32, 4), dout=at("dout", 1, 16, 32), bias=at("bias", 32),
                    initial_state=at("initial_state", 2, 3, 32), dfinal_state=at("dfinal_state", 2, 3, 32),
                    cu_seqlens=at("cu_seqlens", 3, dtype=torch.int32))
        with pytest.raises(ValueError, match=other):
            gdn.gdn_causal_conv1d_bwd(**args)
