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


def scan(at):
    return dict(x=at("x", 1, 16, 32), delta=at("delta", 1, 16, 32), A=at("A", 32, 4), B=at("B", 1, 16, 1, 4),
                C=at("C", 1, 16, 1, 4))


@pytest.mark.parametrize("device", ["cpu", "cuda:1"])
@pytest.mark.parametrize("call", ["scan_fwd", "scan_bwd", "conv_bwd"])
def test_workspaces_are_checked(call, device):
    """The library writes to it, so it is on the device of x."""
    with FakeTensorMode():
        at = lambda name, *s: torch.empty(*s, device="cuda:0")
        ws = torch.empty(1 << 24, dtype=torch.uint8, device=device)
        with pytest.raises(ValueError, match="workspace"):
            if call == "scan_fwd":
                gdn.gdn_selective_scan_fwd(**scan(at), workspace=ws)
            elif call == "scan_bwd":
                gdn.gdn_selective_scan_bwd(**scan(at), dout=at("dout", 1, 16, 32), workspace=ws)
            else:
                gdn.gdn_causal_conv1d_bwd(at("x", 1, 16, 32), at("w", 32, 4), at("dout", 1, 16, 32), workspace=ws)
