"""What the norms' binding says about tensors that are not optional (no GPU: tensors without storage)."""
import pytest
import torch

from gated_deltanet_chunked_gdn_gb300 import binding as gdn

FakeTensorMode = pytest.importorskip("torch._subclasses.fake_tensor").FakeTensorMode


def test_missing_tensors_are_named():
    with FakeTensorMode():
        at = lambda *s: torch.empty(*s, device="cuda:0")  # noqa: E731
        x, w, rstd = at(3, 2, 64), at(64), at(3, 2)
        for call, args, name in ((gdn.gdn_gated_norm_fwd, (x, x, None), "weight"),
                                 (gdn.gdn_gated_norm_bwd, (x, x, None, rstd, x), "weight"),
                                 (gdn.gdn_gated_norm_bwd, (x, x, w, None, x), "rstd"),
                                 (gdn.gdn_gated_norm_bwd, (x, x, w, rstd, None), "dy"),
                                 (gdn.gdn_residual_norm_bwd, (x, x, None, x), "rstd")):
            with pytest.raises(ValueError, match=name):
                call(*args)
