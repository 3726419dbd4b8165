"""The residual norm's autograd function on the CPU (no GPU): the operators that it calls are replaced by their
definitions in 64 bits, with the library's rule that dn and weight come together.  Gradients of every combination of the
optional parts, against differences."""
import itertools

import pytest
import torch

import linear_reference as ref
from gated_deltanet_chunked_gdn_gb300 import linear_layer as mod


def residual_fwd(y, residual, post_weight=None, gate=None, residual_scale=1.0, weight=None, eps=1e-6, save_rstd=False):
    h, n = ref.residual_norm(y, residual, post_weight, gate, residual_scale, weight, eps)
    return h, n, torch.zeros(*y.shape[:-1], 2, dtype=torch.float64)


def residual_bwd(y, residual, rstd, dh, dn=None, post_weight=None, gate=None, residual_scale=1.0, weight=None):
    if (dn is None) != (weight is None):
        raise ValueError("dn and weight come together")
    dh = torch.zeros_like(y) if dh is None else dh
    d = ref.residual_norm(y, residual, post_weight, gate, residual_scale, weight, 1e-3, dh, dn)
    return {n: d.get(n) for n in ("dy", "dresidual", "dpost_weight", "dgate", "dweight")}


@pytest.mark.parametrize("post,gate,weight", 
                         list(itertools.product([False, True], ["none", "channel", "element"], [False, True])))
def test_residual_norm_without_its_parts(monkeypatch, post, gate, weight):
    monkeypatch.setattr(mod.gdn, "gdn_residual_norm_fwd", residual_fwd)
    monkeypatch.setattr(mod.gdn, "gdn_residual_norm_bwd", residual_bwd)
    torch.manual_seed(0)
    leaf = lambda *s: torch.randn(*s, dtype=torch.float64, requires_grad=True)  # noqa: E731
    y, r = leaf(3, 5), leaf(3, 5)
    pw, w = leaf(5) if post else None, leaf(5) if weight else None
    gt = {"none": None, "channel": leaf(5), "element": leaf(3, 5)}[gate]

    def call(*leaves):
        h, n = mod.ResidualNorm.apply(y, r, pw, gt, 0.7, w, 1e-3)
        assert (n is None) == (w is None)
        return h if n is None else (h, n)

    assert torch.autograd.gradcheck(call, [t for t in (y, r, pw, gt, w) if t is not None])
