"""The residual norm's autograd function on the GPU with and without each of its parts, against its gradients' formulas in
64 bits.  fp32 throughout: the tolerance of the operator's own tests, 2e-6."""
import itertools

import pytest
import torch

import linear_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def mod():
    from gated_deltanet_chunked_gdn_gb300 import binding, linear_layer
    binding.load()
    return linear_layer


@pytest.mark.parametrize("post,gate,weight",
                         list(itertools.product([False, True], ["none", "channel", "element"], [False, True])))
def test_residual_norm_parts(mod, post, gate, weight):
    torch.manual_seed(0)
    leaf = lambda *s: torch.randn(*s, device=DEV).requires_grad_()  # noqa: E731
    y, r = leaf(7, 96), leaf(7, 96)
    pw, w = leaf(96) if post else None, leaf(96) if weight else None
    gt = {"none": None, "channel": leaf(96), "element": leaf(7, 96)}[gate]
    h, n = mod.ResidualNorm.apply(y, r, pw, gt, 0.7, w, 1e-3)
    dh, dn = torch.randn_like(h), torch.randn_like(h) if weight else None
    loss = (h * dh).sum() + ((n * dn).sum() if weight else 0.0)
    loss.backward()
    with torch.no_grad():
        want = ref.residual_norm(y, r, pw, gt, 0.7, w, 1e-3, dh, dn)
    for name, t in (("dy", y), ("dresidual", r), ("dpost_weight", pw), ("dgate", gt), ("dweight", w)):
        if t is not None:
            assert ref.rel(t.grad, want[name]) < 2e-6, name
