"""The gated norm in fp32, value by value against 64 bits, with gates far out.

Bounds, relative.  y = z sigmoid(z) w x r: r from a mean of squares (2^-24 sqrt(V / 16), V values over 16 lanes, and the
tree's) and rsqrt (2^-22); the sigmoid's exponential (2^-23) of an exact argument, sum and reciprocal (2^-24 each); four
products (2^-24 each): 8e-7 together; 1e-6.  dz has 1 + z (1 - sigmoid) beside these, which vanishes at z = -1.28; from
z = -3 down it is above 1 in size, from z = 0 up it is: 1e-6 there.  An exponential whose argument is rounded first is
off by |z| 2^-24, 5e-6 at z = -80."""
import pytest
import torch

import linear_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def gdn():
    from gated_deltanet_chunked_gdn_gb300 import binding
    binding.load()
    return binding


@pytest.mark.parametrize("V", [64, 128, 129, 1000])
@pytest.mark.parametrize("lo,hi", [(-80.0, -3.0), (0.0, 80.0)])
def test_gates_far_out(gdn, lo, hi, V):
    torch.manual_seed(V)
    x, dy = 1.0 + torch.rand(40, 2, V, device=DEV), 1.0 + torch.rand(40, 2, V, device=DEV)
    z = lo + (hi - lo) * torch.rand(40, 2, V, device=DEV)
    w = 1.0 + 0.1 * torch.rand(V, device=DEV)
    y, rstd = gdn.gdn_gated_norm_fwd(x, z, w, eps=1e-5, save_rstd=True)
    got = gdn.gdn_gated_norm_bwd(x, z, w, rstd, dy)
    want = ref.gated_norm(x, z, w, 1e-5, dy)
    off = lambda a, b: float(((a.double() - b) / b).abs().max())  # noqa: E731
    assert off(y, ref.gated_norm(x, z, w, 1e-5)) <= 1e-6
    assert off(got["dz"], want["dz"]) <= 1e-6
