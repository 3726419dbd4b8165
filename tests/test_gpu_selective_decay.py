"""GPU: the decays e^{dt A} of the selective scan have next to no bias.

A state is multiplied by its decay once a token, so a decay that is low by b on
average leaves the state low by b times the tokens of its memory, where errors of
either sign add up as the square root of their number.  fp32 numbers below 1 are 6e-8
apart; 1.2e-8, a fifth of that, is allowed for the mean of a decay's relative error.
The rest averages out: the roundings of the products (6e-8 at most, to nearest) over
the 16384 states and 64 tokens of a case, to 1e-10, and those of a rate over the
states (its relative 6e-8 counts by the exponent, at most 0.17 of a token's decay)."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
T, D, S, BAR = 64, 1024, 16, 1.2e-8


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_chunked_gdn_gb300 import binding
    binding.load()
    return binding


def rates(lo, hi, seed):
    """A with e^A = 2^-e, e spread over [lo, hi] by its logarithm."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = torch.rand(D, S, generator=g, device="cuda", dtype=torch.float64)
    return -(math.log(2) * torch.exp(math.log(lo) + r * math.log(hi / lo))).float()


def bias(got, A):
    want = torch.exp(T * A.double())
    return float(((got.double() / want - 1) / T).mean())


@pytest.mark.parametrize("lo,hi", [(4e-3, 0.25), (2e-4, 4e-3)])
@pytest.mark.parametrize("call", ["forward", "backward", "step", "steps of many"])
def test_decays_have_no_bias(gdn, call, lo, hi):
    """No inputs, steps of 1: the state after T tokens is the initial one's T-th decay, the gradient of the initial
    state the final one's."""
    A = rates(lo, hi, 1)
    n = 70 if call == "steps of many" else 1
    t = 1 if call.startswith("steps of") else T
    x, bc = torch.zeros(n, t, D, device="cuda"), torch.zeros(n, t, 1, S, device="cuda")
    args = (x, torch.ones_like(x), A, bc, bc)
    ones = torch.ones(n, D, S, device="cuda")
    if call == "forward":
        got = gdn.gdn_selective_scan_fwd(*args, softplus=False, h0=ones)[1]
    elif call == "backward":
        got = gdn.gdn_selective_scan_bwd(*args, x, softplus=False, h0=ones, dht=ones)["dh0"]
    else:
        got = ones
        for _ in range(T // t):
            gdn.gdn_selective_scan_step(*args, got, softplus=False)
    assert all(abs(bias(s, A)) <= BAR for s in got[:3])


def test_no_step_keeps_the_state(gdn):
    """A step of zero, and a rate of zero, leave every state as it is, to the bit."""
    A = rates(1e-3, 10.0, 2)
    A[:, 0] = 0.0
    g = torch.Generator(device="cuda").manual_seed(3)
    h = torch.randn(1, D, S, generator=g, device="cuda")
    x, bc = torch.zeros(1, 40, D, device="cuda"), torch.zeros(1, 40, 1, S, device="cuda")
    none, some = torch.zeros_like(x), torch.ones_like(x)
    assert torch.equal(gdn.gdn_selective_scan_fwd(x, none, A, bc, bc, softplus=False, h0=h)[1], h)
    assert torch.equal(gdn.gdn_selective_scan_fwd(x, some, A, bc, bc, softplus=False, h0=h)[1][..., 0], h[..., 0])
    assert torch.equal(gdn.gdn_selective_scan_bwd(x, none, A, bc, bc, x, softplus=False, h0=h, dht=h)["dh0"], h)
    state = h.clone()
    gdn.gdn_selective_scan_step(x, none, A, bc, bc, state, softplus=False)
    assert torch.equal(state, h)
