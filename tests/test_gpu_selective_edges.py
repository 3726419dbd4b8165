"""GPU edges of the selective scan where sums overflow or lose terms and rates are
infinite, against closed forms or the 64-bit definition."""
import pytest
import torch

import selective_reference as R
from conftest import rel_fro

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_chunked_gdn_gb300 import binding
    binding.load()
    return binding


def cuda(d):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()}


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("state,adjoint", [(1e30, 1e30), (1e19, 2e18)])
def test_bwd_infinite_rate_gradients(gdn, sign, state, adjoint):
    """No decay and no inputs: dA is the number of tokens times state times adjoint.  Every term is infinite in fp32,
    or every tile finite and the sum of three not: the gradient is an infinity with its sign, not a NaN."""
    T, D, S = 48, 4, 4
    one, bc = torch.ones(1, T, D, device="cuda"), torch.zeros(1, T, 1, S, device="cuda")
    full = lambda v: torch.full((1, D, S), v, device="cuda")
    g = gdn.gdn_selective_scan_bwd(one, one, torch.zeros(D, S, device="cuda"), bc, bc, one, softplus=False,
                                   h0=full(sign * state), dht=full(adjoint))
    assert torch.all(g["dA"] == sign * float("inf"))
