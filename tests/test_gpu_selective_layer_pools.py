"""Prompts of the selective layer into its state pools: slots without a state, packed
prompts, and malformed offsets."""
import pytest
import torch

import selective_reference as R
from conftest import rel_fro

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mod():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_chunked_gdn_gb300 import binding, selective_layer
    binding.load()
    return selective_layer


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def run(layer, u, slots, cu=None, rows=6):
    conv, scan = layer.new_states(rows)
    conv.fill_(3.0), scan.fill_(7.0)
    out = layer.prompt(u, (conv, scan), ints(slots), cu)
    torch.cuda.synchronize()
    return out, conv, scan


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("slots", [[-1, 3, 0], [5, 6, 2], [1, -9, 1000], [-1, -1, 6]])
def test_prompt_slots_outside_the_pools(mod, packed, slots):
    """No state for them, and no other row touched; the rest bit for bit as with three slots."""
    torch.manual_seed(3)
    layer = mod.SelectiveLayer(32, 48, states=8, groups=2, rank=32)
    u = torch.randn(*((1, 60) if packed else (3, 20)), 32, device="cuda").bfloat16()
    cu = ints([0, 31, 33, 60]) if packed else None
    out, conv, scan = run(layer, u, slots, cu)
    ref, conv_ref, scan_ref = run(layer, u, [0, 1, 2], cu)
    assert torch.equal(out, ref)
    for row in range(6):
        if row in slots:
            assert torch.equal(conv[row], conv_ref[slots.index(row)])
            assert torch.equal(scan[row], scan_ref[slots.index(row)])
        else:
            assert torch.all(conv[row] == 3.0) and torch.all(scan[row] == 7.0)


def test_prompt_malformed_offsets(mod):
    torch.manual_seed(4)
    layer = mod.SelectiveLayer(32, 48, states=8, rank=32)
    u = torch.randn(1, 60, 32, device="cuda").bfloat16()
    _, _, scan = run(layer, u, [0, 4, 2], ints([0, 40, 20, 60]))
    assert torch.all(scan == 7.0)


def test_packed_prompt_against_the_definition(mod):
    """Outputs and states of packed prompts against the definitions in 64 bits: activations between the operators are
    rounded to bf16 on one side only, four times: 2e-2 (half of what gradients, rounded on the way back too, get)."""
    torch.manual_seed(5)
    layer = mod.SelectiveLayer(32, 48, states=8, groups=2, rank=32)
    lens = [31, 2, 27]
    u = torch.randn(1, 60, 32, device="cuda").bfloat16()
    out, conv, scan = run(layer, u, [4, 0, 2], ints([0, 31, 33, 60]))
    p = {k: v.detach().double().cpu() for k, v in layer.named_parameters()}
    x, z = (u.double().cpu() @ p["in_proj"].t()).chunk(2, dim=-1)
    x, final = R.conv(x, p["conv_weight"], p["conv_bias"], lens=lens)
    dt, B, C = (x @ p["x_proj"].t()).split([32, 16, 16], dim=-1)
    y, ht = R.scan(x, dt @ p["dt_proj"].t(), -torch.exp(p["A_log"]), B.unflatten(-1, (2, 8)),
                   C.unflatten(-1, (2, 8)), D=p["Dskip"], z=z, dt_bias=p["dt_bias"], lens=lens)
    assert rel_fro(out.double().cpu(), y @ p["out_proj"].t()) <= 2e-2
    at = [4, 0, 2]
    assert rel_fro(scan.double().cpu()[at], ht) <= 2e-2
    assert rel_fro(conv.double().cpu()[at], final) <= 2e-2
