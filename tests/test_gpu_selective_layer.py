"""The selective layer as it is used: gradients through both operators, prompts then
4-bit decode steps against one pass, in a CUDA graph, and the example."""
import importlib.util
import os

import pytest
import torch

import selective_reference as R
from conftest import ROOT, rel_fro

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mod():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_chunked_gdn_gb300 import binding, selective_layer
    binding.load()
    return selective_layer


def test_layer_gradients(mod):
    """Parameter gradients against the definitions in 64 bits.  Every activation between the operators is rounded to
    bf16 (2^-8 a value) on one side only, four times on the way out and again on the way back: 5e-2."""
    torch.manual_seed(0)
    layer = mod.SelectiveLayer(32, 48, states=8, groups=2, rank=32)
    u = torch.randn(2, 40, 32, device="cuda").bfloat16()
    w = torch.randn(2, 40, 32, device="cuda")
    (layer(u).float() * w).sum().backward()
    p = {k: v.detach().double().cpu().requires_grad_() for k, v in layer.named_parameters()}
    x, z = (u.double().cpu() @ p["in_proj"].t()).chunk(2, dim=-1)
    x, _ = R.conv(x, p["conv_weight"], p["conv_bias"])
    dt, B, C = (x @ p["x_proj"].t()).split([32, 16, 16], dim=-1)
    y, _ = R.scan(x, dt @ p["dt_proj"].t(), -torch.exp(p["A_log"]), B.unflatten(-1, (2, 8)), C.unflatten(-1, (2, 8)),
                  D=p["Dskip"], z=z, dt_bias=p["dt_bias"])
    ((y @ p["out_proj"].t()) * w.double().cpu()).sum().backward()
    for k, v in layer.named_parameters():
        assert rel_fro(v.grad.double().cpu(), p[k].grad) <= 5e-2, k


def test_prompt_then_steps_match_one_pass(mod):
    """With the projections replaced by the values of their 4-bit codes (rounded to bf16), prompts and steps equal one
    pass up to bf16 roundings of the weights and activations: 5e-2."""
    torch.manual_seed(1)
    layer = mod.SelectiveLayer(64, 128, rank=32).quantize_()
    with torch.no_grad():
        for k, q in layer.q4.items():
            getattr(layer, k).copy_(mod.dequantize(*q))
    u = torch.randn(3, 24, 64, device="cuda").bfloat16()
    states = layer.new_states(5)
    slots = torch.tensor([4, 1, 0], dtype=torch.int32, device="cuda")
    outs = [layer.prompt(u[:, :20].contiguous(), states, slots)]
    outs += [layer.step(u[:, t].contiguous(), states, slots)[:, None] for t in range(20, 24)]
    with torch.no_grad():
        want = layer(u)
    assert rel_fro(torch.cat(outs, 1).double().cpu(), want.double().cpu()) <= 5e-2
    assert torch.all(states[0][[2, 3]] == 0) and torch.all(states[1][[2, 3]] == 0)


def test_steps_in_a_graph(mod):
    """A captured step replays on new inputs and carries the states on: bit for bit the uncaptured one."""
    torch.manual_seed(2)
    layer = mod.SelectiveLayer(64, 128, rank=32).quantize_()
    slots = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    a, b = layer.new_states(2), layer.new_states(2)
    tokens = torch.randn(3, 2, 64, device="cuda").bfloat16()
    want = [layer.step(t, a, slots) for t in tokens]
    u = tokens[0].clone()
    layer.step(u, b, slots)           # warm-up
    torch.cuda.synchronize()
    for s in b:
        s.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = layer.step(u, b, slots)
    for t, w in zip(tokens, want):
        u.copy_(t)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, w)
    assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_example(mod):
    spec = importlib.util.spec_from_file_location("example", os.path.join(ROOT, "examples", "selective_layer.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses, out = ex.main()
    assert losses[-1] < 0.7 * losses[0] and torch.isfinite(out.float()).all()
