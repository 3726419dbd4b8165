"""The linear attention layer and the stack as they are used: gradients through the operators together, prompts then
4-bit decode steps against one pass, in CUDA graphs, and the example."""
import importlib.util
import os

import pytest
import torch

import linear_reference as ref
import selective_reference as R
from conftest import ROOT

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mod():
    from gated_deltanet_chunked_gdn_gb300 import binding, linear_layer
    binding.load()
    return linear_layer


@pytest.fixture(scope="module")
def selective():
    from gated_deltanet_chunked_gdn_gb300 import selective_layer
    return selective_layer


def attention(q, k, v, g, scale):
    """The recurrence in 64 bits with gradients, by its sums over pairs of tokens: q, k [B, T, H, K] for every value
    head, g [B, T, H]."""
    b = g.cumsum(1)
    d = (b[:, :, None] - b[:, None, :]).masked_fill(
        torch.ones(q.shape[1], q.shape[1], device=q.device).triu(1).bool()[None, :, :, None], -float("inf"))
    w = scale * torch.einsum("bihd,bjhd->bijh", q, k) * torch.exp(d)
    return torch.einsum("bijh,bjhe->bihe", w, v)


def linear_plain(layer, p, u):
    B, T, _ = u.shape
    qk, vz = layer.Hqk * layer.K, layer.Hv * layer.V
    q, k, v, z = (u @ p["in_proj"].t()).split([qk, qk, vz, vz], dim=-1)
    R_ = layer.Hv // layer.Hqk
    q, k = (t.view(B, T, layer.Hqk, layer.K).repeat_interleave(R_, 2) for t in (q, k))
    v, z = v.view(B, T, layer.Hv, -1), z.view(B, T, layer.Hv, -1)
    if layer.decay == "head":
        g = layer.slopes.double().expand(B, T, layer.Hv)
    else:
        g = -torch.exp(p["A_log"]) * torch.nn.functional.softplus(u @ p["a_proj"].t() + p["dt_bias"])
    o = attention(q, k, v, g, layer.K ** -0.5)
    y = torch.nn.functional.silu(z) * p["norm_weight"] * o * ref.rms(o, layer.eps)
    return y.flatten(2) @ p["out_proj"].t()


def doubles(module):
    return {k: v.detach().double().requires_grad_() for k, v in module.named_parameters()}


@pytest.mark.parametrize("decay", ["token", "head"])
def test_layer_gradients(mod, decay):
    """Parameter gradients against the definitions in 64 bits.  Every activation between the operators is rounded to
    bf16 (2^-8 a value at most) on one side only, five times on the way out and again on the way back: 5e-2.  The norm's
    eps is 1: a sequence's first output is scale (q . k) v, and a norm without eps takes the factor q . k out of it, so
    that the gradients of q and k there, scale k (do . v), are sums of terms of size 1 / (q . k) that cancel to
    nothing; what is left of them is the rounding of do, 2^-8 of terms that can be a hundred times all others."""
    torch.manual_seed(0)
    layer = mod.LinearLayer(32, 1, 2, K=64, V=64, decay=decay, eps=1.0)
    u = torch.randn(2, 80, 32, device="cuda").bfloat16()
    w = torch.randn(2, 80, 32, device="cuda")
    out = layer(u)
    (out.float() * w).sum().backward()
    p = doubles(layer)
    want = linear_plain(layer, p, u.double())
    (want * w.double()).sum().backward()
    assert ref.rel(out, want) <= 2e-2
    for k, v in layer.named_parameters():
        assert ref.rel(v.grad, p[k].grad) <= 5e-2, k


@pytest.mark.parametrize("residual", [torch.bfloat16, torch.float32])
def test_stack_gradients(mod, selective, residual):
    """The same through norms, residual sums and a selective layer behind the linear one: twice the roundings, 0.1."""
    torch.manual_seed(1)
    stack = mod.Stack([mod.LinearLayer(32, 1, K=64, V=64, eps=1.0), selective.SelectiveLayer(32, 48, states=8, rank=32)], 32,
                      scale=0.7, residual_dtype=residual)
    with torch.no_grad():
        for q in [stack.first_weight, *stack.post_weights, *stack.gates, *stack.weights]:
            q.add_(0.1 * torch.randn_like(q))
    u = torch.randn(2, 40, 32, device="cuda").bfloat16()
    w = torch.randn(2, 40, 32, device="cuda")
    out = stack(u)
    (out.float() * w).sum().backward()
    p = doubles(stack)

    def sub(prefix):
        return {k[len(prefix):]: v for k, v in p.items() if k.startswith(prefix)}

    def selective_plain(q, x):
        x, z = (x @ q["in_proj"].t()).chunk(2, dim=-1)
        x, _ = R.conv(x.cpu(), q["conv_weight"].cpu(), q["conv_bias"].cpu())
        dt, B, C = (x @ q["x_proj"].cpu().t()).split([32, 8, 8], dim=-1)
        y, _ = R.scan(x, dt @ q["dt_proj"].cpu().t(), -torch.exp(q["A_log"]).cpu(), B.unflatten(-1, (1, 8)),
                      C.unflatten(-1, (1, 8)), D=q["Dskip"].cpu(), z=z.cpu(), dt_bias=q["dt_bias"].cpu())
        return y.to(z.device) @ q["out_proj"].t()

    h = u.double()
    n = h * ref.rms(h, 1e-6) * p["first_weight"]
    for i, mix in enumerate((lambda x: linear_plain(stack.mixers[0], sub("mixers.0."), x),
                             lambda x: selective_plain(sub("mixers.1."), x))):
        y = mix(n)
        h = h + 0.7 * p[f"gates.{i}"] * y * ref.rms(y, 1e-6) * p[f"post_weights.{i}"]
        n = h * ref.rms(h, 1e-6) * p[f"weights.{i}"]
    (n * w.double()).sum().backward()
    assert ref.rel(out, n) <= 3e-2
    for k, v in stack.named_parameters():
        assert ref.rel(v.grad, p[k].grad) <= 0.1, (k, ref.rel(v.grad, p[k].grad))


def test_second_derivatives_raise_and_unused_outputs(mod):
    torch.manual_seed(2)
    y = torch.randn(4, 64, device="cuda", requires_grad=True)
    r = torch.randn(4, 64, device="cuda", requires_grad=True)
    w = torch.ones(64, device="cuda", requires_grad=True)
    h, n = mod.ResidualNorm.apply(y, r, w, None, 1.0, w, 1e-6)
    grads = torch.autograd.grad(h.sum(), (y, r), retain_graph=True)     # no gradient of n
    assert torch.equal(grads[1], torch.ones_like(r))
    g, = torch.autograd.grad(n.square().sum(), y, create_graph=True)    # none of h
    with pytest.raises(RuntimeError, match="first derivatives"):
        g.sum().backward()


@pytest.mark.parametrize("decay", ["token", "head"])
def test_prompt_then_steps_match_one_pass(mod, selective, decay):
    """With the projections replaced by the values of their 4-bit codes (rounded to bf16), prompts and steps equal one
    pass up to bf16 roundings of the weights and activations: 5e-2."""
    torch.manual_seed(3)
    stack = mod.Stack([mod.LinearLayer(64, 1, 2, K=64, V=64, decay=decay), selective.SelectiveLayer(64, 128, rank=32)],
                      64).quantize_()
    with torch.no_grad():
        for m in stack.mixers:
            for k, q in m.q4.items():
                getattr(m, k).copy_(selective.dequantize(*q))
    u = torch.randn(3, 70, 64, device="cuda").bfloat16()
    states = stack.new_states(5)
    slots = torch.tensor([4, 1, 0], dtype=torch.int32, device="cuda")
    outs = [stack.prompt(u[:, :66].contiguous(), states, slots)]
    outs += [stack.step(u[:, t].contiguous(), states, slots)[:, None] for t in range(66, 70)]
    with torch.no_grad():
        want = stack(u)
    assert ref.rel(torch.cat(outs, 1), want) <= 5e-2
    assert bool((states[0][[2, 3]] == 0).all())
    lens = [40, 0, 30]
    cu = torch.tensor([0, 40, 40, 70], dtype=torch.int32, device="cuda")
    packed = u[:1]
    a = stack.prompt(packed, states, slots, cu)
    b = [stack.prompt(packed[:, s:e].contiguous(), stack.new_states(5), slots[:1]) for s, e in ((0, 40), (40, 70))]
    assert ref.rel(a, torch.cat(b, 1)) <= 1e-2 and len(lens) == 3


def test_training_step_and_decode_step_in_graphs(mod):
    torch.manual_seed(4)
    stack = mod.Stack([mod.LinearLayer(64, 1, K=64, V=64), mod.LinearLayer(64, 1, K=64, V=64, decay="head")], 64)
    u, w = torch.randn(2, 100, 64, device="cuda").bfloat16(), torch.randn(2, 100, 64, device="cuda").bfloat16()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(2):
            (stack(u) * w).sum().backward()
    torch.cuda.current_stream().wait_stream(side)
    want = {k: v.grad.clone() / 2 for k, v in stack.named_parameters()}
    for v in stack.parameters():
        v.grad = None
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        (stack(u) * w).sum().backward()
    g.replay()
    torch.cuda.synchronize()
    for k, v in stack.named_parameters():
        # twice a gradient, halved: bf16 sums of two equal values are exact
        assert torch.equal(v.grad, want[k]), k
    stack.quantize_()
    states, slots = stack.new_states(3), torch.tensor([2, 0], dtype=torch.int32, device="cuda")
    tok = torch.randn(2, 64, device="cuda").bfloat16()
    first = stack.step(tok, states, slots).clone()
    states2 = stack.new_states(3)
    torch.cuda.synchronize()
    g2 = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g2):
        out = stack.step(tok, states2, slots)
    g2.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, first) and all(torch.equal(a, b) for a, b in zip(states, states2))


def test_saved_and_loaded(mod):
    torch.manual_seed(5)
    a, b = (mod.LinearLayer(64, 1, K=64, V=64) for _ in range(2))
    assert a.q4 is None
    with pytest.raises(RuntimeError, match="quantize_"):
        a.step(torch.randn(1, 64, device="cuda").bfloat16(), a.new_states(1), torch.zeros(1, dtype=torch.int32, device="cuda"))
    b.load_state_dict(a.quantize_().state_dict())
    assert all(torch.equal(x, y) for k in a.q4 for x, y in zip(a.q4[k], b.q4[k]))
    b.load_state_dict(mod.LinearLayer(64, 1, K=64, V=64).state_dict())
    assert b.q4 is None


def test_example(mod):
    spec = importlib.util.spec_from_file_location("example", os.path.join(ROOT, "examples", "linear_layer.py"))
    ex = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ex)
    losses, out = ex.main(steps=3)
    assert len(losses) == 3 and all(x == x for x in losses) and torch.isfinite(out.float()).all()
