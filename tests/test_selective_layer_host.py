"""The selective layer's own arithmetic on the CPU (no GPU): the operators that it
calls are replaced by their definitions in 64 bits, with the library's rules for
slots."""
import pytest
import torch

import selective_reference as R
from gated_deltanet_chunked_gdn_gb300 import selective_layer as mod


def lens_of(cu):
    return None if cu is None else (cu[1:] - cu[:-1]).tolist()


def conv_fwd(x, weight, bias=None, activation="silu", conv_state=None, cache_indices=None, has_initial_state=None,
             cu_seqlens=None):
    """gdn_causal_conv1d_fwd from zero initial inputs; a slot outside the pool means that nothing is written."""
    lens = lens_of(cu_seqlens)
    if lens is not None and min(lens) < 0:
        return torch.zeros_like(x)
    y, final = R.conv(x, weight, bias, activation, lens=lens)
    if conv_state is not None:
        for n, slot in enumerate(cache_indices.tolist()):
            if 0 <= slot < conv_state.shape[0]:
                conv_state[slot] = final[n].to(conv_state.dtype)
    return y.to(x.dtype)


def scan_fwd(x, delta, A, B, C, D=None, z=None, dt_bias=None, h0=None, cu_seqlens=None, ht=None,
             output_final_state=True, state_indices=None):
    """gdn_selective_scan_fwd; malformed offsets leave ht unwritten, and so does a row outside the pool."""
    lens = lens_of(cu_seqlens)
    if ht is None:
        ht = torch.full((len(lens or x), *A.shape), float("nan"))
    if lens is not None and (min(lens) < 0 or sum(lens) != x.shape[1]):
        return torch.zeros_like(x), ht
    y, h = R.scan(x, delta, A, B, C, D=D, z=z, dt_bias=dt_bias, h0=h0, lens=lens)
    for n, row in enumerate(range(len(h)) if state_indices is None else state_indices.tolist()):
        if 0 <= row < len(ht):
            ht[row] = h[n]
    return y.to(x.dtype), ht


@pytest.fixture
def layer(monkeypatch):
    monkeypatch.setattr(mod.gdn, "gdn_causal_conv1d_fwd", conv_fwd)
    monkeypatch.setattr(mod.gdn, "gdn_selective_scan_fwd", scan_fwd)
    torch.manual_seed(0)
    return mod.SelectiveLayer(8, 6, states=4, rank=32, device="cpu")


def prompt(layer, slots, cu=None):
    torch.manual_seed(1)
    u = torch.randn(3, 5, 8).bfloat16() if cu is None else torch.randn(1, cu[-1], 8).bfloat16()
    conv, scan = layer.new_states(5)
    conv.fill_(3.0), scan.fill_(7.0)
    out = layer.prompt(u, (conv, scan), torch.tensor(slots, dtype=torch.int32),
                       None if cu is None else torch.tensor(cu, dtype=torch.int32))
    return out, conv, scan


@pytest.mark.parametrize("slots", [[-1, 2, 0], [1, 5, 4], [3, -7, 99], [4, 1, -1], [-1, -1, 5]])
@pytest.mark.parametrize("cu", [None, [0, 4, 4, 11]])
def test_prompt_slots_outside_the_pool(layer, slots, cu):
    """A sequence whose slot is outside the pool has no state: both pools' other rows keep their values to the bit,
    and the sequences with slots get the states that they get alone."""
    out, conv, scan = prompt(layer, slots, cu)
    ref, conv_ref, scan_ref = prompt(layer, [0, 1, 2], cu)
    assert torch.equal(out, ref)
    for row in range(5):
        if row in slots:
            assert torch.equal(scan[row], scan_ref[slots.index(row)])
            assert torch.equal(conv[row], conv_ref[slots.index(row)])
        else:
            assert torch.all(scan[row] == 7.0) and torch.all(conv[row] == 3.0)


def test_prompt_malformed_offsets_leave_the_scan_states(layer):
    """The scan writes no final states then, so none may reach the pool."""
    _, _, scan = prompt(layer, [3, 0, 1], [0, 8, 2, 11])
    assert torch.all(scan == 7.0)


def conv_bwd(x, weight, dout, bias=None, activation="silu", cu_seqlens=None):
    leaves = [t.double().requires_grad_() for t in (x, weight, bias)]
    with torch.enable_grad():
        y, _ = R.conv(*leaves, activation, lens=lens_of(cu_seqlens))
    g = torch.autograd.grad(y, leaves, dout.double())
    return {"dx": g[0].to(x.dtype), "dweight": g[1].float(), "dbias": g[2].float()}


def scan_bwd(x, delta, A, B, C, dout, D=None, z=None, dt_bias=None, cu_seqlens=None):
    inp = {"x": x, "delta": delta, "A": A, "B": B, "C": C, "D": D, "z": z, "dt_bias": dt_bias}
    with torch.enable_grad():
        g = R.scan_grads(inp, dout, lens=lens_of(cu_seqlens))
    return {"d" + k: g[k].to(v.dtype) for k, v in inp.items()}


@pytest.fixture
def training(layer, monkeypatch):
    monkeypatch.setattr(mod.gdn, "gdn_causal_conv1d_bwd", conv_bwd)
    monkeypatch.setattr(mod.gdn, "gdn_selective_scan_bwd", scan_bwd)
    return layer


def test_second_derivatives_are_refused(training):
    """They are not built: a penalty on a gradient raises rather than leaving the operators' part of it out."""
    u = torch.randn(2, 7, 8).bfloat16().requires_grad_()
    (du,) = torch.autograd.grad(training(u).float().square().sum(), u, create_graph=True)
    with pytest.raises(RuntimeError, match="first derivatives only"):
        du.float().square().sum().backward()


@pytest.mark.parametrize("op", ["conv", "scan"])
def test_second_derivatives_are_refused_for_constant_upstream_gradients(training, op):
    """The incoming gradient is a constant here, the operator's inputs are not."""
    w = torch.randn(6, 6).requires_grad_()
    v = torch.randn(1, 9, 6)
    u = torch.randn(1, 9, 6).requires_grad_()
    if op == "conv":
        y = mod.CausalConv1d.apply(u @ w, torch.randn(6, 4), torch.randn(6), None)
    else:
        bc = torch.randn(1, 9, 1, 4)
        y = mod.SelectiveScan.apply(u @ w, v, -torch.rand(6, 4), bc, bc, torch.randn(6), v, torch.randn(6), None)
    (du,) = torch.autograd.grad(y.sum(), u, create_graph=True)
    with pytest.raises(RuntimeError, match="first derivatives only"):
        du.square().sum().backward()


@pytest.mark.parametrize("cu", [None, [0, 4, 4, 11]])
def test_first_derivatives(training, cu):
    """Through torch's own operators the layer would have these (with and without a graph of them): bf16 roundings
    on the way, once a tensor, on both sides alike; the recurrences themselves are the same numbers."""
    u = torch.randn(*((2, 7) if cu is None else (1, 11)), 8).bfloat16()
    cu = None if cu is None else torch.tensor(cu, dtype=torch.int32)
    params = list(training.parameters())
    plain = torch.autograd.grad(training(u, cu).float().square().sum(), params)
    graph = torch.autograd.grad(training(u, cu).float().square().sum(), params, create_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(plain, graph))

    x, z = (u @ training.in_proj.t()).chunk(2, dim=-1)
    x, _ = R.conv(x, training.conv_weight, training.conv_bias, lens=lens_of(cu))
    x = x.bfloat16()
    dt, B, C = training._split(x @ training.x_proj.t())
    y, _ = R.scan(x, dt @ training.dt_proj.t(), -torch.exp(training.A_log), B, C, D=training.Dskip, z=z,
                  dt_bias=training.dt_bias, lens=lens_of(cu))
    want = torch.autograd.grad((y.bfloat16() @ training.out_proj.t()).float().square().sum(), params)
    for a, b in zip(plain, want):
        assert (a.double() - b.double()).norm() <= 2e-2 * b.double().norm()


def q4_matvec(x, qweight, scales):
    return (x.double() @ R.q4_weights(qweight, scales).t()).to(x.dtype)


def conv_step(x, weight, bias, activation, conv_state, cache_indices):
    at = cache_indices.long()
    y, final = R.conv(x, weight, bias, activation, conv_state[at])
    conv_state[at] = final.to(conv_state.dtype)
    return y.to(x.dtype)


def scan_step(x, delta, A, B, C, state, D=None, z=None, dt_bias=None, state_indices=None):
    at = state_indices.long()
    y, h = R.scan(x, delta, A, B, C, D=D, z=z, dt_bias=dt_bias, h0=state[at])
    state[at] = h.float()
    return y.to(x.dtype)


@pytest.fixture
def serving(layer, monkeypatch):
    monkeypatch.setattr(mod.gdn, "gdn_causal_conv1d_fwd", conv_step)
    monkeypatch.setattr(mod.gdn, "gdn_selective_scan_step", scan_step)
    monkeypatch.setattr(mod.gdn, "gdn_q4_matvec", q4_matvec)
    layer = mod.SelectiveLayer(32, 64, states=4, rank=32, device="cpu")
    with torch.no_grad():
        layer.A_log += 0.1
    return layer


def step(layer):
    u = torch.randn(2, 32, generator=torch.Generator().manual_seed(2)).bfloat16()
    return layer.step(u, layer.new_states(2), torch.tensor([1, 0], dtype=torch.int32))


def test_step_wants_the_4_bit_weights(serving):
    with pytest.raises(RuntimeError, match="quantize_"):
        step(serving)


def test_4_bit_weights_are_saved_and_loaded(serving):
    """A checkpoint of a quantized layer gives a new one the same step, whose own weights need not be near the codes."""
    want = step(serving.quantize_())
    other = mod.SelectiveLayer(32, 64, states=4, rank=32, device="cpu")
    other.load_state_dict(serving.state_dict())
    assert torch.equal(step(other), want)
    assert all(torch.equal(a, b) for k in serving.q4 for a, b in zip(serving.q4[k], other.q4[k]))
    outer = torch.nn.Sequential(mod.SelectiveLayer(32, 64, states=4, rank=32, device="cpu"))   # within another module
    outer.load_state_dict({"0." + k: v for k, v in serving.state_dict().items()})
    assert torch.equal(step(outer[0]), want)


def test_4_bit_weights_do_not_outlive_a_checkpoint_without_them(serving):
    plain = mod.SelectiveLayer(32, 64, states=4, rank=32, device="cpu")
    serving.quantize_().load_state_dict(plain.state_dict())
    with pytest.raises(RuntimeError, match="quantize_"):
        step(serving)
    assert torch.equal(step(serving.quantize_()), step(plain.quantize_()))


def test_4_bit_weights_move_with_the_layer(serving):
    moved = serving.quantize_().to("meta")
    tensors = [t for pair in moved.q4.values() for t in pair] + [moved.A]
    assert len(tensors) == 9 and all(t.is_meta for t in tensors)
    assert all(moved.q4[k][0].dtype == torch.uint8 for k in moved.q4)
