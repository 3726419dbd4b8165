"""Cut sequences of the selective scan in the shapes that are copied 16 bytes at a
time, the backward's longest segment, and packed training through the layer, against
the 64-bit definitions.  Bars as for whole sequences: outputs 1e-5, gradients 5e-5
(relative Frobenius), and a rounding of bf16, 2^-8, for tensors of that type."""
import pytest
import torch

import selective_reference as R
from conftest import rel_fro

pytestmark = pytest.mark.gpu
BF16 = 2.0 ** -8


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_chunked_gdn_gb300 import binding
    binding.load()
    return binding


def cuda(d):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()}


def offsets(lens):
    return None if lens is None else torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32,
                                                  device="cuda")


def tol(t, f32):
    return f32 + (BF16 if t.dtype == torch.bfloat16 else 0.0)


SHAPES = [(2, 700, 64, 16, 1, None), (1, 650, 128, 16, 2, None), (2, 500, 64, 8, 1, None), (1, 500, 32, 64, 1, None),
          (1, 0, 64, 16, 1, [300, 0, 700, 3, 128, 129, 257]), (1, 0, 96, 32, 3, [129, 400, 16])]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,D,S,G,lens", SHAPES)
def test_cut_forward(gdn, dtype, B, T, D, S, G, lens):
    inp = R.make_scan(B, T, D, S, G, dtype, init=True, lens=lens, seed=D + S)
    y, ht = gdn.gdn_selective_scan_fwd(**cuda(inp), cu_seqlens=offsets(lens))
    y_ref, ht_ref = R.scan(**inp, lens=lens)
    assert rel_fro(y.double().cpu(), y_ref) <= tol(y, 1e-5)
    assert rel_fro(ht.cpu(), ht_ref) <= 1e-5


def check_bwd(got, want, inp):
    for k, v in inp.items():
        assert rel_fro(got["d" + k].double().cpu(), want[k]) <= tol(v, 5e-5), k


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,D,S,G,lens", SHAPES)
def test_cut_backward(gdn, dtype, B, T, D, S, G, lens):
    inp = R.make_scan(B, T, D, S, G, dtype, init=True, lens=lens, seed=D + S + 1)
    g = torch.Generator().manual_seed(3)
    dout, dht = torch.randn(inp["x"].shape, generator=g).to(inp["x"].dtype), torch.randn(inp["h0"].shape, generator=g)
    got = gdn.gdn_selective_scan_bwd(**cuda(inp), dout=dout.cuda(), dht=dht.cuda(), cu_seqlens=offsets(lens))
    check_bwd(got, R.scan_grads(inp, dout, dht, lens=lens), inp)


def test_backward_longer_than_a_segment_may_be(gdn):
    """Sequences of more than 8192 tokens, as many as fill the device, are cut all the same.  All but two of them have
    no upstream gradient, so that the parameters' are those two's."""
    B, T, D, S, two = 77, 8200, 8, 4, [3, 70]
    inp = R.make_scan(B, T, D, S, 1, "f32", init=True, seed=9)
    g = torch.Generator().manual_seed(4)
    dout, dht = torch.zeros(B, T, D), torch.zeros(B, D, S)
    dout[two], dht[two] = torch.randn(2, T, D, generator=g), torch.randn(2, D, S, generator=g)
    got = gdn.gdn_selective_scan_bwd(**cuda(inp), dout=dout.cuda(), dht=dht.cuda())
    each = {k for k in inp if k not in ("A", "D", "dt_bias")}
    small = {k: v[two] if k in each else v for k, v in inp.items()}
    for k in each:
        rest = got["d" + k].clone()
        rest[two] = 0
        assert not rest.any(), k
    got = {"d" + k: got["d" + k][two] if k in each else got["d" + k] for k in inp}
    check_bwd(got, R.scan_grads(small, dout[two], dht[two]), small)


def test_layer_gradients_packed(gdn):
    """Packed training through the layer: parameter gradients as for equal lengths (activations rounded to bf16 on one
    side only, four times on the way out and again on the way back: 5e-2)."""
    from gated_deltanet_chunked_gdn_gb300 import selective_layer as mod
    torch.manual_seed(0)
    layer = mod.SelectiveLayer(32, 48, states=8, groups=2, rank=32)
    lens = [33, 0, 1, 150, 2, 14]
    u = torch.randn(1, 200, 32, device="cuda").bfloat16().requires_grad_()
    w = torch.randn(1, 200, 32, device="cuda")
    (layer(u, offsets(lens)).float() * w).sum().backward()
    p = {k: v.detach().double().cpu().requires_grad_() for k, v in layer.named_parameters()}
    u64 = u.detach().double().cpu().requires_grad_()
    x, z = (u64 @ p["in_proj"].t()).chunk(2, dim=-1)
    x, _ = R.conv(x, p["conv_weight"], p["conv_bias"], lens=lens)
    dt, B, C = (x @ p["x_proj"].t()).split([32, 16, 16], dim=-1)
    y, _ = R.scan(x, dt @ p["dt_proj"].t(), -torch.exp(p["A_log"]), B.unflatten(-1, (2, 8)), C.unflatten(-1, (2, 8)),
                  D=p["Dskip"], z=z, dt_bias=p["dt_bias"], lens=lens)
    ((y @ p["out_proj"].t()) * w.double().cpu()).sum().backward()
    for k, v in layer.named_parameters():
        assert rel_fro(v.grad.double().cpu(), p[k].grad) <= 5e-2, k
    assert rel_fro(u.grad.double().cpu(), u64.grad) <= 5e-2


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,D,S,G,lens", [(5, 20, 50, 16, 1, None), (5, 700, 6, 30, 1, None),
                                            (1, 0, 64, 16, 2, [300, 0, 700, 1, 129]), (1, 0, 7, 3, 1, [5, 0, 1, 40, 16])])
def test_final_states_into_a_pool(gdn, dtype, B, T, D, S, G, lens):
    """Rows of a pool as a map gives them, bit for bit the states in order; no state outside, no other row touched."""
    inp = cuda(R.make_scan(B, T, D, S, G, dtype, init=True, lens=lens, seed=T))
    y, ht = gdn.gdn_selective_scan_fwd(**inp, cu_seqlens=offsets(lens))
    slots = [6, -1, 0, 9, 3]                                     # nine rows: the fourth is past them
    pool = torch.full((9, D, S), 7.0, device="cuda")
    y2, same = gdn.gdn_selective_scan_fwd(**inp, cu_seqlens=offsets(lens), ht=pool,
                                          state_indices=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    assert same is pool and torch.equal(y, y2)
    for row in range(9):
        assert torch.equal(pool[row], ht[slots.index(row)]) if row in slots else torch.all(pool[row] == 7.0)


def test_malformed_offsets_leave_the_pool(gdn):
    inp = cuda(R.make_scan(1, 30, 16, 4, 1, "f32", seed=11))
    inp.pop("h0")
    pool = torch.full((4, 16, 4), 7.0, device="cuda")
    for bad in ([0, 20, 10, 30], [0, 10, 20, 29], [0, 10, 40, 30]):
        gdn.gdn_selective_scan_fwd(**inp, cu_seqlens=torch.tensor(bad, dtype=torch.int32, device="cuda"), ht=pool,
                                   state_indices=torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda"))
        assert torch.all(pool == 7.0)
