"""The 64-bit definitions that the selective layer's GPU tests compare with,
checked on the CPU: closed forms, splitting, and gradients by differences."""
import pytest
import torch

import selective_reference as R


def test_scan_closed_forms():
    # one token: h = dt x B (+ decayed h0), y = (C.h + D x) silu(z), by hand
    one = lambda v, *s: torch.tensor(v, dtype=torch.float64).reshape(s)
    y, ht = R.scan(one([3.0], 1, 1, 1), one([0.5], 1, 1, 1), one([-2.0, 0.0], 1, 2), one([1.0, 4.0], 1, 1, 1, 2),
                   one([2.0, -1.0], 1, 1, 1, 2), D=one([10.0], 1), softplus=False, h0=one([1.0, 1.0], 1, 1, 2))
    e = torch.exp(torch.tensor(-1.0, dtype=torch.float64))
    assert torch.allclose(ht[0, 0], torch.stack([e + 1.5, one(7.0)]))
    assert torch.allclose(y.reshape(()), 2 * (e + 1.5) - 7 + 30)
    # no decay (A = 0): the state is a running sum
    x = torch.arange(1.0, 6.0).reshape(1, 5, 1)
    ones = torch.ones(1, 5, 1, 1)
    y, ht = R.scan(x, torch.ones(1, 5, 1), torch.zeros(1, 1), ones, ones, softplus=False)
    assert torch.allclose(y.flatten(), x.double().flatten().cumsum(0)) and ht.item() == 15


def test_scan_packed_and_split():
    lens = [4, 0, 7]
    i = R.make_scan(1, 0, 6, 3, 2, "f32", init=True, lens=lens)
    y, ht = R.scan(**i, lens=lens)
    for n, (a, b) in enumerate([(0, 4), (4, 4), (4, 11)]):
        cut = {k: v[:, a:b] if k in ("x", "delta", "B", "C", "z") else v for k, v in i.items()}
        cut["h0"] = i["h0"][n:n + 1]
        ys, hs = R.scan(**cut)
        assert torch.equal(y[:, a:b], ys) and torch.equal(ht[n], hs[0])


@pytest.mark.parametrize("softplus", [True, False])
def test_scan_gradients_against_differences(softplus):
    i = R.make_scan(2, 9, 4, 3, 2, "f32", init=True, seed=1)
    i = {k: v.double() for k, v in i.items()}
    if not softplus:
        i["delta"], i["dt_bias"] = 0.1 * i["delta"].abs(), 0.1 * i["dt_bias"].abs()
    g = torch.Generator().manual_seed(2)
    dout, dht = torch.randn(2, 9, 4, generator=g), torch.randn(2, 4, 3, generator=g)
    loss = lambda v: (lambda y, h: (y * dout).sum() + (h * dht).sum())(*R.scan(**v, softplus=softplus))
    grads = R.scan_grads(i, dout, dht, softplus=softplus)
    for k, v in i.items():
        e = torch.randn(v.shape, generator=g, dtype=torch.float64)
        eps = 1e-5
        diff = (loss(i | {k: v + eps * e}) - loss(i | {k: v - eps * e})) / (2 * eps)
        assert abs(diff - (grads[k] * e).sum()) <= 1e-8 * (grads[k].norm() * e.norm() + 1)


def test_conv_definition():
    x = torch.tensor([1.0, 2.0, 3.0]).reshape(1, 3, 1)
    w = torch.tensor([[10.0, 1.0]])
    y, final = R.conv(x, w, torch.tensor([0.5]), "none", torch.tensor([4.0]).reshape(1, 1, 1))
    assert y.flatten().tolist() == [41.5, 12.5, 23.5] and final.item() == 3.0


def test_q4_definition():
    q = torch.tensor([[0x98, 0x0F]], dtype=torch.uint8)       # codes 8, 9, 15, 0
    assert R.q4_weights(q, torch.tensor([[2.0]])).tolist() == [[0.0, 2.0, 14.0, -16.0]]
    z = torch.tensor([[9]], dtype=torch.uint8)
    assert R.q4_weights(q, torch.tensor([[1.0]]), z).tolist() == [[-1.0, 0.0, 6.0, -9.0]]
