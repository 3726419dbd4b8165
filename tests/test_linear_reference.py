"""The 64-bit references of linear attention and of the norms: their gradients against central differences (CPU)."""
import pytest
import torch

import linear_reference as ref

f64 = dict(dtype=torch.float64)


def differences(fn, tensors, step=1e-6):
    """Central differences of the scalar fn over every element of the tensors."""
    out = []
    for t in tensors:
        g = torch.zeros_like(t)
        for i in range(t.numel()):
            old = t.view(-1)[i].item()
            t.view(-1)[i] = old + step
            a = fn()
            t.view(-1)[i] = old - step
            b = fn()
            t.view(-1)[i] = old
            g.view(-1)[i] = (a - b) / (2 * step)
        out.append(g)
    return out


# a difference's error: step^2 times a third derivative of order one, and 1e-16 / step of the function's rounding
TOL = 1e-7


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("cu", [None, [0, 3, 3, 4]])
def test_linear_attention_gradients(per_head, cu):
    torch.manual_seed(0)
    B, T = (2, 4) if cu is None else (1, 4)
    N = B if cu is None else 3
    q, k = torch.randn(B, T, 1, 3, **f64), torch.randn(B, T, 1, 3, **f64)
    v, do = torch.randn(B, T, 2, 2, **f64), torch.randn(B, T, 2, 2, **f64)
    g = -torch.rand(*((2,) if per_head else (B, T, 2)), **f64)
    h0, dht = torch.randn(N, 2, 3, 2, **f64), torch.randn(N, 2, 3, 2, **f64)
    c = None if cu is None else torch.tensor(cu, dtype=torch.int32)

    def loss():
        o, ht = ref.forward(q, k, v, g, 0.7, h0, c)
        return float((o * do).sum() + (ht * dht).sum())

    got = ref.backward(q, k, v, g, do, 0.7, h0, dht, c)
    for name, want in zip(("dq", "dk", "dv", "dg", "dh0"), differences(loss, (q, k, v, g, h0))):
        assert float((got[name] - want).abs().max()) < TOL, name


def test_gated_norm_gradients():
    torch.manual_seed(1)
    x, z, dy, w = torch.randn(3, 2, 5, **f64), torch.randn(3, 2, 5, **f64), torch.randn(3, 2, 5, **f64), torch.randn(5, **f64)
    got = ref.gated_norm(x, z, w, 1e-3, dy)
    want = differences(lambda: float((ref.gated_norm(x, z, w, 1e-3) * dy).sum()), (x, z, w))
    for name, d in zip(("dx", "dz", "dweight"), want):
        assert float((got[name] - d).abs().max()) < TOL, name


@pytest.mark.parametrize("gate", ["none", "channel", "element"])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
def test_residual_norm_gradients(gate, post, pre):
    torch.manual_seed(2)
    y, r, dh, dn = (torch.randn(3, 4, **f64) for _ in range(4))
    pw = torch.randn(4, **f64) if post else None
    w = torch.randn(4, **f64) if pre else None
    gt = {"none": None, "channel": torch.randn(4, **f64), "element": torch.randn(3, 4, **f64)}[gate]

    def loss():
        h, n = ref.residual_norm(y, r, pw, gt, 0.6, w, 1e-3)
        return float((h * dh).sum() + ((n * dn).sum() if pre else 0.0))

    got = ref.residual_norm(y, r, pw, gt, 0.6, w, 1e-3, dh, dn if pre else None)
    names = {"dy": y, "dresidual": r, "dpost_weight": pw, "dgate": gt, "dweight": w}
    names = {k: t for k, t in names.items() if t is not None}
    for (name, _), d in zip(names.items(), differences(loss, list(names.values()))):
        assert float((got[name] - d).abs().max()) < TOL, name
