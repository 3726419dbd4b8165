"""Linear attention and the norms over tensors of more than 2^31 elements, and over one very long sequence.  The last
head's (row's, slot's) results are compared with those of a call on it alone; the two calls may cut a sequence
differently, so that only sums' orders differ."""
import pytest
import torch

import linear_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def gdn():
    from gated_deltanet_chunked_gdn_gb300 import binding
    binding.load()
    return binding


@pytest.mark.parametrize("dtype,T,Hv", [(BF, 66000, 256), (F32, 34000, 512)])
def test_more_than_2_31_elements(gdn, dtype, T, Hv):
    """Tolerances: two fp32 results of the same sums in another order, 4e-6; bf16 outputs may round to neighbours
    (2^-8 of the value, where the sums differ at a border), 1e-3 over all."""
    torch.manual_seed(0)
    K, V = 64, 128
    assert T * Hv * V > 2 ** 31
    q, k = torch.randn(1, T, 1, K, device=DEV).to(dtype), (torch.randn(1, T, 1, K, device=DEV) * 0.1).to(dtype)
    g = -0.2 * torch.rand(1, T, Hv, device=DEV)
    v = torch.empty(1, T, Hv, V, device=DEV, dtype=dtype)
    for h in range(0, Hv, 32):
        v[:, :, h:h + 32] = torch.randn(1, T, 32, V, device=DEV, dtype=dtype)
    o, ht = gdn.gdn_linear_attn_fwd(q, k, v, g, scale=0.25)
    last = v[:, :, -1:].contiguous(), g[:, :, -1:].contiguous()
    wo, wh = gdn.gdn_linear_attn_fwd(q, k, *last, scale=0.25)
    tol = 1e-3 if dtype is BF else 4e-6
    assert ref.rel(o[:, :, -1:], wo) < tol and ref.rel(ht[:, -1:], wh) < 4e-6
    assert ref.rel(o[:, -300:, :2], gdn.gdn_linear_attn_fwd(q, k, v[:, :, :2].contiguous(), g[:, :, :2].contiguous(),
                                                            scale=0.25)[0][:, -300:]) < tol
    got = gdn.gdn_linear_attn_bwd(q, k, v, g, o, scale=0.25)
    want = gdn.gdn_linear_attn_bwd(q, k, *last, o[:, :, -1:].contiguous(), scale=0.25)
    assert ref.rel(got["dv"][:, :, -1:], want["dv"]) < tol
    assert ref.rel(got["dg"][:, :, -1:], want["dg"]) < 1e-5


def test_one_long_sequence_is_its_parts(gdn):
    torch.manual_seed(1)
    T, cut = 150000, 70016
    q, k = torch.randn(1, T, 1, 64, device=DEV).to(BF), (0.1 * torch.randn(1, T, 1, 64, device=DEV)).to(BF)
    v, g = torch.randn(1, T, 1, 64, device=DEV).to(BF), -0.01 * torch.rand(1, T, 1, device=DEV)
    o, ht = gdn.gdn_linear_attn_fwd(q, k, v, g, scale=0.25)
    a = lambda t: t[:, :cut].contiguous()  # noqa: E731
    b = lambda t: t[:, cut:].contiguous()  # noqa: E731
    o1, h1 = gdn.gdn_linear_attn_fwd(*map(a, (q, k, v, g)), scale=0.25)
    o2, h2 = gdn.gdn_linear_attn_fwd(*map(b, (q, k, v, g)), scale=0.25, h0=h1)
    assert ref.rel(torch.cat((o1, o2), 1), o) < 1e-3 and ref.rel(h2, ht) < 4e-6
    d = gdn.gdn_linear_attn_bwd(q, k, v, g, o, scale=0.25)
    d2 = gdn.gdn_linear_attn_bwd(*map(b, (q, k, v, g)), b(o), scale=0.25, h0=h1)
    d1 = gdn.gdn_linear_attn_bwd(*map(a, (q, k, v, g)), a(o), scale=0.25, dht=d2["dh0"])
    for n in ("dq", "dk", "dv", "dg"):
        assert ref.rel(torch.cat((d1[n], d2[n]), 1), d[n]) < (1e-5 if n == "dg" else 1e-3), n


def test_pool_of_more_than_2_31_elements(gdn):
    torch.manual_seed(2)
    slots, Hv, K, V = 1030, 32, 256, 256
    pool = torch.zeros(slots, Hv, K, V, device=DEV)
    assert pool.numel() > 2 ** 31
    at = torch.tensor([slots - 1, 0], dtype=torch.int32, device=DEV)
    q, k = torch.randn(2, 1, 1, K, device=DEV).to(BF), torch.randn(2, 1, 1, K, device=DEV).to(BF)
    v, g = torch.randn(2, 1, Hv, V, device=DEV).to(BF), -torch.rand(2, 1, Hv, device=DEV)
    pool[-1] = 1.0
    o = gdn.gdn_linear_attn_step(q, k, v, g, pool, state_indices=at)
    small = torch.zeros(2, Hv, K, V, device=DEV)
    small[0] = 1.0
    assert torch.equal(o, gdn.gdn_linear_attn_step(q, k, v, g, small))
    assert torch.equal(pool[[-1, 0]], small) and bool((pool[1:-1] == 0).all())
    pool[-1] = 7.0
    gdn.gdn_linear_attn_fwd(q, k, v, g, ht=pool, state_indices=at)
    assert torch.equal(pool[[-1, 0]], gdn.gdn_linear_attn_fwd(q, k, v, g)[1])


def test_norms_over_more_than_2_31_elements(gdn):
    torch.manual_seed(3)
    rows, H, V = 540000, 32, 128
    x = torch.empty(rows, H, V, device=DEV, dtype=BF)
    for r in range(0, rows, 60000):
        x[r:r + 60000] = torch.randn(60000, H, V, device=DEV, dtype=BF)
    w = torch.rand(V, device=DEV)
    y, rstd = gdn.gdn_gated_norm_fwd(x, x, w, save_rstd=True)
    a = x[-1000:].contiguous()
    assert torch.equal(y[-1000:], gdn.gdn_gated_norm_fwd(a, a, w)[0])
    d = gdn.gdn_gated_norm_bwd(x, x, w, rstd, y)
    e = gdn.gdn_gated_norm_bwd(a, a, w, rstd[-1000:].contiguous(), y[-1000:].contiguous())
    assert torch.equal(d["dx"][-1000:], e["dx"]) and torch.equal(d["dz"][-1000:], e["dz"])
    del d, rstd
    x, y = x.view(rows, H * V), y.view(rows, H * V)
    w = torch.rand(H * V, device=DEV)
    h, n, rs = gdn.gdn_residual_norm_fwd(y, x, post_weight=w, weight=w, save_rstd=True)
    b = [t[-100:].contiguous() for t in (y, x, h, n, rs)]
    h2, n2, _ = gdn.gdn_residual_norm_fwd(b[0], b[1], post_weight=w, weight=w)
    assert torch.equal(h[-100:], h2) and torch.equal(n[-100:], n2)
    d = gdn.gdn_residual_norm_bwd(y, x, rs, h, n, post_weight=w, weight=w)
    e = gdn.gdn_residual_norm_bwd(b[0], b[1], b[4], b[2], b[3], post_weight=w, weight=w)
    assert torch.equal(d["dy"][-100:], e["dy"]) and torch.equal(d["dresidual"][-100:], e["dresidual"])
