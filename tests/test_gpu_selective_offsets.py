"""GPU: tensors of more than 2^31 elements (or bytes of weights) through the selective
layer's operators; the ends are compared with the 64-bit definitions on slices that
stand for themselves.  Bars as at small sizes (each operator's own tests)."""
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
    yield binding
    torch.cuda.empty_cache()


def big(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s, dtype=torch.bfloat16: torch.randn(*s, generator=g, device="cuda", dtype=dtype)


def test_scan_bwd(gdn):
    """States and adjoints fade within a few tokens, so the last tokens' gradients come from the last 120."""
    T, D, S = 66000, 33000, 4
    rn = big(1)
    x, delta, dout, B, C = rn(1, T, D), rn(1, T, D), rn(1, T, D), rn(1, T, 1, S), rn(1, T, 1, S)
    A, bias = torch.full((D, S), -8.0, device="cuda"), torch.full((D,), 2.0, device="cuda")
    got = gdn.gdn_selective_scan_bwd(x, delta, A, B, C, dout, dt_bias=bias)
    for sl in (slice(0, 5), slice(D - 5, D)):
        cut = lambda t: t[:, -120:, sl].cpu()
        inp = {"x": cut(x), "delta": cut(delta), "A": A[sl].cpu(), "B": B[:, -120:].cpu(), "C": C[:, -120:].cpu(),
               "dt_bias": bias[sl].cpu()}
        want = R.scan_grads(inp, cut(dout))
        for k in ("x", "delta"):
            assert rel_fro(got["d" + k][:, -40:, sl].double().cpu(), want[k][:, -40:]) <= 5e-5 + BF16


def test_conv_bwd(gdn):
    T, D = 70000, 32768
    rn = big(2)
    x, dout = rn(1, T, D), rn(1, T, D)
    w = rn(D, 4, dtype=torch.float32) / 2
    got = gdn.gdn_causal_conv1d_bwd(x, w, dout)
    for sl in (slice(0, 8), slice(D - 8, D)):
        leaves = [t.double().requires_grad_() for t in (x[:, -60:, sl].cpu(), w[sl].cpu())]
        y, _ = R.conv(*leaves)
        (dx,) = torch.autograd.grad((y * dout[:, -60:, sl].double().cpu()).sum(), leaves[:1])
        assert rel_fro(got["dx"][:, -40:, sl].double().cpu(), dx[:, -40:]) <= 1e-5 + BF16


@pytest.mark.parametrize("n", [2, 70])
def test_step(gdn, n):
    """The pool's last slots lie past 2^31 states."""
    slots, D, S = 9000, 4096, 64
    pool = torch.zeros(slots, D, S, device="cuda")
    inp = R.make_scan(n, 1, D, S, 1, "f32", seed=3)
    del inp["h0"]
    h0 = torch.randn(n, D, S, generator=torch.Generator().manual_seed(4))
    at = torch.arange(slots - n, slots)
    pool[at] = h0.cuda()
    y = gdn.gdn_selective_scan_step(**{k: v.cuda() for k, v in inp.items()}, state=pool, state_indices=at.int().cuda())
    few = [0, n - 1]
    small = {k: v[few] if k in ("x", "delta", "B", "C", "z") else v for k, v in inp.items()}
    y_ref, ht_ref = R.scan(**small, h0=h0[few])
    assert rel_fro(y[few].cpu(), y_ref) <= 1e-5 and rel_fro(pool[at[few]].cpu(), ht_ref) <= 1e-5
    assert not pool[: slots - n].any()


def test_q4(gdn):
    N, K, group = 140000, 32768, 128
    g = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (0.01 * (0.5 + torch.rand(N, K // group, generator=g, device="cuda"))).bfloat16()
    x = torch.randn(3, K, generator=g, device="cuda").bfloat16()
    y = gdn.gdn_q4_matvec(x, q, scales)
    for rows in (slice(0, 20), slice(N - 20, N)):
        w = R.q4_weights(q[rows].cpu(), scales[rows].cpu())
        want, size = x.double().cpu() @ w.t(), x.double().abs().cpu() @ w.abs().t()
        assert ((y[:, rows].double().cpu() - want).abs() <= 2e-6 * size + BF16 * want.abs()).all()
