"""GPU parity of the product with 4-bit weights against its definition in 64 bits.

Bars, per output: codes, zero points and their differences are exact, products
are exact in fp32 (8 bits times at most 24, in three parts for fp32 x), and the
fp32 sums of K products and their scaled group sums round by at most about
(K + groups) 2^-24 of sum |x w|, in practice by the square root of that: 2e-6 of
sum |x w| covers K = 8192.  A bf16 output rounds by 2^-8 of its value."""
import pytest
import torch

import selective_reference as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_chunked_gdn_gb300 import binding
    binding.load()
    return binding


def make(M, N, K, group, dtype, sdt, zeros, bias, seed=0):
    g = torch.Generator().manual_seed(seed)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}
    return {"x": torch.randn(M, K, generator=g).to(dt[dtype]),
            "qweight": torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8),
            "scales": (0.01 * (0.5 + torch.rand(N, K // group, generator=g))).to(dt[sdt]),
            "zeros": torch.randint(0, 16, (N, K // group), generator=g, dtype=torch.uint8) if zeros else None,
            "bias": torch.randn(N, generator=g) if bias else None}


def check(gdn, i):
    y = gdn.gdn_q4_matvec(**{k: v.cuda() if v is not None else None for k, v in i.items()})
    torch.cuda.synchronize()
    w = R.q4_weights(i["qweight"], i["scales"], i["zeros"])
    x = i["x"].double()
    want, size = x @ w.t(), x.abs() @ w.abs().t()
    if i["bias"] is not None:
        want, size = want + i["bias"].double(), size + i["bias"].double().abs()
    bound = 2e-6 * size + (2.0 ** -8 * want.abs() if i["x"].dtype == torch.bfloat16 else 0.0)
    err = (y.double().cpu() - want).abs()
    assert y.dtype == i["x"].dtype and bool((err <= bound).all()), float((err / bound).max())
    return y


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group", [32, 64, 96, 128, 256])
@pytest.mark.parametrize("M,N", [(1, 1), (1, 40), (3, 17), (8, 64), (9, 33), (32, 100), (45, 16)])
def test_q4_shapes(gdn, dtype, group, M, N):
    check(gdn, make(M, N, 3 * group, group, dtype, "f32" if group == 64 else "bf16", zeros=M % 2 == 0, bias=N % 2 == 0,
                    seed=M))


@pytest.mark.parametrize("K,group", [(32, 32), (128, 128), (8192, 128), (8192, 8192), (4128, 32), (5120, 1024)])
def test_q4_lengths(gdn, K, group):
    for M in (1, 5):
        check(gdn, make(M, 200, K, group, "bf16", "bf16", True, True, seed=K))
    check(gdn, make(2, 50, K, group, "f32", "f32", True, False, seed=K + 1))


def test_q4_many_rows_of_weights(gdn):
    """Enough of them for 32 a warp, and a last tile that is not full."""
    check(gdn, make(6, 14700, 192, 64, "bf16", "bf16", True, True, seed=2))
    check(gdn, make(14, 14603, 160, 32, "bf16", "f32", True, False, seed=4))
    check(gdn, make(2, 14700, 256, 128, "f32", "f32", False, True, seed=6))


@pytest.mark.parametrize("N,K", [(4096, 4096), (1000, 11008), (12288, 2048)])
def test_q4_large(gdn, N, K):
    check(gdn, make(4, N, K, 32, "bf16", "bf16", False, True, seed=5))


def test_q4_strided_rows_leading_dims_and_streams(gdn):
    i = {k: v.cuda() if v is not None else None for k, v in make(6, 70, 256, 64, "bf16", "bf16", True, True).items()}
    y = gdn.gdn_q4_matvec(**i)
    wide = torch.zeros(6, 301, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:259] = i["x"]
    assert torch.equal(y, gdn.gdn_q4_matvec(**(i | {"x": wide[:, 3:259]})))
    assert torch.equal(y.view(2, 3, 70), gdn.gdn_q4_matvec(**(i | {"x": i["x"].view(2, 3, 256)})))
    s, out = torch.cuda.Stream(), torch.zeros_like(y)
    s.wait_stream(torch.cuda.current_stream())
    gdn.gdn_q4_matvec(**i, y=out, stream=s.cuda_stream)
    s.synchronize()
    assert torch.equal(y, out)
    assert gdn.gdn_q4_matvec(**(i | {"x": i["x"][:0]})).shape == (0, 70)


def test_q4_rows_do_not_mix_and_extremes(gdn):
    """A row with an infinity or NaN leaves the others alone; fp32 near its largest value stays finite."""
    for dtype in ("bf16", "f32"):
        i = make(4, 40, 128, 32, dtype, "f32", False, False, seed=3)
        want = check(gdn, i)
        i["x"][1, 7], i["x"][3, 9] = float("inf"), float("nan")
        y = gdn.gdn_q4_matvec(**{k: v.cuda() if v is not None else None for k, v in i.items()})
        assert torch.equal(y[[0, 2]], want[[0, 2]]) and not torch.isfinite(y[3]).any()
        code = (i["qweight"][:, 3] >> 4).double() - 8
        sign = torch.sign(code)
        assert torch.equal(y[1].double().cpu()[sign != 0], (sign * float("inf"))[sign != 0])
    i = make(1, 16, 32, 32, "f32", "f32", False, False)
    i["x"].zero_()
    i["x"][0, 0], i["scales"][:] = 3.4e38, 1e-3
    assert torch.isfinite(check(gdn, i)).all()


def test_q4_refusals(gdn):
    i = {k: v.cuda() if v is not None else None for k, v in make(2, 8, 128, 64, "bf16", "f32", True, True).items()}
    call = lambda **kw: gdn.gdn_q4_matvec(**(i | kw))
    for kw in (dict(x=i["x"][:, :64]), dict(x=i["x"].half()), dict(scales=i["scales"][:4]), dict(x=i["x"].cpu()),
               dict(zeros=i["zeros"].int()), dict(bias=i["bias"].bfloat16()),
               dict(x=i["x"].t().contiguous().t())):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(gdn.GDNError):   # groups of 16
        call(scales=torch.ones(8, 8, device="cuda"), zeros=None)
