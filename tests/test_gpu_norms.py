"""The norms around a block on the GPU against their definitions in 64 bits.

Tolerances: bf16 outputs are rounded once, 2^-8 of the value, and what is rounded is an fp32 result (2e-6): 2^-8 as a
relative Frobenius error.  fp32 outputs: a mean of D squares added over threads and then over a tree (about 2^-24
sqrt(D / threads)), rsqrt (2^-22), a sigmoid (2^-22) and a handful of products: 1e-6; sums over rows add their 2^-24
like their squares: 2e-6."""
import pytest
import torch

import linear_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def tol(t):
    return 2 ** -8 if t.dtype is BF else 2e-6


@pytest.fixture(scope="module")
def gdn():
    from gated_deltanet_chunked_gdn_gb300 import binding
    binding.load()
    return binding


def off(got, want, terms):
    """Relative error; over a single element r (a - xhat a xhat) is r a times eps r^2, the difference of two terms that
    agree in all but the last few bits: each is off by a few 2^-24 of itself, so its error is taken relative to r a."""
    if got.shape[-1] > 1:
        return ref.rel(got, want)
    return float(torch.linalg.vector_norm(got.double() - want) / torch.linalg.vector_norm(terms))


def gated(rows, H, V, dtype, gate=True, seed=0):
    torch.manual_seed(seed)
    x, dy = (2 * torch.randn(rows, H, V, device=DEV)).to(dtype), torch.randn(rows, H, V, device=DEV).to(dtype)
    z = torch.randn(rows, H, V, device=DEV).to(dtype) if gate else None
    return x, z, 1 + 0.1 * torch.randn(V, device=DEV), dy


def check_gated(gdn, x, z, w, dy, eps=1e-5):
    y, rstd = gdn.gdn_gated_norm_fwd(x, z, w, eps=eps, save_rstd=True)
    assert ref.rel(y, ref.gated_norm(x, z, w, eps)) < tol(y)
    got = gdn.gdn_gated_norm_bwd(x, z, w, rstd, dy)
    want = ref.gated_norm(x, z, w, eps, dy)
    gate = z.double() * torch.sigmoid(z.double()) if z is not None else 1.0
    ra = dy.double() * gate * w.double() * ref.rms(x.double(), eps)
    for n, t in want.items():
        assert (off(got[n], t, ra) if n == "dx" else ref.rel(got[n], t)) < tol(got[n]), n
    return y, got


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("V", [1, 3, 8, 16, 21, 37, 64, 100, 128, 130, 200, 256, 257, 512, 520, 1000, 2048, 4100, 9001,
                               16384])
def test_gated_widths(gdn, V, dtype):
    for rows, H in ((1, 1), (5, 3), (67, 2)):
        check_gated(gdn, *gated(rows, H, V, dtype))
    check_gated(gdn, *gated(7, 2, V, dtype, gate=False))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_gated_many_rows(gdn, dtype):
    check_gated(gdn, *gated(3001, 17, 128, dtype))


@pytest.mark.parametrize("dtype", [F32, BF])
def test_gated_slices_and_odd_addresses(gdn, dtype):
    x, z, w, dy = gated(33, 4, 64, dtype)
    y0, g0 = check_gated(gdn, x, z, w, dy)
    wide = torch.full((33, 3 * 256 + 1), float("nan"), device=DEV).to(dtype)
    for at in (256, 257):
        xs, zs = wide[:, at:at + 256].unflatten(1, (4, 64)), wide[:, 512:768].unflatten(1, (4, 64))
        if at == 257:
            zs = z
        xs.copy_(x)
        zs.copy_(z)
        y, g = check_gated(gdn, xs, zs, w, dy)
        assert ref.rel(y, y0) < tol(y)
    store = torch.empty(33 * 256 + 1, device=DEV).to(dtype)
    odd = store[1:].view(33, 4, 64)
    odd.copy_(x)
    check_gated(gdn, odd, z, w, dy)


def test_gated_extremes(gdn):
    """A row of zeros has a finite norm and gradients; gates far out saturate; NaN stays in its row."""
    x, z, w, dy = gated(4, 2, 128, F32)
    x[0] = 0
    z[1] = 200.0
    z[2] = -200.0
    y, rstd = gdn.gdn_gated_norm_fwd(x, z, w, eps=1e-5, save_rstd=True)
    got = gdn.gdn_gated_norm_bwd(x, z, w, rstd, dy)
    assert bool((y[0] == 0).all()) and all(bool(torch.isfinite(t).all()) for t in (y, got["dx"], got["dz"], got["dweight"]))
    check_gated(gdn, x, z, w, dy)
    x[3, 1, 5] = float("nan")
    y2, _ = gdn.gdn_gated_norm_fwd(x, z, w, eps=1e-5)
    assert bool(torch.isnan(y2[3, 1]).all()) and torch.equal(y2[:3], y[:3]) and torch.equal(y2[3, 0], y[3, 0])


def residual(rows, D, dtype, rdtype, post=True, gate="channel", pre=True, seed=0):
    torch.manual_seed(seed)
    r = lambda dt: torch.randn(rows, D, device=DEV).to(dt)  # noqa: E731
    w = lambda: 1 + 0.1 * torch.randn(D, device=DEV)  # noqa: E731
    return dict(y=r(dtype), residual=3 * r(rdtype), post_weight=w() if post else None,
                gate={"none": None, "channel": w() - 0.5, "element": torch.rand(rows, D, device=DEV).to(dtype)}[gate],
                weight=w() if pre else None), r(rdtype), r(dtype) if pre else None


def check_residual(gdn, x, dh, dn, scale=0.6, eps=1e-5):
    h, n, rstd = gdn.gdn_residual_norm_fwd(**x, residual_scale=scale, eps=eps, save_rstd=True)
    args = (x["y"], x["residual"], x["post_weight"], x["gate"], scale, x["weight"], eps)
    wh, wn = ref.residual_norm(*args)
    assert ref.rel(h, wh) < tol(h)
    assert (n is None) == (wn is None) and (n is None or ref.rel(n, wn) < tol(n))
    got = gdn.gdn_residual_norm_bwd(x["y"], x["residual"], rstd, dh, dn, post_weight=x["post_weight"], gate=x["gate"],
                                    residual_scale=scale, weight=x["weight"])
    if dh is None and dn is None:
        return h, n, got
    want = ref.residual_norm(*args, dh=dh, dn=dn)
    # over a single column every gradient is made of differences and sums that may cancel: errors are taken relative to
    # the terms, dh and the two that the norms' backward passes subtract, which add like their squares.  Those two are
    # r a and r a hhat^2 with hhat = h r, and h, a sum of two parts that may cancel, is off by 2^-24 of the parts: by
    # that times r in hhat, 2 r |parts| in hhat^2
    d = dh.double().abs() if dh is not None else 0.0
    if dn is not None:
        r, res = ref.rms(wh, eps), x["residual"].double()
        d = d + (dn.double() * x["weight"].double()).abs() * r * (1 + 2 * r * (res.abs() + (wh - res).abs()))
    du = d * scale * (x["gate"].double() if x["gate"] is not None else 1.0)
    ra = du * x["post_weight"].double() * ref.rms(x["y"].double(), eps) if x["post_weight"] is not None else du
    terms = {"dy": ra, "dresidual": d, "dpost_weight": du, "dgate": d * scale,
             "dweight": dn.double() if dn is not None else None}
    for name in ("dy", "dresidual", "dpost_weight", "dgate", "dweight"):
        assert (got[name] is None) == (name not in want), name
        if name in want:
            e = off(got[name], want[name], terms[name])
            assert e < tol(got[name]), (name, e)
    return h, n, got


TYPES = [(F32, F32), (BF, F32), (BF, BF)]


@pytest.mark.parametrize("dtype,rdtype", TYPES)
@pytest.mark.parametrize("D", [1, 7, 64, 100, 114, 256, 257, 512, 1000, 1024, 1030, 2048, 2500, 4096, 5001, 8192, 16000,
                               16384])
def test_residual_widths(gdn, D, dtype, rdtype):
    for rows in (1, 37):
        check_residual(gdn, *residual(rows, D, dtype, rdtype))


@pytest.mark.parametrize("dtype,rdtype", TYPES)
@pytest.mark.parametrize("gate", ["none", "channel", "element"])
@pytest.mark.parametrize("post,pre", [(True, True), (True, False), (False, True), (False, False)])
def test_residual_parts(gdn, post, pre, gate, dtype, rdtype):
    for D in (256, 1001):
        check_residual(gdn, *residual(29, D, dtype, rdtype, post, gate, pre))


def test_residual_many_rows_without_dh(gdn):
    x, _, dn = residual(5003, 512, BF, F32, gate="element")
    check_residual(gdn, x, None, dn)


def test_residual_in_place_and_slices(gdn):
    x, dh, dn = residual(19, 512, BF, BF)
    h, n, rstd = gdn.gdn_residual_norm_fwd(**x, save_rstd=True)
    r = x["residual"].clone()
    h2, n2, _ = gdn.gdn_residual_norm_fwd(**{**x, "residual": r}, h=r)
    assert h2 is r and torch.equal(h, r) and torch.equal(n, n2)
    wide = torch.full((19, 1100), float("nan"), device=DEV, dtype=BF)
    for at in (8, 3):
        ys = wide[:, at:at + 512]
        ys.copy_(x["y"])
        assert ref.rel(gdn.gdn_residual_norm_fwd(**{**x, "y": ys})[1], n) < 2 ** -8
        check_residual(gdn, {**x, "y": ys}, dh, dn)


def test_empty_and_leading_dimensions(gdn):
    x, z, w, dy = gated(0, 2, 64, BF)
    y, rstd = gdn.gdn_gated_norm_fwd(x, z, w, save_rstd=True)
    assert y.shape == (0, 2, 64) and bool((gdn.gdn_gated_norm_bwd(x, z, w, rstd, dy)["dweight"] == 0).all())
    r, dh, dn = residual(0, 64, BF, F32)
    assert bool((gdn.gdn_residual_norm_bwd(r["y"], r["residual"], torch.empty(0, 2, device=DEV), dh, dn,
                                           post_weight=r["post_weight"], gate=r["gate"],
                                           weight=r["weight"])["dweight"] == 0).all())
    x, z, w, dy = gated(6, 2, 64, BF)
    a = gdn.gdn_gated_norm_fwd(x, z, w)[0]
    b = gdn.gdn_gated_norm_fwd(x.view(2, 3, 2, 64), z.view(2, 3, 2, 64), w)[0]
    assert torch.equal(a, b.view(6, 2, 64))


def test_the_same_bits_captured_and_on_another_stream(gdn):
    x, z, w, dy = gated(300, 4, 128, BF)
    r, dh, dn = residual(300, 520, BF, F32, gate="element")

    def run(stream=None):
        y, rs = gdn.gdn_gated_norm_fwd(x, z, w, save_rstd=True, stream=stream)
        g = gdn.gdn_gated_norm_bwd(x, z, w, rs, dy, stream=stream)
        h, n, rs2 = gdn.gdn_residual_norm_fwd(**r, save_rstd=True, stream=stream)
        g2 = gdn.gdn_residual_norm_bwd(r["y"], r["residual"], rs2, dh, dn, post_weight=r["post_weight"],
                                       gate=r["gate"], weight=r["weight"], stream=stream)
        return [y, g["dx"], g["dz"], g["dweight"], h, n, *(g2[k] for k in ("dy", "dresidual", "dgate", "dweight",
                                                                         "dpost_weight"))]

    want = run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = run(side.cuda_stream)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
