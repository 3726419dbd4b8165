"""GPU gradients of the selective state space scan and of the causal convolution
against automatic differentiation of their definitions in 64 bits.

Bars (relative Frobenius).  A gradient is a sum of products of the forward's
quantities, each with the forward's relative error (1e-5 allowed there), of two
recurrences, state and adjoint, and their sums over tokens or channels may
cancel: 5e-5.  Gradients of bf16 tensors round once more, by 2^-8 of a value."""
import pytest
import torch

import selective_reference as R
from conftest import rel_fro

pytestmark = pytest.mark.gpu
F32 = 5e-5
TOL = {torch.bfloat16: F32 + 2.0 ** -8, torch.float32: F32}
NAMES = {"x": "dx", "delta": "ddelta", "A": "dA", "B": "dB", "C": "dC", "D": "dD", "z": "dz", "dt_bias": "ddt_bias",
         "h0": "dh0"}


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
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")


def upstream(inp, lens=None, end=True, seed=1):
    g = torch.Generator().manual_seed(seed)
    N = len(lens) if lens is not None else inp["x"].shape[0]
    dout = torch.randn(inp["x"].shape, generator=g).to(inp["x"].dtype)
    return dout, torch.randn(N, *inp["A"].shape, generator=g) if end else None


def check(gdn, inp, lens=None, softplus=True, end=True, seed=1):
    dout, dht = upstream(inp, lens, end, seed)
    got = gdn.gdn_selective_scan_bwd(**cuda(inp), dout=dout.cuda(), dht=dht.cuda() if end else None,
                                     softplus=softplus, cu_seqlens=offsets(lens) if lens is not None else None)
    torch.cuda.synchronize()
    want = R.scan_grads(inp, dout, dht, softplus=softplus, lens=lens)
    for k, name in NAMES.items():
        if inp.get(k) is None:
            assert got[name] is None
            continue
        assert got[name].dtype == inp[k].dtype and got[name].shape == inp[k].shape
        err = rel_fro(got[name].double().cpu(), want[k])
        assert err <= TOL[inp[k].dtype], (name, err)
    return got


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,D,S,G", [(1, 1, 1, 1, 1), (2, 5, 7, 3, 1), (1, 16, 64, 4, 2), (3, 33, 48, 8, 4),
                                       (2, 50, 300, 16, 2), (1, 47, 36, 12, 3), (2, 35, 40, 24, 1),
                                       (1, 40, 24, 32, 2), (2, 31, 20, 50, 1), (1, 40, 12, 64, 4)])
def test_bwd_shapes(gdn, dtype, B, T, D, S, G):
    check(gdn, R.make_scan(B, T, D, S, G, dtype, init=T % 2 == 1, seed=T), end=T % 3 != 0)


@pytest.mark.parametrize("gate,bias,skip,softplus", [(False, True, True, True), (True, False, False, True),
                                                     (False, False, True, False), (True, True, False, False)])
def test_bwd_optional_parts(gdn, gate, bias, skip, softplus):
    inp = R.make_scan(2, 40, 32, 16, 1, "f32", gate=gate, bias=bias and softplus, skip=skip, seed=3)
    if not softplus:
        inp["delta"] = 0.05 * inp["delta"].abs()
    check(gdn, inp, softplus=softplus)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bwd_packed(gdn, dtype):
    lens = [5, 0, 1, 16, 17, 90, 0, 31, 1]
    check(gdn, R.make_scan(1, 0, 44, 16, 2, dtype, init=True, lens=lens, seed=4), lens)


@pytest.mark.parametrize("S", [2, 8, 16, 30, 64])
def test_bwd_cut_sequences(gdn, S):
    check(gdn, R.make_scan(2, 600, 6, S, 1, "f32", init=True, seed=5))
    lens = [300, 0, 500, 3, 128, 129]
    check(gdn, R.make_scan(1, 0, 10, S, 2, "f32", init=True, lens=lens, seed=6), lens)


def test_bwd_many_sequences(gdn):
    """More sequences than CTAs share: a CTA walks several and keeps its sums."""
    lens = [1 + i % 5 for i in range(700)]
    check(gdn, R.make_scan(1, 0, 300, 4, 1, "f32", init=True, lens=lens, seed=7), lens)


@pytest.mark.parametrize("i", range(8))
def test_bwd_random_draw(gdn, i):
    r = torch.Generator().manual_seed(70 + i)
    ri = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=r))
    G = ri(1, 4)
    lens = [ri(0, 90) for _ in range(ri(1, 6))] + [1] if i % 3 else None
    check(gdn, R.make_scan(ri(1, 3), ri(1, 150), G * ri(1, 40), ri(1, 40), G, "bf16" if i % 2 else "f32",
                           gate=bool(ri(0, 1)), init=bool(ri(0, 1)), lens=lens, seed=i), lens, seed=i)


def test_bwd_slices_and_runs_alike(gdn):
    """Column slices of one wide row as inputs; bit for bit the contiguous call, twice and on another stream."""
    B, T, D, S, G = 2, 300, 24, 8, 2
    inp = R.make_scan(B, T, D, S, G, "bf16", seed=7)
    dout = upstream(inp)[0].cuda()
    wide = torch.zeros(B, T, 3 * D + 2 * G * S + 1, dtype=torch.bfloat16, device="cuda")
    views, at = {}, 1
    for k in ("x", "delta", "z", "B", "C"):
        n = D if k in ("x", "delta", "z") else G * S
        v = wide[..., at:at + n]
        at += n
        views[k] = v if n == D else v.unflatten(-1, (G, S))
        views[k].copy_(inp[k])
    a = gdn.gdn_selective_scan_bwd(**(cuda(inp) | views), dout=dout)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        b = gdn.gdn_selective_scan_bwd(**cuda(inp), dout=dout)
    torch.cuda.synchronize()
    for k in NAMES.values():
        assert (a[k] is None and b[k] is None) or torch.equal(a[k], b[k]), k


def test_bwd_against_differences(gdn):
    """<gradient, v> against central differences of the 64-bit forward."""
    inp = R.make_scan(1, 40, 12, 5, 2, "f32", init=True, seed=8)
    dout, dht = upstream(inp)
    got = gdn.gdn_selective_scan_bwd(**cuda(inp), dout=dout.cuda(), dht=dht.cuda())
    d64 = {k: v.double() for k, v in inp.items()}
    loss = lambda v: (lambda y, h: (y * dout.double()).sum() + (h * dht.double()).sum())(*R.scan(**v))
    g = torch.Generator().manual_seed(9)
    for k, name in NAMES.items():
        e = torch.randn(inp[k].shape, generator=g, dtype=torch.float64)
        diff = (loss(d64 | {k: d64[k] + 1e-5 * e}) - loss(d64 | {k: d64[k] - 1e-5 * e})) / 2e-5
        have = got[name].double().cpu()
        assert abs(diff - (have * e).sum()) <= F32 * have.norm() * e.norm(), name


def test_bwd_malformed_and_refusals(gdn):
    inp = cuda(R.make_scan(1, 30, 16, 4, 1, "f32", seed=11))
    inp.pop("h0")
    cu = torch.tensor([0, 20, 10, 30], dtype=torch.int32, device="cuda")
    p = gdn._scan_problem(inp["x"], inp["delta"], inp["A"], inp["B"], inp["C"], None, None, None, True, cu, ())
    got = gdn.gdn_selective_scan_bwd(**inp, dout=torch.zeros_like(inp["x"]), cu_seqlens=cu)
    assert gdn.gdn_selective_scan_get_device_status(p, got["workspace"]) == gdn.DEV_BAD_CU_SEQLENS
    with pytest.raises(ValueError):
        gdn.gdn_selective_scan_bwd(**inp, dout=torch.zeros(1, 29, 16, device="cuda"))
    with pytest.raises(ValueError):
        gdn.gdn_selective_scan_bwd(**inp, dout=torch.zeros_like(inp["x"]), dht=torch.zeros(1, 16, 5, device="cuda"))
    with pytest.raises(gdn.GDNError):
        gdn.gdn_selective_scan_bwd(**inp, dout=torch.zeros_like(inp["x"]),
                                   workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))


# ------------------------------------------------------- causal convolution

def check_conv(gdn, dtype, B, T, D, W, act, lens=None, init=False, final=False, bias=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    if lens is not None:
        B, T = 1, sum(lens)
    N = len(lens) if lens is not None else B
    rn = lambda *s: torch.randn(*s, generator=g)
    inp = {"x": rn(B, T, D).to(dt), "weight": rn(D, W) * W ** -0.5, "bias": 0.1 * rn(D) if bias else None,
           "initial_state": rn(N, W - 1, D).to(dt) if init else None}
    dout, dfin = rn(B, T, D).to(dt), rn(N, W - 1, D).to(dt) if final else None
    got = gdn.gdn_causal_conv1d_bwd(**cuda(inp), dout=dout.cuda(), activation=act,
                                    dfinal_state=dfin.cuda() if final else None,
                                    cu_seqlens=offsets(lens) if lens is not None else None)
    torch.cuda.synchronize()
    leaves = {k: v.double().requires_grad_() for k, v in inp.items() if v is not None}
    y, fin = R.conv(**leaves, activation=act, lens=lens)
    total = (y * dout.double()).sum() + ((fin * dfin.double()).sum() if final else 0.0)
    want = dict(zip(leaves, torch.autograd.grad(total, list(leaves.values()), allow_unused=True)))
    # sums of at most W products (dx) or of all tokens' (dweight, dbias), each with a few roundings and two
    # approximate SiLU factors (about 2^-22 each)
    for k, name in (("x", "dx"), ("weight", "dweight"), ("bias", "dbias"), ("initial_state", "dinitial_state")):
        if inp[k] is None:
            assert got[name] is None
        elif want[k] is not None and want[k].numel():
            err = rel_fro(got[name].double().cpu(), want[k])
            assert err <= (1e-5 if inp[k].dtype == torch.float32 else 1e-5 + 2.0 ** -8), (name, err)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("W", [1, 2, 3, 4])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_conv_bwd_fixed(gdn, dtype, W, act):
    check_conv(gdn, dtype, 3, 150, 48, W, act, init=W > 1 and act == "silu", final=W > 1, seed=W)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_conv_bwd_packed(gdn, dtype):
    """Sequences that are empty, shorter than the window, or cross the 256-token runs."""
    lens = [5, 1, 0, 130, 2, 64, 300, 3, 256, 255, 1, 0]
    for W in (2, 4):
        check_conv(gdn, dtype, 1, 0, 72, W, "silu", lens=lens, init=True, final=True, seed=W)
    check_conv(gdn, dtype, 1, 0, 72, 4, "none", lens=lens, bias=False, seed=9)


def test_conv_bwd_long(gdn):
    check_conv(gdn, "f32", 2, 1500, 8, 4, "silu", init=True, final=True, seed=3)
    check_conv(gdn, "bf16", 1, 700, 1048, 3, "silu", seed=4)


def test_conv_bwd_malformed_and_refusals(gdn):
    x = torch.randn(1, 60, 32, device="cuda")
    w = torch.randn(32, 4, device="cuda")
    bad = torch.tensor([0, 10, 70, 60], dtype=torch.int32, device="cuda")
    got = gdn.gdn_causal_conv1d_bwd(x, w, torch.ones_like(x), cu_seqlens=bad, activation="none")
    ref = gdn.gdn_causal_conv1d_bwd(x[:, :10].contiguous(), w, torch.ones(1, 10, 32, device="cuda"),
                                    activation="none")
    torch.cuda.synchronize()
    assert torch.equal(got["dx"][:, :10], ref["dx"]) and torch.equal(got["dweight"], ref["dweight"])
    for kw in (dict(x=x[..., :12].contiguous()), dict(weight=torch.zeros(32, 5, device="cuda"))):
        args = dict(x=x, weight=w) | kw
        if args["x"].shape[-1] == 12:
            args["weight"] = torch.zeros(12, 4, device="cuda")
        with pytest.raises(gdn.GDNError):
            gdn.gdn_causal_conv1d_bwd(**args, dout=torch.zeros_like(args["x"]))
    with pytest.raises(ValueError):
        gdn.gdn_causal_conv1d_bwd(x, w, torch.zeros(1, 59, 32, device="cuda"))
    with pytest.raises(ValueError):
        gdn.gdn_causal_conv1d_bwd(x, w, x, initial_state=torch.zeros(1, 4, 32, device="cuda"))
