"""GPU edges of the selective scan where sums overflow or lose terms and rates are
infinite, against closed forms or the 64-bit definition."""
import pytest
import torch

import selective_reference as R
from conftest import rel_fro

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_chunked_gdn_gb300 import binding
    binding.load()
    return binding


def cuda(d):
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()}


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("state,adjoint", [(1e30, 1e30), (1e19, 2e18)])
def test_bwd_infinite_rate_gradients(gdn, sign, state, adjoint):
    """No decay and no inputs: dA is the number of tokens times state times adjoint.  Every term is infinite in fp32,
    or every tile finite and the sum of three not: the gradient is an infinity with its sign, not a NaN."""
    T, D, S = 48, 4, 4
    one, bc = torch.ones(1, T, D, device="cuda"), torch.zeros(1, T, 1, S, device="cuda")
    full = lambda v: torch.full((1, D, S), v, device="cuda")
    g = gdn.gdn_selective_scan_bwd(one, one, torch.zeros(D, S, device="cuda"), bc, bc, one, softplus=False,
                                   h0=full(sign * state), dht=full(adjoint))
    assert torch.all(g["dA"] == sign * float("inf"))


@pytest.mark.parametrize("S,D", [(16, 9984), (64, 2560)])
def test_bwd_parameter_sums_keep_small_terms(gdn, S, D):
    """Sequences of 2048 tokens that one CTA walks from end to start, where the last four are 2^24 and the others 1:
    with dout = 1, B = 1, C = 0, no decay and dht = 1 / S, dD and ddt_bias are the sum of x, every term exact.  A lane
    adds up to four terms of a tile (three roundings), the tiles with compensation (two), the lanes of a channel
    (four): 9 * 2^-24 of a sum of positive terms.  dA is the sum of dt / S times the state before the token: up to 16 terms
    of a tile a lane (15), two for the tiles, four for the state's own sum of 2^24s: 21 * 2^-24."""
    T, u = 2048, 2.0 ** -24
    x = torch.ones(1, T, D, device="cuda")
    x[:, -4:] = 2.0 ** 24
    one, B = torch.ones_like(x), torch.ones(1, T, 1, S, device="cuda")
    zero = torch.zeros(D, device="cuda")
    g = gdn.gdn_selective_scan_bwd(x, 0.5 * one, torch.zeros(D, S, device="cuda"), B, torch.zeros_like(B), one,
                                   softplus=False, D=zero, dt_bias=zero, dht=torch.full((1, D, S), 1 / S, device="cuda"))
    want = x.double().sum((0, 1))
    for k in ("dD", "ddt_bias"):
        assert ((g[k].double() - want).abs() <= 9 * u * want).all(), k
    before = 0.5 * (x[0].double().cumsum(0) - x[0].double())
    want = (0.5 / S * before.sum(0))[:, None]
    assert ((g["dA"].double() - want).abs() <= 21 * u * want).all()


def test_bwd_infinite_skip_gradients(gdn):
    """The sum of dD over the tiles stays an infinity, too."""
    x = torch.full((1, 48, 4), 1e30, device="cuda")
    bc = torch.ones(1, 48, 1, 4, device="cuda")
    zero = torch.zeros(4, device="cuda")
    g = gdn.gdn_selective_scan_bwd(x, torch.ones_like(x), torch.zeros(4, 4, device="cuda"), bc, torch.zeros_like(bc), x,
                                   softplus=False, D=zero, dt_bias=zero, dht=torch.full((1, 4, 4), -1e30, device="cuda"))
    assert torch.all(g["dD"] == float("inf"))


def test_bwd_infinite_bias_gradients(gdn):
    """.. and that of ddt_bias: steps so small that the states stay finite (else adjoint times state times a rate of
    0 is a NaN of its own, in each token's ddelta)."""
    x = torch.full((1, 48, 4), 1e30, device="cuda")
    bc = torch.ones(1, 48, 1, 4, device="cuda")
    g = gdn.gdn_selective_scan_bwd(x, torch.full_like(x, 1e-30), torch.zeros(4, 4, device="cuda"), bc,
                                   torch.zeros_like(bc), x, softplus=False, dt_bias=torch.zeros(4, device="cuda"),
                                   dht=torch.full((1, 4, 4), -1e30, device="cuda"))
    assert torch.all(g["ddelta"] == -float("inf")) and torch.all(g["ddt_bias"] == -float("inf"))


def offsets(lens):
    return torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device="cuda")


def infinite_rates(T, D, S, G, lens=None, seed=3):
    """Some states forget everything at each token: a rate of -infinity, or one whose base-2 form overflows."""
    inp = R.make_scan(2, T, D, S, G, "f32", init=True, lens=lens, seed=seed)
    inp["A"][:, 1], inp["A"][::2, 2] = -float("inf"), -3e38
    return inp


@pytest.mark.parametrize("T,D,S,G,lens", [(21, 6, 4, 1, None), (16, 8, 8, 2, None), (1, 5, 16, 1, None),
                                          (37, 40, 16, 2, None), (700, 6, 30, 1, None),
                                          (0, 10, 16, 2, [300, 0, 5, 129])])
def test_infinite_rates(gdn, T, D, S, G, lens):
    """Outputs and states are those of the definition, whatever the last tile's padding; bar as for other rates."""
    inp = infinite_rates(T, D, S, G, lens)
    y, ht = gdn.gdn_selective_scan_fwd(**cuda(inp), cu_seqlens=None if lens is None else offsets(lens))
    y_ref, ht_ref = R.scan(**inp, lens=lens)
    assert rel_fro(y.cpu(), y_ref) <= 1e-5 and rel_fro(ht.cpu(), ht_ref) <= 1e-5


@pytest.mark.parametrize("T,D,S,G,lens", [(21, 6, 4, 1, None), (37, 40, 16, 2, None), (200, 6, 30, 1, None),
                                          (0, 10, 16, 2, [130, 0, 5, 70])])
def test_bwd_infinite_rates(gdn, T, D, S, G, lens):
    """The gradients that the definition has then: all but those of the steps, where it is 0 times infinity."""
    inp = infinite_rates(T, D, S, G, lens)
    g = torch.Generator().manual_seed(5)
    dout, dht = torch.randn(inp["x"].shape, generator=g), torch.randn(inp["h0"].shape, generator=g)
    got = gdn.gdn_selective_scan_bwd(**cuda(inp), dout=dout.cuda(), dht=dht.cuda(),
                                     cu_seqlens=None if lens is None else offsets(lens))
    want = R.scan_grads(inp, dout, dht, lens=lens)
    for k in ("x", "A", "B", "C", "D", "z", "h0"):
        assert rel_fro(got["d" + k].cpu(), want[k]) <= 5e-5, k


@pytest.mark.parametrize("N,T", [(3, 1), (70, 1), (2, 5)])
def test_step_infinite_rates(gdn, N, T):
    inp = R.make_scan(N, T, 24, 16, 2, "f32", init=True, seed=6)
    inp["A"][:, 1], inp["A"][::2, 2] = -float("inf"), -3e38
    y_ref, ht_ref = R.scan(**inp)
    d = cuda(inp)
    state = d.pop("h0").clone()
    y = gdn.gdn_selective_scan_step(**d, state=state)
    assert rel_fro(y.cpu(), y_ref) <= 1e-5 and rel_fro(state.cpu(), ht_ref) <= 1e-5


CUT = [(3, 700, 6, 30, 1, None), (2, 3000, 64, 16, 1, None), (1, 0, 10, 16, 2, [300, 0, 700, 3, 128, 129]),
       (200, 40, 32, 16, 1, None)]   # the last: whole sequences, several to a CTA


@pytest.mark.parametrize("B,T,D,S,G,lens", CUT)
def test_states_in_place(gdn, B, T, D, S, G, lens):
    """ht given as h0: bit for bit the call with a tensor of its own, cut sequences too."""
    inp = cuda(R.make_scan(B, T, D, S, G, "f32", init=True, lens=lens, seed=7))
    cu = None if lens is None else offsets(lens)
    y, ht = gdn.gdn_selective_scan_fwd(**inp, cu_seqlens=cu)
    for _ in range(3):
        state = inp["h0"].clone()
        y2, _ = gdn.gdn_selective_scan_fwd(**(inp | {"h0": state}), ht=state, cu_seqlens=cu)
        assert torch.equal(y, y2) and torch.equal(ht, state)


@pytest.mark.parametrize("B,T,D,S,G,lens", CUT)
@pytest.mark.parametrize("which", ["h0", "dht"])
def test_bwd_states_in_place(gdn, B, T, D, S, G, lens, which):
    """dh0 written over h0 or over dht (the C call; the binding allocates its own)."""
    inp = cuda(R.make_scan(B, T, D, S, G, "f32", init=True, lens=lens, seed=8))
    cu = None if lens is None else offsets(lens)
    dout, dht = torch.randn_like(inp["x"]), torch.randn_like(inp["h0"])
    want = gdn.gdn_selective_scan_bwd(**inp, dout=dout, dht=dht, cu_seqlens=cu)
    p = gdn._scan_problem(inp["x"], inp["delta"], inp["A"], inp["B"], inp["C"], inp["D"], inp["z"], inp["dt_bias"], True,
                          cu, ())
    over = {"h0": inp["h0"].clone(), "dht": dht.clone()}
    out = {k: torch.empty_like(v) for k, v in want.items() if k not in ("dh0", "workspace")}
    ws = want["workspace"]
    st = gdn.load().gdn_selective_scan_bwd(
        p, *(inp[k].data_ptr() for k in ("x", "delta", "A", "B", "C", "D", "z", "dt_bias")), over["h0"].data_ptr(),
        0 if cu is None else cu.data_ptr(), dout.data_ptr(), over["dht"].data_ptr(),
        *(out[k].data_ptr() for k in ("dx", "ddelta", "dA", "dB", "dC", "dD", "dz", "ddt_bias")),
        over[which].data_ptr(), ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == gdn.GDN_OK
    assert torch.equal(over[which], want["dh0"]) and all(torch.equal(v, want[k]) for k, v in out.items())


@pytest.mark.parametrize("low", [float("-inf"), torch.finfo(torch.bfloat16).min])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_masked_steps(gdn, dtype, low):
    """Tokens whose delta is -infinity or the type's lowest number make no step: they keep the state and get no
    gradient of their step; a sequence of nothing else keeps its initial state."""
    lens = [40, 17, 300]
    inp = R.make_scan(1, 0, 32, 16, 2, dtype, init=True, lens=lens, seed=9)
    inp["delta"][:, 5:60:3], inp["delta"][:, 40:57], inp["delta"][:, 100] = low, low, low
    y, ht = gdn.gdn_selective_scan_fwd(**cuda(inp), cu_seqlens=offsets(lens))
    y_ref, ht_ref = R.scan(**inp, lens=lens)
    more = 2.0 ** -8 if dtype == "bf16" else 0.0
    assert rel_fro(y.double().cpu(), y_ref) <= 1e-5 + more and rel_fro(ht.cpu(), ht_ref) <= 1e-5
    assert torch.equal(ht[1].cpu(), inp["h0"][1])
    state = inp["h0"].cuda()
    rest = {k: v for k, v in cuda(inp).items() if k != "h0"}
    ys = gdn.gdn_selective_scan_step(**rest, state=state, cu_seqlens=offsets(lens))
    assert rel_fro(ys.double().cpu(), y_ref) <= 1e-5 + more and torch.equal(state[1].cpu(), inp["h0"][1])
    g = torch.Generator().manual_seed(10)
    dout, dht = torch.randn(y_ref.shape, generator=g).to(inp["x"].dtype), torch.randn(ht_ref.shape, generator=g)
    got = gdn.gdn_selective_scan_bwd(**cuda(inp), dout=dout.cuda(), dht=dht.cuda(), cu_seqlens=offsets(lens))
    want = R.scan_grads(inp, dout, dht, lens=lens)
    for k, v in inp.items():
        assert rel_fro(got["d" + k].double().cpu(), want[k]) <= 5e-5 + (more if v.dtype == torch.bfloat16 else 0.0), k
    assert not got["ddelta"][:, 40:57].any()
