"""GPU parity of the selective state space scan (prompts and single tokens)
against its definition in 64 bits.

Bars.  The inputs are the same numbers on both sides, so only the kernels' own
rounding counts.  A state is a sum of products of fp32 factors: a decay carries
the rounding of dt (a few 2^-24), of its exponent (|dt A| 2^-24 and ex2's 2^-22)
and is applied once a token, with errors that fade as fast as the state does;
the sums round once a token.  1e-5 of the norm leaves a factor of about ten.  An
output rounds once more to its type: bf16 keeps 8 significant bits, so by at most
2^-8 of each value."""
import pytest
import torch

import selective_reference as R
from conftest import rel_fro

pytestmark = pytest.mark.gpu
F32 = 1e-5
TOL = {"bf16": F32 + 2.0 ** -8, "f32": F32}


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


def check(gdn, inp, dtype, lens=None, softplus=True):
    y, ht = gdn.gdn_selective_scan_fwd(**cuda(inp), softplus=softplus,
                                       cu_seqlens=offsets(lens) if lens is not None else None)
    torch.cuda.synchronize()
    y_ref, ht_ref = R.scan(**inp, softplus=softplus, lens=lens)
    assert y.dtype == inp["x"].dtype and y.shape == inp["x"].shape
    assert rel_fro(y.double().cpu(), y_ref) <= TOL[dtype]
    assert rel_fro(ht.cpu(), ht_ref) <= F32


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,T,D,S,G", [(1, 1, 1, 1, 1), (2, 5, 7, 3, 1), (1, 16, 64, 4, 2), (3, 33, 48, 8, 4),
                                       (2, 100, 130, 16, 2), (1, 47, 36, 12, 3), (2, 65, 40, 24, 1),
                                       (1, 70, 24, 32, 2), (2, 31, 20, 50, 1), (1, 90, 12, 64, 4)])
def test_scan_shapes(gdn, dtype, B, T, D, S, G):
    check(gdn, R.make_scan(B, T, D, S, G, dtype, init=T % 2 == 1, seed=T), dtype)


@pytest.mark.parametrize("gate,bias,skip,softplus", [(False, True, True, True), (True, False, False, True),
                                                     (False, False, True, False), (True, True, False, False)])
def test_scan_optional_parts(gdn, gate, bias, skip, softplus):
    inp = R.make_scan(2, 40, 32, 16, 1, "f32", gate=gate, bias=bias and softplus, skip=skip, seed=3)
    if not softplus:
        inp["delta"] = 0.05 * inp["delta"].abs()
    check(gdn, inp, "f32", softplus=softplus)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_scan_packed(gdn, dtype):
    """Empty and one-token sequences, lengths around the tile's 16 tokens."""
    lens = [5, 0, 1, 16, 17, 130, 0, 31, 1]
    check(gdn, R.make_scan(1, 0, 44, 16, 2, dtype, init=True, lens=lens, seed=4), dtype, lens)


@pytest.mark.parametrize("S", [2, 8, 16, 30, 64])
def test_scan_cut_sequences(gdn, S):
    """Few channels and long sequences: cut into segments that run side by side, the states chained."""
    check(gdn, R.make_scan(2, 700, 6, S, 1, "f32", init=True, seed=5), "f32")
    lens = [300, 0, 700, 3, 128, 129, 257]
    check(gdn, R.make_scan(1, 0, 10, S, 2, "f32", init=True, lens=lens, seed=6), "f32", lens)


@pytest.mark.parametrize("i", range(10))
def test_scan_random_draw(gdn, i):
    r = torch.Generator().manual_seed(50 + i)
    ri = lambda lo, hi: int(torch.randint(lo, hi + 1, (1,), generator=r))
    G = ri(1, 4)
    dtype = "bf16" if i % 2 else "f32"
    lens = [ri(0, 150) for _ in range(ri(1, 7))] if i % 3 else None
    inp = R.make_scan(ri(1, 3), ri(1, 200), G * ri(1, 40), ri(1, 40), G, dtype, gate=bool(ri(0, 1)),
                      init=bool(ri(0, 1)), lens=lens, seed=i)
    check(gdn, inp, dtype, lens)


def test_scan_slices_of_wider_rows(gdn):
    """x, z, delta, B and C as column slices at an odd offset of one projection's rows."""
    B, T, D, S, G = 2, 37, 24, 8, 2
    inp = R.make_scan(B, T, D, S, G, "bf16", seed=7)
    wide = torch.zeros(B, T, 3 * D + 2 * G * S + 1, dtype=torch.bfloat16, device="cuda")
    views, at = {}, 1
    for k in ("x", "delta", "z", "B", "C"):
        n = D if k in ("x", "delta", "z") else G * S
        v = wide[..., at:at + n]
        at += n
        views[k] = v if n == D else v.unflatten(-1, (G, S))
        views[k].copy_(inp[k])
    y, ht = gdn.gdn_selective_scan_fwd(**(cuda(inp) | views))
    y2, ht2 = gdn.gdn_selective_scan_fwd(**cuda(inp))
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(ht, ht2)
    pool, pool2 = torch.zeros(B, D, S, device="cuda"), torch.zeros(B, D, S, device="cuda")
    rest = {k: v for k, v in cuda(inp).items() if k not in ("h0", *views)}
    ys = gdn.gdn_selective_scan_step(**rest, **views, state=pool)
    yc = gdn.gdn_selective_scan_step(**{k: v for k, v in cuda(inp).items() if k != "h0"}, state=pool2)
    assert torch.equal(ys, yc) and torch.equal(pool, pool2)


def test_scan_steep_and_flat_decays(gdn):
    """Steps and rates from nothing to states that vanish within a token; e^{dt A} underflows to zero."""
    inp = R.make_scan(1, 60, 32, 16, 1, "f32", seed=8)
    inp["A"] = -torch.logspace(-4, 4, 16).repeat(32, 1).contiguous()
    inp["dt_bias"] = torch.linspace(-30, 30, 32)
    check(gdn, inp, "f32")


def test_scan_on_another_stream_and_twice(gdn):
    inp = cuda(R.make_scan(2, 300, 64, 16, 1, "bf16", init=True, seed=9))
    torch.cuda.synchronize()
    y, ht = gdn.gdn_selective_scan_fwd(**inp)
    s = torch.cuda.Stream()
    y2, ht2 = torch.empty_like(y), torch.empty_like(ht)
    ws = torch.empty(64 << 20, dtype=torch.uint8, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    gdn.gdn_selective_scan_fwd(**inp, y=y2, ht=ht2, workspace=ws, stream=s.cuda_stream)
    s.synchronize()
    y3, _ = gdn.gdn_selective_scan_fwd(**inp, stream=s.cuda_stream)   # its own workspace, on that stream
    s.synchronize()
    assert torch.equal(y, y3)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(ht, ht2)


def test_scan_all_sequences_empty(gdn):
    inp = R.make_scan(1, 0, 20, 8, 1, "bf16", init=True, lens=[0, 0, 0], seed=15)
    d = cuda(inp)
    y, ht = gdn.gdn_selective_scan_fwd(**d, cu_seqlens=offsets([0, 0, 0]))
    assert y.shape == (1, 0, 20) and torch.equal(ht, d["h0"])
    dht = torch.randn_like(ht)
    g = gdn.gdn_selective_scan_bwd(**d, dout=torch.empty_like(d["x"]), dht=dht, cu_seqlens=offsets([0, 0, 0]))
    torch.cuda.synchronize()
    assert torch.equal(g["dh0"], dht) and torch.all(g["dA"] == 0) and torch.all(g["dD"] == 0)
    state = d.pop("h0").clone()
    before = state.clone()
    gdn.gdn_selective_scan_step(**d, state=state, cu_seqlens=offsets([0, 0, 0]))
    assert torch.equal(state, before)


def test_scan_offsets_past_32_bits(gdn):
    """More than 2^31 elements in x; states fade within a few tokens, so the last ones stand for themselves."""
    T, D, S = 66000, 33000, 4
    g = torch.Generator(device="cuda").manual_seed(10)
    big = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.bfloat16)
    x, delta, B, C = big(1, T, D), big(1, T, D), big(1, T, 1, S), big(1, T, 1, S)
    A = torch.full((D, S), -8.0, device="cuda")
    bias = torch.full((D,), 2.0, device="cuda")
    y, ht = gdn.gdn_selective_scan_fwd(x, delta, A, B, C, dt_bias=bias)
    torch.cuda.synchronize()
    for sl in (slice(0, 5), slice(D - 5, D)):
        cut = lambda t: t[:, -80:, sl].cpu()
        y_ref, ht_ref = R.scan(cut(x), cut(delta), A[sl].cpu(), B[:, -80:].cpu(), C[:, -80:].cpu(),
                               dt_bias=bias[sl].cpu())
        assert rel_fro(y[:, -40:, sl].double().cpu(), y_ref[:, -40:]) <= TOL["bf16"]
        assert rel_fro(ht[:, sl].cpu(), ht_ref) <= F32


def test_scan_malformed_cu_seqlens(gdn):
    inp = cuda(R.make_scan(1, 30, 16, 4, 1, "f32", seed=11))
    for bad in ([0, 20, 10, 30], [1, 10, 20, 30], [0, 10, 20, 29], [0, 10, 40, 30]):
        cu = torch.tensor(bad, dtype=torch.int32, device="cuda")
        y, ht = torch.full_like(inp["x"], 7.0), torch.full((3, 16, 4), 7.0, device="cuda")
        p = gdn._scan_problem(inp["x"], inp["delta"], inp["A"], inp["B"], inp["C"], None, None, None, True, cu, ())
        ws = torch.empty(gdn.gdn_selective_scan_fwd_workspace_size(p), dtype=torch.uint8, device="cuda")
        gdn.gdn_selective_scan_fwd(inp["x"], inp["delta"], inp["A"], inp["B"], inp["C"], cu_seqlens=cu, y=y, ht=ht,
                                   workspace=ws)
        assert gdn.gdn_selective_scan_get_device_status(p, ws) == gdn.DEV_BAD_CU_SEQLENS
        assert gdn.gdn_selective_scan_get_device_status(p, ws) == gdn.DEV_OK
        assert torch.all(y == 7.0) and torch.all(ht == 7.0)


# ------------------------------------------------------------- single tokens

@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("D,S,G", [(1, 1, 1), (130, 16, 2), (65, 7, 5), (40, 24, 1), (300, 4, 1), (24, 64, 2)])
def test_step_state_pool(gdn, dtype, D, S, G):
    n = 5
    inp = R.make_scan(n, 1, D, S, G, dtype, seed=D)
    del inp["h0"]
    pool = torch.randn(9, D, S, generator=torch.Generator().manual_seed(1))
    slots = [3, 0, -1, 8, 9]   # two sequences without a slot
    state = pool.cuda()
    y = gdn.gdn_selective_scan_step(**cuda(inp), state=state,
                                    state_indices=torch.tensor(slots, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    want = pool.double().clone()
    h0 = torch.stack([pool[s] if 0 <= s < 9 else torch.zeros(D, S) for s in slots])
    y_ref, ht_ref = R.scan(**inp, h0=h0)
    for i, s in enumerate(slots):
        if 0 <= s < 9:
            want[s] = ht_ref[i]
        else:
            y_ref[i] = 0
            assert torch.all(y[i] == 0)
    assert rel_fro(y.double().cpu(), y_ref) <= TOL[dtype]
    assert rel_fro(state.cpu(), want) <= F32
    untouched = [i for i in range(9) if i not in slots]
    assert torch.equal(state.cpu()[untouched], pool[untouched])


@pytest.mark.parametrize("dtype,D,S", [("bf16", 70, 16), ("f32", 33, 5), ("bf16", 40, 32), ("f32", 20, 64), ("bf16", 9, 3)])
def test_step_many_sequences(gdn, dtype, D, S):
    """Enough sequences that threads take several, their number not a multiple of that."""
    n = 101
    inp = R.make_scan(n, 1, D, S, 1, dtype, seed=D)
    del inp["h0"]
    pool = torch.randn(n + 20, D, S, generator=torch.Generator().manual_seed(2))
    slots = torch.randperm(n + 20, generator=torch.Generator().manual_seed(3))[:n]
    slots[[0, 7, 50, 100]] = torch.tensor([-1, n + 20, -2, -5])
    state = pool.cuda()
    y = gdn.gdn_selective_scan_step(**cuda(inp), state=state, state_indices=slots.int().cuda())
    torch.cuda.synchronize()
    has = (slots >= 0) & (slots < n + 20)
    h0 = torch.zeros(n, D, S)
    h0[has] = pool[slots[has]]
    y_ref, ht_ref = R.scan(**inp, h0=h0)
    y_ref[~has] = 0
    want = pool.double().clone()
    want[slots[has]] = ht_ref[has]
    assert torch.all(y[~has.cuda()] == 0)
    assert rel_fro(y.double().cpu(), y_ref) <= TOL[dtype]
    assert rel_fro(state.cpu(), want) <= F32


def test_step_several_tokens_packed(gdn):
    lens = [3, 0, 5, 1]
    inp = R.make_scan(1, 0, 50, 16, 1, "bf16", init=True, lens=lens, seed=12)
    state = inp["h0"].cuda()
    rest = {k: v for k, v in cuda(inp).items() if k != "h0"}
    y = gdn.gdn_selective_scan_step(**rest, state=state, cu_seqlens=offsets(lens))
    y_ref, ht_ref = R.scan(**inp, lens=lens)
    assert rel_fro(y.double().cpu(), y_ref) <= TOL["bf16"]
    assert rel_fro(state.cpu(), ht_ref) <= F32
    # offsets that leave the batch or decrease: those sequences are skipped
    bad = torch.tensor([0, 3, 99, 2, 2], dtype=torch.int32, device="cuda")
    state, y = inp["h0"].cuda(), torch.full_like(rest["x"], 7.0)
    gdn.gdn_selective_scan_step(**rest, state=state, cu_seqlens=bad, y=y)
    assert torch.all(y[:, 3:] == 7.0) and not torch.any(y[:, :3] == 7.0)
    assert torch.equal(state[1:].cpu(), inp["h0"][1:])


def test_prompt_then_steps(gdn):
    """A prompt, then tokens one by one on its final states, equal one pass over all of them."""
    T, steps = 50, 4
    inp = R.make_scan(2, T + steps, 70, 16, 1, "f32", seed=13)
    full = {k: v for k, v in cuda(inp).items() if k != "h0"}
    part = lambda a, b: {k: v[:, a:b].contiguous() if k in ("x", "delta", "B", "C", "z") else v
                         for k, v in full.items()}
    y, state = gdn.gdn_selective_scan_fwd(**part(0, T))
    ys = [y] + [gdn.gdn_selective_scan_step(**part(t, t + 1), state=state) for t in range(T, T + steps)]
    y_ref, ht_ref = R.scan(**inp)
    assert rel_fro(torch.cat(ys, 1).cpu(), y_ref) <= F32
    assert rel_fro(state.cpu(), ht_ref) <= F32


def test_scan_refusals(gdn):
    inp = {k: v for k, v in cuda(R.make_scan(2, 8, 12, 4, 2, "f32", seed=14)).items() if k != "h0"}
    call = lambda **kw: gdn.gdn_selective_scan_fwd(**(inp | kw))
    for kw in (dict(A=inp["A"][:, :3]), dict(A=inp["A"].bfloat16()), dict(B=inp["B"].bfloat16()),
               dict(z=inp["z"][:, :4]), dict(x=inp["x"].cpu()), dict(dt_bias=inp["dt_bias"][:5]),
               dict(delta=inp["delta"].transpose(1, 2).contiguous().transpose(1, 2)),
               dict(h0=torch.zeros(3, 12, 4, device="cuda"))):
        with pytest.raises(ValueError):
            call(**kw)
    wide = torch.zeros(1, 4, 1, 65, device="cuda")
    with pytest.raises(gdn.GDNError):   # more than 64 states
        gdn.gdn_selective_scan_fwd(inp["x"][:1, :4].contiguous(), inp["x"][:1, :4].contiguous(),
                                   torch.zeros(12, 65, device="cuda"), wide, wide)
    with pytest.raises(gdn.GDNError):   # G does not divide D
        b5 = torch.zeros(2, 8, 5, 4, device="cuda")
        call(B=b5, C=b5)
    with pytest.raises(gdn.GDNError):   # workspace too small
        call(workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(gdn.GDNError):   # fewer slots than sequences without a slot map
        gdn.gdn_selective_scan_step(**inp, state=torch.zeros(1, 12, 4, device="cuda"))
