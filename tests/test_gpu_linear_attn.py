"""Decayed linear attention on the GPU against the recurrence in 64 bits.

Tolerances, relative Frobenius errors.  fp32: sums of up to K + V + 64 fp32 products; the rounding errors of n additions
add like their squares to about sqrt(n) 2^-24 (1.3e-6 for n = 448), with the decays' exponentials (2^-22) and the sums
from chunk to chunk beside them: 4e-6.  bf16 outputs: the output's own rounding, that of the weights between tokens and
that of the state's copy, each 2^-8 of the value at most and 0.43 of that in the mean square over a binade, adding like
their squares: sqrt(3) 0.43 2^-8 = 2.9e-3 over many elements, and dq, dk are of the same form: 4e-3.  Final states and gradients that stay in fp32 keep fp32 tolerances whatever the inputs' type
(1e-5: products of terms in two bf16 parts, 2^-17 of each)."""
import pytest
import torch

import linear_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
O_TOL = {torch.float32: 4e-6, torch.bfloat16: 4e-3}
S_TOL = {torch.float32: 4e-6, torch.bfloat16: 1e-5}


@pytest.fixture(scope="module")
def gdn():
    from gated_deltanet_chunked_gdn_gb300 import binding
    binding.load()
    return binding


def make(B, T, Hqk, Hv, K, V, dtype, seed=0, lens=None, per_head=False, init=True, strong=0.0):
    torch.manual_seed(seed)
    cu = None
    N = B
    if lens is not None:
        cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEV)
        B, T, N = 1, sum(lens), len(lens)
    q = torch.randn(B, T, Hqk, K, device=DEV).to(dtype)
    k = (torch.randn(B, T, Hqk, K, device=DEV) * K ** -0.5).to(dtype)
    v, do = torch.randn(B, T, Hv, V, device=DEV).to(dtype), torch.randn(B, T, Hv, V, device=DEV).to(dtype)
    if per_head:
        g = -torch.rand(Hv, device=DEV) * 0.3
    else:
        g = -torch.rand(B, T, Hv, device=DEV) * torch.rand(Hv, device=DEV)
        if strong:
            g = torch.where(torch.rand(B, T, Hv, device=DEV) < 0.05, torch.full_like(g, -strong), g)
    h0 = 0.3 * torch.randn(N, Hv, K, V, device=DEV) if init else None
    dht = 0.3 * torch.randn(N, Hv, K, V, device=DEV) if init else None
    return dict(q=q, k=k, v=v, g=g, do=do, h0=h0, dht=dht, cu=cu)


def check_fwd(gdn, x, scale=0.25):
    o, ht = gdn.gdn_linear_attn_fwd(x["q"], x["k"], x["v"], x["g"], scale=scale, h0=x["h0"], cu_seqlens=x["cu"])
    wo, wh = ref.forward(x["q"], x["k"], x["v"], x["g"], scale, x["h0"], x["cu"])
    dt = x["v"].dtype
    assert o.dtype == dt and ref.rel(o, wo) < O_TOL[dt], ref.rel(o, wo)
    assert ref.rel(ht, wh) < S_TOL[dt], ref.rel(ht, wh)


def check_bwd(gdn, x, scale=0.25):
    got = gdn.gdn_linear_attn_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], scale=scale, h0=x["h0"], dht=x["dht"],
                                  cu_seqlens=x["cu"], want_dh0=True)
    want = ref.backward(x["q"], x["k"], x["v"], x["g"], x["do"], scale, x["h0"], x["dht"], x["cu"])
    dt = x["v"].dtype
    for n in ("dq", "dk", "dv", "dg", "dh0"):
        e = ref.rel(got[n], want[n])
        assert e < (O_TOL if n in ("dq", "dk", "dv") else S_TOL)[dt], (n, e)


BF, F32 = torch.bfloat16, torch.float32
DIMS = [(1, 1, 64, 64), (1, 2, 128, 128), (2, 2, 64, 128), (1, 3, 128, 64), (1, 1, 256, 64), (1, 1, 128, 256),
        (1, 2, 256, 256), (1, 1, 64, 256), (1, 1, 256, 128)]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("Hqk,Hv,K,V", DIMS)
def test_head_dims(gdn, Hqk, Hv, K, V, dtype):
    x = make(2, 147, Hqk, Hv, K, V, dtype)
    check_fwd(gdn, x)
    check_bwd(gdn, x)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("T", [1, 2, 63, 64, 65, 127, 128, 129, 700])
def test_lengths(gdn, T, dtype):
    x = make(3, T, 1, 2, 128, 128, dtype, seed=T, init=T % 2 == 0, per_head=T % 3 == 0)
    check_fwd(gdn, x)
    check_bwd(gdn, x)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lens", [[1], [5, 0, 64, 1, 130, 0], [0, 0, 3], [200, 1, 1, 1, 63, 64, 65], [1] * 40, [300, 17]])
def test_packed(gdn, lens, dtype):
    for per_head in (False, True):
        x = make(1, 0, 2, 4, 64, 128, dtype, lens=lens, per_head=per_head)
        check_fwd(gdn, x)
        check_bwd(gdn, x)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_many_sequences(gdn, dtype):
    """More sequences than one tile of the tables' running sum."""
    x = make(1, 0, 1, 1, 64, 64, dtype, lens=[i % 3 for i in range(2100)])
    check_fwd(gdn, x)
    check_bwd(gdn, x)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("strong", [50.0, 800.0, float("inf")])
def test_strong_decays(gdn, strong, dtype):
    """Tokens that start the state anew; behind them the sums of the decays keep their precision."""
    x = make(2, 300, 1, 2, 128, 128, dtype, strong=strong)
    check_fwd(gdn, x)
    got = gdn.gdn_linear_attn_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], scale=0.25, h0=x["h0"], dht=x["dht"])
    want = ref.backward(x["q"], x["k"], x["v"], x["g"].clamp(min=-1e4), x["do"], 0.25, x["h0"], x["dht"])
    for n in ("dq", "dk", "dv", "dg", "dh0"):
        assert ref.rel(got[n], want[n]) < (O_TOL if n in ("dq", "dk", "dv") else S_TOL)[dtype], n


@pytest.mark.parametrize("dtype", [F32, BF])
def test_no_decay_and_growth(gdn, dtype):
    x = make(1, 260, 1, 1, 64, 64, dtype)
    x["g"] = torch.zeros_like(x["g"])
    check_fwd(gdn, x)
    check_bwd(gdn, x)
    x["g"] = torch.full_like(x["g"], 0.02)
    check_fwd(gdn, x)
    check_bwd(gdn, x)


@pytest.mark.parametrize("dtype", [F32, BF])
def test_slices_of_wider_rows(gdn, dtype):
    B, T, Hqk, Hv, K, V = 2, 150, 2, 4, 64, 128
    x = make(B, T, Hqk, Hv, K, V, dtype)
    wide = torch.full((B, T, 2 * Hqk * K + Hv * V + 8), float("nan"), device=DEV).to(dtype)
    views = {}
    for name, at, n, H in (("q", 0, Hqk * K, Hqk), ("k", Hqk * K, Hqk * K, Hqk), ("v", 2 * Hqk * K, Hv * V, Hv)):
        views[name] = wide[..., at:at + n].unflatten(-1, (H, -1))
        views[name].copy_(x[name])
    y = {**x, **views}
    args = lambda d: (d["q"], d["k"], d["v"], d["g"])  # noqa: E731
    a, b = gdn.gdn_linear_attn_fwd(*args(x), h0=x["h0"]), gdn.gdn_linear_attn_fwd(*args(y), h0=x["h0"])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a = gdn.gdn_linear_attn_bwd(*args(x), x["do"], h0=x["h0"], dht=x["dht"])
    b = gdn.gdn_linear_attn_bwd(*args(y), x["do"], h0=x["h0"], dht=x["dht"])
    for n in ("dq", "dk", "dv", "dg", "dh0"):
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("dtype", [F32, BF])
def test_values_beside_a_sequence_do_not_matter(gdn, dtype):
    """NaN and infinities in the tokens next to a sequence's ragged end stay out of it."""
    lens = [70, 61, 130]
    x = make(1, 0, 1, 2, 128, 128, dtype, lens=lens)
    bad = {n: x[n].clone() for n in ("q", "k", "v", "do")}
    for n in bad:
        bad[n][:, 70:131] = float("nan") if n != "v" else float("inf")
    y = {**x, **bad}
    a = gdn.gdn_linear_attn_fwd(x["q"], x["k"], x["v"], x["g"], h0=x["h0"], cu_seqlens=x["cu"])
    b = gdn.gdn_linear_attn_fwd(y["q"], y["k"], y["v"], y["g"], h0=x["h0"], cu_seqlens=x["cu"])
    ga = gdn.gdn_linear_attn_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], h0=x["h0"], dht=x["dht"], cu_seqlens=x["cu"])
    gb = gdn.gdn_linear_attn_bwd(y["q"], y["k"], y["v"], y["g"], y["do"], h0=x["h0"], dht=x["dht"], cu_seqlens=x["cu"])
    for s in (slice(0, 70), slice(131, 261)):
        assert torch.equal(a[0][:, s], b[0][:, s])
        for n in ("dq", "dk", "dv", "dg"):
            assert torch.equal(ga[n][:, s], gb[n][:, s]), n
    for n in (0, 2):
        assert torch.equal(a[1][n], b[1][n]) and torch.equal(ga["dh0"][n], gb["dh0"][n])


@pytest.mark.parametrize("dtype", [F32, BF])
def test_pool_rows_and_states_in_place(gdn, dtype):
    x = make(3, 90, 1, 2, 64, 64, dtype)
    o, ht = gdn.gdn_linear_attn_fwd(x["q"], x["k"], x["v"], x["g"], h0=x["h0"])
    pool = torch.full((5, 2, 64, 64), 7.0, device=DEV)
    rows = torch.tensor([4, -1, 1], dtype=torch.int32, device=DEV)
    o2, _ = gdn.gdn_linear_attn_fwd(x["q"], x["k"], x["v"], x["g"], h0=x["h0"], ht=pool, state_indices=rows)
    assert torch.equal(o, o2) and torch.equal(pool[4], ht[0]) and torch.equal(pool[1], ht[2])
    assert bool((pool[[0, 2, 3]] == 7.0).all())
    h = x["h0"].clone()
    gdn.gdn_linear_attn_fwd(x["q"], x["k"], x["v"], x["g"], h0=h, ht=h)
    assert torch.equal(h, ht)
    assert gdn.gdn_linear_attn_fwd(x["q"], x["k"], x["v"], x["g"], output_final_state=False)[1] is None


@pytest.mark.parametrize("dtype", [F32, BF])
def test_long_sequences_states_in_place(gdn, dtype):
    """Sequences cut into segments: the final state may take the initial one's place, dh0 that of dht."""
    x = make(2, 3000, 1, 2, 128, 128, dtype, strong=0)
    args = (x["q"], x["k"], x["v"], x["g"])
    o, ht = gdn.gdn_linear_attn_fwd(*args, h0=x["h0"])
    g = gdn.gdn_linear_attn_bwd(*args, x["do"], h0=x["h0"], dht=x["dht"])
    for _ in range(5):
        h = x["h0"].clone()
        o2, _ = gdn.gdn_linear_attn_fwd(*args, h0=h, ht=h)
        assert torch.equal(o, o2) and torch.equal(h, ht)
    check_fwd(gdn, x)
    check_bwd(gdn, x)
    assert torch.equal(g["dh0"], gdn.gdn_linear_attn_bwd(*args, x["do"], h0=x["h0"], dht=x["dht"])["dh0"])


def test_malformed_offsets_write_nothing(gdn):
    for bad in ([0, 50, 40, 100], [1, 50, 60, 100], [0, 50, 60, 99], [0, -3, 60, 100], [0, 200, 60, 100]):
        for dtype in (F32, BF):
            x = make(1, 0, 1, 1, 128, 128, dtype, lens=[40, 30, 30])
            cu = torch.tensor(bad, dtype=torch.int32, device=DEV)
            o, ht = torch.full_like(x["v"], 3.0), torch.full((3, 1, 128, 128), 3.0, device=DEV)
            p = gdn._linear_problem(x["q"], x["k"], x["v"], x["g"], cu)
            ws = torch.zeros(gdn.gdn_linear_attn_fwd_workspace_size(p), dtype=torch.uint8, device=DEV)
            gdn.gdn_linear_attn_fwd(x["q"], x["k"], x["v"], x["g"], cu_seqlens=cu, o=o, ht=ht, workspace=ws)
            assert gdn.gdn_linear_attn_get_device_status(ws) == gdn.DEV_BAD_CU_SEQLENS
            assert gdn.gdn_linear_attn_get_device_status(ws) == gdn.DEV_OK
            assert bool((o == 3.0).all()) and bool((ht == 3.0).all())
            ws = torch.zeros(gdn.gdn_linear_attn_bwd_workspace_size(p), dtype=torch.uint8, device=DEV)
            gdn.gdn_linear_attn_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], h0=x["h0"], cu_seqlens=cu, workspace=ws)
            assert gdn.gdn_linear_attn_get_device_status(ws) == gdn.DEV_BAD_CU_SEQLENS


# ------------------------------------------------------------------- decode

@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("N,Hqk,Hv,K,V", [(1, 1, 1, 64, 64), (3, 2, 4, 128, 128), (70, 4, 8, 64, 128),
                                          (2, 1, 3, 256, 256), (5, 2, 2, 128, 64), (40, 1, 8, 256, 64)])
def test_step(gdn, N, Hqk, Hv, K, V, dtype):
    for T in (1, 3):
        x = make(N, T, Hqk, Hv, K, V, dtype, seed=N)
        pool = torch.randn(N + 3, Hv, K, V, device=DEV)
        before = pool.clone()
        slots = torch.randperm(N + 3, device=DEV)[:N].to(torch.int32)
        if N > 2:
            slots[1] = N + 3
        o = gdn.gdn_linear_attn_step(x["q"], x["k"], x["v"], x["g"], pool, scale=0.25, state_indices=slots)
        live = slots < N + 3
        at = slots[live].long()
        wo, wh = ref.forward(x["q"][live], x["k"][live], x["v"][live], x["g"][live], 0.25, before[at])
        # one rounding of o; the state's update is one fp32 operation after another on fp32 inputs
        assert ref.rel(o[live], wo) < (2 ** -8 if dtype is BF else 2e-6)
        assert ref.rel(pool[at], wh) < 1e-6
        rest = torch.ones(N + 3, dtype=torch.bool, device=DEV)
        rest[at] = False
        assert torch.equal(pool[rest], before[rest])
        assert bool((o[~live] == 0).all())


def test_step_packed_and_per_head(gdn):
    lens = [1, 3, 0, 2]
    x = make(1, 0, 1, 2, 128, 128, F32, lens=lens, per_head=True)
    pool = x["h0"].clone()
    o = gdn.gdn_linear_attn_step(x["q"], x["k"], x["v"], x["g"], pool, scale=0.25, cu_seqlens=x["cu"])
    wo, wh = ref.forward(x["q"], x["k"], x["v"], x["g"], 0.25, x["h0"], x["cu"])
    assert ref.rel(o, wo) < 2e-6 and ref.rel(pool, wh) < 1e-6


def test_step_more_heads_than_one_launch_takes(gdn):
    N, H = 1100, 64
    x = make(N, 1, 1, H, 64, 64, BF)
    pool = x["h0"].clone()
    o = gdn.gdn_linear_attn_step(x["q"], x["k"], x["v"], x["g"], pool, scale=0.25)
    wo, wh = ref.forward(x["q"][-80:], x["k"][-80:], x["v"][-80:], x["g"][-80:], 0.25, x["h0"][-80:])
    assert ref.rel(o[-80:], wo) < 2 ** -8 and ref.rel(pool[-80:], wh) < 1e-6


def test_prompt_then_steps_continue_it(gdn):
    x = make(2, 140, 1, 2, 128, 128, F32, init=False)
    cut = lambda a, b: [x[n][:, a:b].contiguous() for n in ("q", "k", "v", "g")]  # noqa: E731
    o, ht = gdn.gdn_linear_attn_fwd(*cut(0, 140))
    pool = torch.zeros(2, 2, 128, 128, device=DEV)
    slots = torch.tensor([1, 0], dtype=torch.int32, device=DEV)
    gdn.gdn_linear_attn_fwd(*cut(0, 137), ht=pool, state_indices=slots)
    for t in range(137, 140):
        s = gdn.gdn_linear_attn_step(*cut(t, t + 1), pool, state_indices=slots)
        assert ref.rel(s, o[:, t:t + 1]) < 8e-6   # two ways to the same sums
    assert ref.rel(pool[[1, 0]], ht) < 8e-6


# ------------------------------------------------------- runs and their streams

@pytest.mark.parametrize("dtype", [F32, BF])
def test_the_same_bits_every_run_and_on_other_streams(gdn, dtype):
    x = make(1, 0, 2, 4, 128, 128, dtype, lens=[700, 3, 260])
    args = (x["q"], x["k"], x["v"], x["g"])
    first = gdn.gdn_linear_attn_fwd(*args, h0=x["h0"], cu_seqlens=x["cu"])
    grads = gdn.gdn_linear_attn_bwd(*args, x["do"], h0=x["h0"], dht=x["dht"], cu_seqlens=x["cu"])
    side = torch.cuda.Stream()
    for _ in range(3):
        o, ht = gdn.gdn_linear_attn_fwd(*args, h0=x["h0"], cu_seqlens=x["cu"], stream=side.cuda_stream)
        g = gdn.gdn_linear_attn_bwd(*args, x["do"], h0=x["h0"], dht=x["dht"], cu_seqlens=x["cu"],
                                    stream=side.cuda_stream)
        side.synchronize()
        assert torch.equal(o, first[0]) and torch.equal(ht, first[1])
        for n in ("dq", "dk", "dv", "dg", "dh0"):
            assert torch.equal(g[n], grads[n]), n


@pytest.mark.parametrize("dtype", [F32, BF])
def test_captured_and_replayed(gdn, dtype):
    x = make(2, 200, 1, 2, 128, 128, dtype)
    args = (x["q"], x["k"], x["v"], x["g"])
    pool = x["h0"].clone()
    step = [t[:, :1].contiguous() for t in args]
    gdn.gdn_linear_attn_fwd(*args)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, ht = gdn.gdn_linear_attn_fwd(*args, h0=x["h0"])
        g = gdn.gdn_linear_attn_bwd(*args, x["do"], h0=x["h0"], dht=x["dht"])
        s = gdn.gdn_linear_attn_step(*step, pool)
    y = make(2, 200, 1, 2, 128, 128, dtype, seed=9)
    for n in ("q", "k", "v", "g", "h0", "do", "dht"):
        x[n].copy_(y[n])
    for a, n in zip(step, ("q", "k", "v", "g")):
        a.copy_(y[n][:, :1])
    pool.copy_(y["h0"])
    graph.replay()
    wo, wh = gdn.gdn_linear_attn_fwd(y["q"], y["k"], y["v"], y["g"], h0=y["h0"])
    wg = gdn.gdn_linear_attn_bwd(y["q"], y["k"], y["v"], y["g"], y["do"], h0=y["h0"], dht=y["dht"])
    p2 = y["h0"].clone()
    ws = gdn.gdn_linear_attn_step(*[y[n][:, :1].contiguous() for n in ("q", "k", "v", "g")], p2)
    assert torch.equal(o, wo) and torch.equal(ht, wh) and torch.equal(s, ws) and torch.equal(pool, p2)
    for n in ("dq", "dk", "dv", "dg", "dh0"):
        assert torch.equal(g[n], wg[n]), n


@pytest.mark.parametrize("dtype,V", [(BF, 128), (BF, 256), (F32, 128)])
@pytest.mark.parametrize("per_head", [False, True])
def test_no_tokens_at_all(gdn, per_head, dtype, V):
    """Packed batches whose sequences are all empty: states pass through, the decays' gradients are zero."""
    x = make(1, 0, 2, 4, 64, V, dtype, lens=[0, 0, 0], per_head=per_head)
    o, ht = gdn.gdn_linear_attn_fwd(x["q"], x["k"], x["v"], x["g"], h0=x["h0"], cu_seqlens=x["cu"])
    assert o.shape == x["v"].shape and torch.equal(ht, x["h0"])
    got = gdn.gdn_linear_attn_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], h0=x["h0"], dht=x["dht"],
                                  cu_seqlens=x["cu"])
    assert torch.equal(got["dh0"], x["dht"]) and got["dg"].shape == x["g"].shape and not got["dg"].any()


@pytest.mark.parametrize("K,V", [(64, 64), (64, 256), (128, 64), (256, 128), (256, 256)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_wide_heads_and_ragged_chunks(gdn, dtype, K, V):
    """Every head dim in packed batches whose chunks end inside a tile, decays that are strong now and then."""
    x = make(1, 0, 2, 6, K, V, dtype, lens=[1, 63, 0, 65, 200, 17], seed=K + V, strong=30.0)
    check_fwd(gdn, x)
    check_bwd(gdn, x)


@pytest.mark.parametrize("dtype,K,V", [(F32, 64, 128), (F32, 256, 64), (BF, 256, 128)])
def test_large_values_keep_their_neighbours_bits(gdn, dtype, K, V):
    """Channels of very different sizes: every term of a value has to arrive, the small ones under large ones too."""
    x = make(1, 260, 1, 2, K, V, dtype, seed=3)
    x["q"] = x["q"] * torch.logspace(-4, 4, K, device=DEV).to(dtype)
    x["k"] = x["k"] * torch.logspace(4, -4, K, device=DEV).to(dtype)
    x["v"] = x["v"] * torch.logspace(-5, 5, V, device=DEV).to(dtype)
    x["h0"] = None   # (a state beside products of these sizes would only add to them)
    o, ht = gdn.gdn_linear_attn_fwd(x["q"], x["k"], x["v"], x["g"], scale=1.0)
    wo, wh = ref.forward(x["q"], x["k"], x["v"], x["g"], 1.0, None, None)
    for e in range(0, V, 16):   # each band of columns against its own norm
        assert ref.rel(o[..., e:e + 16], wo[..., e:e + 16]) < O_TOL[dtype]
        assert ref.rel(ht[..., e:e + 16], wh[..., e:e + 16]) < S_TOL[dtype]


@pytest.mark.parametrize("K,V", [(128, 128), (64, 256)])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_dh0_in_the_place_of_h0_or_dht(gdn, dtype, K, V):
    """The C call's promise: dh0 may be h0 or dht, the same pointer; every output as with a buffer of its own."""
    x = make(2, 2100, 1, 2, K, V, dtype)
    want = gdn.gdn_linear_attn_bwd(x["q"], x["k"], x["v"], x["g"], x["do"], scale=0.25, h0=x["h0"], dht=x["dht"])
    p = gdn._linear_problem(x["q"], x["k"], x["v"], x["g"], None)
    ws = torch.zeros(gdn.gdn_linear_attn_bwd_workspace_size(p), dtype=torch.uint8, device=DEV)
    for place in ("h0", "dht"):
        h0, dht = x["h0"].clone(), x["dht"].clone()
        dh0 = h0 if place == "h0" else dht
        out = [torch.empty_like(want[n]) for n in ("dq", "dk", "dv", "dg")] + [dh0]
        st = gdn._call(0, gdn.load().gdn_linear_attn_bwd, p, *(x[n].data_ptr() for n in ("q", "k", "v", "g")), 0.25,
                       h0.data_ptr(), 0, x["do"].data_ptr(), dht.data_ptr(), *(t.data_ptr() for t in out),
                       ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
        assert st == 0
        for n, t in zip(("dq", "dk", "dv", "dg", "dh0"), out):
            assert torch.equal(t, want[n]), (place, n)


@pytest.mark.parametrize("dtype,K,V", [(F32, 64, 128), (F32, 256, 256), (BF, 256, 128)])
def test_two_calls_at_once_and_a_captured_one(gdn, dtype, K, V):
    """Calls on two streams share the device's tensor memory; a captured call replays to the same bits."""
    x = make(2, 700, 2, 4, K, V, dtype)
    y = make(1, 0, 2, 4, K, V, dtype, lens=[300, 5, 900], seed=1)

    def run(z):
        o, ht = gdn.gdn_linear_attn_fwd(z["q"], z["k"], z["v"], z["g"], h0=z["h0"], cu_seqlens=z["cu"])
        d = gdn.gdn_linear_attn_bwd(z["q"], z["k"], z["v"], z["g"], z["do"], h0=z["h0"], dht=z["dht"],
                                    cu_seqlens=z["cu"])
        return [o, ht] + [d[n] for n in ("dq", "dk", "dv", "dg", "dh0")]

    want = run(x), run(y)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = [None, None]
    for _ in range(3):
        for i, (s, z) in enumerate(zip(streams, (x, y))):
            with torch.cuda.stream(s):
                got[i] = run(z)
    torch.cuda.synchronize()
    for w, t in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, t))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = run(y)
    for _ in range(2):
        for t in held:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want[1], held))
