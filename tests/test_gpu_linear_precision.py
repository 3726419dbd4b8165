"""What decayed linear attention keeps of its inputs' bits, against 64 bits: states that are carried over many chunks by
slow decays, outputs that are rounded once.

Bounds.  A state multiplied and added to once a chunk (or once a token, in the step) takes a rounding each time, 2^-24
of itself at most and 2.5e-8 in the mean square over a binade; n of them add like their squares, and no more count than
the state's memory holds, 1 / (2 |g|) tokens for squares: 2.5e-8 sqrt(n), beside 2e-7 for the exponentials (2^-23), the
products of fp32 values and their sums within a chunk.  A decay that is itself off by some 1e-8 a chunk, always to one
side, adds up over the memory and goes past it.  bf16 outputs are rounded once: their error is compared with that
of rounding the 64-bit value.  Another operand kept in one bf16 term is off by as much again (sqrt(2) of it together); the
exponentials' 2^-22 and operands in two terms (2^-17) are not seen beside it: 1.05."""
import math

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


def carried(n):
    """The bound above for n roundings, one after the other."""
    return 2e-7 + 2.5e-8 * math.sqrt(n)


def once(got, want):
    """A bf16 output against its own rounding."""
    own = ref.rel(want.to(BF), want)
    assert ref.rel(got, want) <= 1.05 * own, (ref.rel(got, want), own)


def slow(dtype, T, g, Hv=2, K=64, V=64, per_head=False, seed=0):
    torch.manual_seed(seed)
    x = dict(q=torch.randn(1, T, 1, K, device=DEV).to(dtype),
             k=(torch.randn(1, T, 1, K, device=DEV) * K ** -0.5).to(dtype),
             v=torch.randn(1, T, Hv, V, device=DEV).to(dtype),
             g=torch.full((Hv,) if per_head else (1, T, Hv), g, device=DEV))
    return x, torch.randn(1, T, Hv, V, device=DEV).to(dtype), torch.randn(1, Hv, K, V, device=DEV)


def final_states(x, h0):
    """The sum over the tokens that the recurrence is, every decay an exponential of its own."""
    T, Hv = x["v"].shape[1:3]
    g = x["g"].double().expand(T, Hv) if x["g"].dim() == 1 else x["g"][0].double()
    b = g.cumsum(0)
    w = torch.exp(b[-1] - b)
    k, v = x["k"][0, :, 0].double(), x["v"][0].double()
    return torch.stack([(k * w[:, h:h + 1]).t() @ v[:, h] + torch.exp(b[-1, h]) * h0[0, h].double()
                        for h in range(Hv)])[None]


def first_adjoints(x, do, dht, scale):
    T, Hv = x["v"].shape[1:3]
    g = x["g"].double().expand(T, Hv) if x["g"].dim() == 1 else x["g"][0].double()
    b = g.cumsum(0)
    q, d = x["q"][0, :, 0].double(), do[0].double()
    return torch.stack([scale * (q * torch.exp(b[:, h:h + 1])).t() @ d[:, h] + torch.exp(b[-1, h]) * dht[0, h].double()
                        for h in range(Hv)])[None]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("g", [-1e-3, -1e-4, -1e-5])
def test_slow_decays_over_many_chunks(gdn, g, per_head, dtype):
    T = 100000
    x, do, h0 = slow(dtype, T, g, per_head=per_head)
    bound = carried(min(T, 0.5 / -g) / 64)
    _, ht = gdn.gdn_linear_attn_fwd(**x, h0=h0)
    assert ref.rel(ht, final_states(x, h0)) <= bound
    d = gdn.gdn_linear_attn_bwd(**x, dout=do, scale=0.25, h0=h0, dht=h0)
    assert ref.rel(d["dh0"], first_adjoints(x, do, h0, 0.25)) <= bound


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("g", [-1e-3, -1e-5, 0.0])
def test_gradients_of_slow_decays(gdn, g, dtype):
    """dg is a sum over pairs of tokens of fp32 products, each token's with a state at its end: 1e-6 beside what the
    states carry."""
    x, do, h0 = slow(dtype, 4096, g, Hv=1, K=128, V=128)
    d = gdn.gdn_linear_attn_bwd(**x, dout=do, scale=0.25, h0=h0, dht=h0)
    want = ref.backward(x["q"], x["k"], x["v"], x["g"], do, 0.25, h0, h0)
    for n in ("dg", "dh0"):
        assert ref.rel(d[n], want[n]) <= 1e-6 + carried(64), n
    if dtype is BF:
        for n in ("dq", "dk", "dv"):
            once(d[n], want[n])


@pytest.mark.parametrize("g", [-1e-3, -1e-5])
def test_many_steps_of_a_slow_decay(gdn, g):
    T = 20000
    x, _, h0 = slow(F32, T, g)
    pool = h0.clone()
    gdn.gdn_linear_attn_step(**x, state=pool)
    assert ref.rel(pool, final_states(x, h0)) <= carried(min(T, 0.5 / -g))


DIMS = [(K, V) for K in (64, 128, 256) for V in (64, 128, 256)]


@pytest.mark.parametrize("K,V", DIMS)
@pytest.mark.parametrize("g", [0.0, -2.0 ** -8, -0.3])
def test_outputs_are_rounded_once(gdn, g, K, V):
    """Where the state makes up o (slow decays, an initial state) as where the chunk does."""
    x, _, h0 = slow(BF, 333, g, K=K, V=V, seed=K + V)
    for a, init in ((333, h0), (333, None), (5, 4 * h0), (1, h0)):
        y = {n: t[:, :a].contiguous() for n, t in x.items()}
        o, ht = gdn.gdn_linear_attn_fwd(**y, scale=0.25, h0=init)
        want, wh = ref.forward(y["q"], y["k"], y["v"], y["g"], 0.25, init)
        once(o, want)
        assert ref.rel(ht, wh) <= carried(6)


@pytest.mark.parametrize("K,V", DIMS)
@pytest.mark.parametrize("Hqk", [1, 2])
@pytest.mark.parametrize("g", [0.0, -2.0 ** -8, -0.3])
def test_gradients_are_rounded_once(gdn, g, Hqk, K, V):
    x, do, h0 = slow(BF, 333, g, K=K, V=V, seed=K + V)
    if Hqk == 2:   # heads of their own write dq and dk themselves
        x["q"], x["k"] = (torch.cat((x[n], x[n].flip(1)), 2) for n in ("q", "k"))
    for a, init in ((333, h0), (333, None), (70, h0)):
        y = {n: t[:, :a].contiguous() for n, t in x.items()}
        d = gdn.gdn_linear_attn_bwd(**y, dout=do[:, :a].contiguous(), scale=0.25, h0=init, dht=init, want_dh0=True)
        want = ref.backward(y["q"], y["k"], y["v"], y["g"], do[:, :a], 0.25, init, init)
        for n in ("dq", "dk", "dv"):
            once(d[n], want[n])
        # fp32 whatever the inputs' type
        assert ref.rel(d["dh0"], want["dh0"]) <= carried(6)
        assert ref.rel(d["dg"], want["dg"]) <= 1e-6


def test_the_same_bits_with_the_device_full(gdn):
    """More CTAs than run at once, several of them an SM."""
    for K, V in ((128, 128), (64, 128), (128, 64), (64, 64)):
        torch.manual_seed(K)
        q, k = (torch.randn(2, 2048, 16, K, device=DEV).to(BF) for _ in range(2))
        v, g = torch.randn(2, 2048, 16, V, device=DEV).to(BF), -0.02 * torch.rand(2, 2048, 16, device=DEV)
        runs = [gdn.gdn_linear_attn_fwd(q, k, v, g) for _ in range(8)]
        assert all(torch.equal(a, b) for r in runs[1:] for a, b in zip(runs[0], r))
        # the last head alone: other segments, sums in another order
        o, _ = gdn.gdn_linear_attn_fwd(*(t[:, :, -1:].contiguous() for t in (q, k, v, g)))
        assert ref.rel(o, runs[0][0][:, :, -1:]) < 5e-4


@pytest.mark.parametrize("lens", [[3, 0, 64, 100, 1], [700, 5]])
def test_packed_outputs_are_rounded_once(gdn, lens):
    T = sum(lens)
    x, do, _ = slow(BF, T, -2.0 ** -8, K=128, V=128)
    cu = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32, device=DEV)
    h0 = torch.randn(len(lens), 2, 128, 128, device=DEV)
    o, ht = gdn.gdn_linear_attn_fwd(**x, scale=0.25, h0=h0, cu_seqlens=cu)
    want, wh = ref.forward(x["q"], x["k"], x["v"], x["g"], 0.25, h0, cu)
    once(o, want)
    assert ref.rel(ht, wh) <= carried(11)
    d = gdn.gdn_linear_attn_bwd(**x, dout=do, scale=0.25, h0=h0, dht=h0, cu_seqlens=cu)
    want = ref.backward(x["q"], x["k"], x["v"], x["g"], do, 0.25, h0, h0, cu)
    for n in ("dq", "dk", "dv"):
        once(d[n], want[n])
