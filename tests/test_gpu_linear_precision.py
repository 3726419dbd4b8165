"""What decayed linear attention keeps of its inputs' bits, against 64 bits: states that are carried over many chunks by
slow decays.

Bounds.  A state multiplied and added to once a chunk (or once a token, in the step) takes a rounding each time, 2^-24
of itself at most and 2.5e-8 in the mean square over a binade; n of them add like their squares, and no more count than
the state's memory holds, 1 / (2 |g|) tokens for squares: 2.5e-8 sqrt(n), beside 2e-7 for the exponentials (2^-23), the
products of fp32 values and their sums within a chunk.  A decay that is itself off by some 1e-8 a chunk, always to one
side, would pass that: it adds up over the memory."""
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


@pytest.mark.parametrize("g", [-1e-3, -1e-5])
def test_many_steps_of_a_slow_decay(gdn, g):
    T = 20000
    x, _, h0 = slow(F32, T, g)
    pool = h0.clone()
    gdn.gdn_linear_attn_step(**x, state=pool)
    assert ref.rel(pool, final_states(x, h0)) <= carried(min(T, 0.5 / -g))
