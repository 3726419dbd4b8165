"""Calls of the delta rule's and the convolution's entry points on another stream than
the current one: the blocks that a call allocates itself are not written before work
queued earlier on the current stream is done with their memory, and not given out
again before the other stream is done with them."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gdn():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from gated_deltanet_chunked_gdn_gb300 import binding
    binding.load()
    return binding


@pytest.fixture(scope="module")
def busy():
    """Some tens of milliseconds of work on the current stream, in buffers of its own."""
    a, c = (torch.zeros(8192, 8192, dtype=torch.bfloat16, device="cuda") for _ in range(2))

    def run():
        for _ in range(60):
            torch.mm(a, a, out=c)
    run()
    torch.cuda.synchronize()
    return run


def entry(gdn, name):
    """call(stream) -> a dict of every tensor that the call has allocated and returns."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    if name == "conv_fwd":
        x, w = rn(2, 1024, 1024).bfloat16(), rn(1024, 4)
        return lambda s: {"y": gdn.gdn_causal_conv1d_fwd(x, w, stream=s)}
    B, T, H, K = (2, 512, 16, 128) if name != "recurrent" else (2048, 1, 8, 64)
    q, k = (torch.nn.functional.normalize(rn(B, T, H, K), dim=-1).bfloat16() for _ in range(2))
    v, gate, beta = rn(B, T, H, K).bfloat16(), -rn(B, T, H).abs(), torch.sigmoid(rn(B, T, H))
    if name == "recurrent":
        state = torch.zeros(1, H, K, K, device="cuda")
        none = torch.full((B,), -1, dtype=torch.int32, device="cuda")   # no state: the same every time
        return lambda s: {"o": gdn.gdn_recurrent_fwd(q, k, v, gate, beta, torch.zeros(H, device="cuda"), state,
                                                     state_indices=none, stream=s)}
    if name == "chunk_bwd":   # (dq and dk are sums in an order of their own: dv stands for the result)
        return lambda s: {n: t for n, t in reversed(gdn.gdn_chunk_bwd(q, k, v, gate, beta, v, stream=s).items())
                          if n != "dh0"}
    if name == "chunk_staged":
        return lambda s: dict(zip(("o", "ht", "workspace"), gdn.gdn_chunk_fwd_staged(q, k, v, gate, beta, stream=s)))
    return lambda s: dict(zip(("o", "ht"), gdn.gdn_chunk_fwd(q, k, v, gate, beta, stream=s)))


NAMES = ["chunk_fwd", "chunk_staged", "chunk_bwd", "recurrent", "conv_fwd"]
REPEATS = ("o", "ht", "y", "dv")


def nbytes(t):
    return t.numel() * t.element_size()


@pytest.mark.parametrize("name", NAMES)
def test_memory_still_read_here(gdn, busy, name):
    """Work on the current stream that reads blocks freed just before the call sees their old values."""
    call = entry(gdn, name)
    ref = call(None)
    torch.cuda.synchronize()
    blocks = [torch.full((nbytes(t),), 7, dtype=torch.uint8, device="cuda") for t in ref.values()]
    copies = [torch.empty_like(b) for b in blocks]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy()
    for b, c in zip(blocks, copies):
        c.copy_(b)
    del blocks, b
    got = call(s.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.all(c == 7) for c in copies)
    assert all(torch.equal(got[k], ref[k]) for k in ref if k in REPEATS)


@pytest.mark.parametrize("name", NAMES)
def test_memory_dropped_here(gdn, busy, name):
    """Blocks allocated on the current stream after the call's results are dropped keep what they are filled with."""
    call = entry(gdn, name)
    ref = call(None)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        busy()
    got = call(s.cuda_stream)
    kept = next((k for k in ref if k in REPEATS), None) if len(ref) > 1 else None
    keep = got.get(kept)
    sizes = [nbytes(t) for k, t in got.items() if k != kept]
    del got
    fresh = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.all(f == 7) for f in fresh)
    assert keep is None or torch.equal(keep, ref[kept])


def test_host_call_workspace(gdn, busy):
    """The streamed call on host tensors: its workspace too waits for what is queued here."""
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.nn.functional.normalize(torch.randn(4, 256, 8, 128, generator=g), dim=-1).bfloat16()
               for _ in range(3))
    gate, beta = -torch.rand(4, 256, 8, generator=g), torch.rand(4, 256, 8, generator=g)
    p = gdn.problem_of(q, v, 64)
    n = max(int(gdn.gdn_chunk_fwd_host_workspace_size(p)), 256)
    ref = gdn.gdn_chunk_fwd_host(q, k, v, gate, beta)
    block = torch.full((n,), 7, dtype=torch.uint8, device="cuda")
    copy = torch.empty_like(block)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    busy()
    copy.copy_(block)
    del block
    got = gdn.gdn_chunk_fwd_host(q, k, v, gate, beta, stream=s.cuda_stream)
    assert torch.all(copy == 7) and torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
