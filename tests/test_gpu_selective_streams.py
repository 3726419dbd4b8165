"""Calls of the selective layer's operators on another stream than the current one:
the blocks that a call allocates itself are not written before work queued earlier
on the current stream is done with their memory, and not given out again before the
other stream is done with them."""
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


def scan_inputs():
    g = torch.Generator(device="cuda").manual_seed(1)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")
    bf = lambda *s: rn(*s).bfloat16()
    return {"x": bf(2, 1024, 1024), "delta": bf(2, 1024, 1024), "A": -rn(1024, 16).abs(), "B": bf(2, 1024, 1, 16),
            "C": bf(2, 1024, 1, 16), "z": bf(2, 1024, 1024), "D": rn(1024), "dt_bias": rn(1024) - 3}


def operator(gdn, name):
    """call(stream) -> a dict of every tensor that the call has allocated and returns."""
    i = scan_inputs()
    if name == "scan_fwd":
        return lambda s: dict(zip(("y", "ht"), gdn.gdn_selective_scan_fwd(**i, stream=s)))
    if name == "scan_bwd":
        return lambda s: {k: v for k, v in gdn.gdn_selective_scan_bwd(**i, dout=i["z"], stream=s).items()
                          if v is not None}
    if name == "scan_step":
        i = {k: v.reshape(2048, 1, *v.shape[2:]) if v.dim() > 2 else v for k, v in i.items()}
        state = torch.zeros(1, 1024, 16, device="cuda")
        none = torch.full((2048,), -1, dtype=torch.int32, device="cuda")   # no state: zeros, the same every time
        return lambda s: {"y": gdn.gdn_selective_scan_step(**i, state=state, state_indices=none, stream=s)}
    if name == "conv_bwd":
        w = torch.randn(1024, 4, device="cuda")
        return lambda s: {k: v for k, v in gdn.gdn_causal_conv1d_bwd(i["x"], w, i["z"], stream=s).items()
                          if v is not None}
    x = i["x"].view(2048, 1024)[:64]
    q = torch.randint(0, 256, (32768, 512), dtype=torch.uint8, device="cuda")
    sc = torch.rand(32768, 8, device="cuda").bfloat16()
    return lambda s: {"y": gdn.gdn_q4_matvec(x, q, sc, stream=s)}


NAMES = ["scan_fwd", "scan_bwd", "scan_step", "conv_bwd", "q4"]


def nbytes(t):
    return t.numel() * t.element_size()


@pytest.mark.parametrize("name", NAMES)
def test_memory_still_read_here(gdn, busy, name):
    """Work on the current stream that reads blocks freed just before the call sees their old values."""
    call = operator(gdn, name)
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
    assert all(torch.equal(got[k], ref[k]) for k in ref if k != "workspace")


@pytest.mark.parametrize("name", NAMES)
def test_memory_dropped_here(gdn, busy, name):
    """Blocks allocated on the current stream after the call's results are dropped keep what they are filled with."""
    call = operator(gdn, name)
    ref = call(None)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        busy()
    got = call(s.cuda_stream)
    kept = next(iter(ref))
    keep = got[kept] if len(ref) > 1 else None
    sizes = [nbytes(t) for k, t in got.items() if k != kept or keep is None]
    del got
    fresh = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    torch.cuda.synchronize()
    assert all(torch.all(f == 7) for f in fresh)
    assert keep is None or torch.equal(keep, ref[kept])
