"""Bounded waits of linear attention's fp32 gradients, exercised on the GPU without a fault: the test hook makes the wait
for one batch of products run out in some of the first CTA's warps (its products do end).  The launch has to end all the
same, report it, spoil nothing but that CTA's tokens, and leave a workspace on which the next call is exact."""
import ctypes

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def gdn():
    from gated_deltanet_chunked_gdn_gb300 import binding
    lib = binding.load()
    lib.gdn_selftest_linear_grads_timeout.argtypes = (
        [ctypes.POINTER(binding.LinearProblem)] + [ctypes.c_void_p] * 4 + [ctypes.c_float] + [ctypes.c_void_p] * 6 +
        [ctypes.c_size_t, ctypes.c_int, ctypes.c_uint, ctypes.c_void_p])
    lib.gdn_selftest_linear_grads_timeout.restype = ctypes.c_int
    return binding


# batches of products: K / 64, then K / 128 times V / 64 and one, then V / 128 times K / 64
@pytest.mark.parametrize("K,V,batches", [(128, 128, 7), (256, 256, 22), (256, 128, 14)])
def test_waits_that_run_out_in_some_warps(gdn, K, V, batches):
    torch.manual_seed(0)
    q, k = torch.randn(1, 150, 2, K, device=DEV), torch.randn(1, 150, 2, K, device=DEV)
    v, do = torch.randn(1, 150, 2, V, device=DEV), torch.randn(1, 150, 2, V, device=DEV)
    g = -torch.rand(1, 150, 2, device=DEV)
    want = gdn.gdn_linear_attn_bwd(q, k, v, g, do, scale=0.25)
    ws, lib = want["workspace"], gdn.load()
    p = gdn._linear_problem(q, k, v, g, None)
    stream = torch.cuda.current_stream().cuda_stream
    names = ("dq", "dk", "dv", "dg")

    def call(batch, warps):
        out = [torch.zeros_like(want[n]) for n in names]
        st = lib.gdn_selftest_linear_grads_timeout(p, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), 0.25,
                                                   do.data_ptr(), *(t.data_ptr() for t in out), ws.data_ptr(),
                                                   ws.numel(), batch, warps, stream)
        assert st == 0
        torch.cuda.synchronize()   # the launch ends
        return out, gdn.gdn_linear_attn_get_device_status(ws)

    for batch in range(batches):
        for warps in (0x0001, 0x8000, 0x0220, 0xfffe, 0x00ff, 0xffff):
            out, status = call(batch, warps)
            assert status == gdn.DEV_WAIT_TIMEOUT, (batch, warps)
            for n, t in zip(names, out):
                a, b = t.clone(), want[n].clone()
                a[:, :64, 0] = 0
                b[:, :64, 0] = 0
                assert torch.equal(a, b), (batch, warps, n)
    out, status = call(batches, 0xffff)   # there is no such batch
    assert status == gdn.DEV_OK and all(torch.equal(t, want[n]) for n, t in zip(names, out))
    again = gdn.gdn_linear_attn_bwd(q, k, v, g, do, scale=0.25, workspace=ws)
    assert gdn.gdn_linear_attn_get_device_status(ws) == gdn.DEV_OK
    assert all(torch.equal(again[n], want[n]) for n in names)
