"""Malformed offsets: the backward pass leaves every gradient as it was, in each of its forms (bf16 on the tensor cores,
fp32, bf16 with a head dim of 256; heads that share q and k, whose dq and dk a launch of its own adds; fixed decays, whose
dg another adds)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def gdn():
    from gated_deltanet_chunked_gdn_gb300 import binding
    binding.load()
    return binding


@pytest.mark.parametrize("bad", [[0, 50, 40, 100], [1, 50, 60, 100], [0, 50, 60, 99], [0, -3, 60, 100],
                                 [0, 200, 60, 100], [0, 50, 60, 101]])
@pytest.mark.parametrize("dtype,K,V", [(BF, 128, 128), (BF, 64, 128), (BF, 256, 128), (BF, 64, 256), (F32, 128, 64),
                                       (F32, 256, 256)])
@pytest.mark.parametrize("Hqk", [1, 2])
@pytest.mark.parametrize("per_head", [False, True])
def test_gradients_stay_as_they_were(gdn, bad, dtype, K, V, Hqk, per_head):
    q, k = (torch.randn(1, 100, Hqk, K, device=DEV).to(dtype) for _ in range(2))
    v, do = (torch.randn(1, 100, 2, V, device=DEV).to(dtype) for _ in range(2))
    g = -torch.rand(2, device=DEV) if per_head else -torch.rand(1, 100, 2, device=DEV)
    cu = torch.tensor(bad, dtype=torch.int32, device=DEV)
    h0, dht = torch.randn(3, 2, K, V, device=DEV), torch.randn(3, 2, K, V, device=DEV)
    p = gdn._linear_problem(q, k, v, g, cu)
    ws = torch.zeros(gdn.gdn_linear_attn_bwd_workspace_size(p), dtype=torch.uint8, device=DEV)
    out = [torch.full_like(t, 3.0) for t in (q, k, v, g, h0)]
    st = gdn.load().gdn_linear_attn_bwd(p, q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), 0.25, h0.data_ptr(),
                                        cu.data_ptr(), do.data_ptr(), dht.data_ptr(), *(t.data_ptr() for t in out),
                                        ws.data_ptr(), ws.numel(), torch.cuda.current_stream().cuda_stream)
    assert st == 0 and gdn.gdn_linear_attn_get_device_status(ws) == gdn.DEV_BAD_CU_SEQLENS
    for n, t in zip(("dq", "dk", "dv", "dg", "dh0"), out):
        assert bool((t == 3.0).all()), n


def test_each_call_leaves_its_own_word(gdn):
    """Good and bad calls in turn on a stream that does not wait for the default one."""
    q = torch.randn(1, 100, 1, 64, device=DEV)
    g = -torch.rand(1, 100, 1, device=DEV)
    good, bad = (torch.tensor(c, dtype=torch.int32, device=DEV) for c in ([0, 50, 100], [0, 50, 99]))
    p = gdn._linear_problem(q, q, q, g, good)
    ws = torch.zeros(gdn.gdn_linear_attn_fwd_workspace_size(p), dtype=torch.uint8, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for i in range(50):
            for cu, want in ((bad, gdn.DEV_BAD_CU_SEQLENS), (good, gdn.DEV_OK), (bad, gdn.DEV_BAD_CU_SEQLENS)):
                gdn.gdn_linear_attn_fwd(q, q, q, g, cu_seqlens=cu, workspace=ws)
                assert gdn.gdn_linear_attn_get_device_status(ws) == want
            assert gdn.gdn_linear_attn_get_device_status(ws) == gdn.DEV_OK
