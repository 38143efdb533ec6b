"""Edges of the serving calls on the GPU that a server meets and the tests of single calls do not."""
import pytest
import torch

import ring_attention_slope_gb300 as slope
from test_gpu_serving import i32, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    slope.build()
    slope.load()
    assert slope.device_status() == (0, 0)
    yield
    torch.cuda.synchronize()
    assert slope.device_status() == (0, 0)


# ---------------------------------------------------------------- no tokens

@pytest.mark.parametrize("Hq,H,dqk,dv", [(8, 1, 64, 64), (4, 4, 192, 128)])
def test_calls_without_tokens(Hq, H, dqk, dv):
    """Outputs left to the calls, as a server's step without sequences makes them."""
    q, k, v = rand(0, Hq, dqk).cuda(), rand(0, H, dqk).cuda(), rand(0, H, dv).cuda()
    for cu in ([0], [0, 0], [0] * 300):
        out, lse = slope.attn_varlen(q, k, v, cu)
        assert out.shape == (0, Hq, dv) and lse.shape == (Hq, 0) and out.dtype == torch.bfloat16
    cache, none = slope.KV4Cache(4, 16, H, dqk, dv), i32([])
    slope.kv4_write(cache, k, v, none)
    assert [x.shape for x in slope.kv4_read(cache, none)] == [(0, H, dqk), (0, H, dv)]
    for pages in (0, 4):
        for q_len in (1, 5):
            out, lse = slope.kv4_attn(q, cache, torch.zeros(0, pages, dtype=torch.int32, device="cuda"), none, q_len=q_len)
            assert out.shape == (0, Hq, dv) and lse.shape == (Hq, 0)
