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


# ---------------------------------------------------------------- a cache whose memory moves

def test_cache_data_replaced():
    """Pages taken elsewhere and back: calls use the tensor that is there, and leave the old one alone."""
    n_pages, page, H, d, T = 3, 16, 2, 64, 40
    k, v, slots = rand(T, H, d, seed=1).cuda(), rand(T, H, d, seed=2).cuda(), i32(range(T))
    cache = slope.KV4Cache(n_pages, page, H, d, d)
    old = cache.data
    old.zero_()
    slope.kv4_write(cache, k, v, slots)
    first, (want_k, want_v) = old.clone(), slope.kv4_read(cache, slots)
    cache.data = torch.zeros(old.numel() + 100, dtype=torch.uint8, device="cuda")
    slope.kv4_write(cache, v, k, slots)
    assert torch.equal(old, first) and not torch.equal(cache.data[:old.numel()], first) and (cache.data[old.numel():] == 0).all()
    cache.data = old
    got = slope.kv4_read(cache, slots)
    assert torch.equal(got[0], want_k) and torch.equal(got[1], want_v)
    table, lens, q = i32([[0, 1, 2]]), i32([T]), rand(1, 8, d, seed=3).cuda()
    out, lse = slope.kv4_attn(q, cache, table, lens)
    cache.data.set_(torch.cat([first, first]))  # in place: other memory behind the same tensor
    old_out, old_lse = slope.kv4_attn(q, cache, table, lens)
    assert torch.equal(out, old_out) and torch.equal(lse, old_lse)
