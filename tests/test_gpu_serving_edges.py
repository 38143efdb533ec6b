"""Edges of the serving calls on the GPU that a server meets and the tests of single calls do not."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import ring_attention_slope_gb300 as slope
from test_gpu_serving import check_varlen, i32, packed, rand

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


# ---------------------------------------------------------------- memory that a call allocates

def outputs_of_the_calls(stream=None):
    """One of each call with its outputs left to it, rows that no sequence or slot covers among them."""
    T, H, d = 40, 2, 64
    q, k = rand(T, 8, d, seed=4).cuda(), rand(T, H, d, seed=5).cuda()
    cache, slots = slope.KV4Cache(3, 16, H, d, d, data=torch.zeros(3 * H * 1280, dtype=torch.uint8, device="cuda")), i32(range(T))
    slots[-1] = -1
    torch.cuda.synchronize()
    return [*slope.qk_norm_rope(q, k, stream=stream), *slope.attn_varlen(q, k, k, [5, 30], stream=stream),
            *slope.kv4_read(cache, slots, stream=stream),
            *slope.kv4_attn(q[:1], cache, i32([[0, 1, 2]]), i32([T]), stream=stream)]


@pytest.mark.parametrize("side", [False, True])
def test_deterministic_fill_of_what_is_not_written(side):
    """With deterministic algorithms PyTorch fills uninitialised memory, rows that a call leaves as they were too."""
    stream = torch.cuda.Stream() if side else None
    for t in outputs_of_the_calls(stream):  # blocks of these sizes with other numbers in them, freed again
        t.fill_(7)
    torch.cuda.synchronize()
    del t
    torch.use_deterministic_algorithms(True)
    try:
        _, _, out, lse, k, v, *_ = outputs_of_the_calls(stream)
    finally:
        torch.use_deterministic_algorithms(False)
    torch.cuda.synchronize()
    for rest in (out[:5], out[30:], lse[:, :5], lse[:, 30:], k[-1], v[-1]):
        assert torch.isnan(rest).all()
    for written in (out[5:30], lse[:, 5:30], k[:-1], v[:-1]):
        assert torch.isfinite(written).all()


def test_dispatch_modes_see_the_allocations():
    class Watch(TorchDispatchMode):
        seen = []

        def __torch_dispatch__(self, func, types, args=(), kwargs=None):
            r = func(*args, **(kwargs or {}))
            if "empty" in str(func):
                self.seen.append(r.data_ptr())
            return r

    with Watch():
        outputs = outputs_of_the_calls()
    torch.cuda.synchronize()
    assert {t.data_ptr() for t in outputs} <= set(Watch.seen)


# ---------------------------------------------------------------- long lists of wide prompts

MANY = [(11 * i) % 47 if i % 9 else 0 for i in range(290)] + [1, 300, 0, 129, 700]  # three launches, empty ones among them


@pytest.mark.parametrize("dqk,dv", [(128, 128), (192, 64), (192, 128), (128, 64), (64, 128)])
@pytest.mark.parametrize("Hq,H", [(2, 2), (8, 2), (5, 1)])
def test_varlen_many_wide_sequences(dqk, dv, Hq, H):
    """More sequences than a launch takes, where launches overlap and claim their tiles at run time."""
    q, k, v, cu = packed(MANY, Hq, H, dqk, dv, 400, lead=2, tail=9)
    for x in (q, k, v):
        x[:2] = x[cu[-1]:] = float("nan")
    check_varlen(q, k, v, cu)


@pytest.mark.parametrize("dqk,dv,Hq,H", [(128, 128, 4, 1), (192, 128, 2, 2), (192, 64, 8, 2)])
def test_varlen_wide_captured(dqk, dv, Hq, H):
    """Replays find the claimed tiles' counters as the capture's launches did, between calls outside the graph too."""
    q, k, v, cu = packed(MANY, Hq, H, dqk, dv, 410)
    q, k, v = q.cuda(), k.cuda(), v.cuda()
    ref, rl = slope.attn_varlen(q, k, v, cu)
    out, lse = torch.zeros_like(ref), torch.zeros_like(rl)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for _ in range(2):
            slope.attn_varlen(q, k, v, cu, out=out, lse=lse)
    for _ in range(3):
        out.zero_()
        lse.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref) and torch.equal(lse, rl)
        again, al = slope.attn_varlen(q, k, v, cu)
        assert torch.equal(again, ref) and torch.equal(al, rl)
