"""The calls on the 16-bit paged cache as programs use them: on streams, in graphs, after kernels that make their
arguments, over memory farther apart than 2^31 elements, in other layouts."""
import math

import pytest
import torch

import kv_oracle as ko
import ring_attention_slope_gb300 as slope
from test_gpu_kv import check, check_evict, check_weights, evict_case, i32, on_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    slope.build()
    slope.load()
    assert slope.device_status() == (0, 0)
    yield
    torch.cuda.synchronize()
    assert slope.device_status() == (0, 0)


def test_same_bits_on_streams_at_once():
    batch = ko.Batch([3000, 500, 77], [40, 1, 5], 16, 2, 64, 64, 64, seed=1)
    cache, table, n, cu = on_gpu(batch)
    q = batch.q.cuda()
    out, lse = slope.kv_attn(q, cache, table, n, cu_q=cu)
    weights = torch.zeros(batch.n_pages, 2, 64, device="cuda")
    slope.kv_attn_weights(q, cache, table, n, lse, weights, cu_q=cu, accumulate=False)
    check(out, lse, ko.attention(batch))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    results = []
    for _ in range(10):
        for s in streams:
            o, l = slope.kv_attn(q, cache, table, n, cu_q=cu, stream=s)
            with torch.cuda.stream(s):
                w = torch.zeros_like(weights)
            slope.kv_attn_weights(q, cache, table, n, l, w, cu_q=cu, accumulate=False, stream=s)
            results.append((o, l, w))
    torch.cuda.synchronize()
    for o, l, w in results:
        assert torch.equal(o, out) and torch.equal(l, lse) and torch.equal(w, weights)


@pytest.mark.parametrize("heads", [(8, 1, 64, 64), (4, 2, 128, 128)], ids=str)
def test_a_graph_follows_lengths_tables_and_rows(heads):
    """One capture, replayed for other lengths, pages and splits of the rows."""
    batches = [ko.Batch(lens, new, *heads, 16, seed=s)
               for s, (lens, new) in enumerate((([900, 40, 300], [1, 1, 30]), ([5, 1200, 33], [5, 20, 7]), ([64, 65, 2], [32, 0, 0])))]
    pages, width = max(b.n_pages for b in batches), max(b.table.shape[1] for b in batches)
    H, Hkv, dqk, dv = heads
    k, v = (torch.zeros(pages, Hkv, 16, d, dtype=torch.bfloat16, device="cuda") for d in (dqk, dv))
    cache = slope.KVCache(pages, 16, Hkv, dqk, dv, k=k, v=v)
    q = torch.zeros(32, H, dqk, dtype=torch.bfloat16, device="cuda")
    table, n, cu = torch.zeros(3, width, dtype=torch.int32, device="cuda"), i32([0, 0, 0]), i32([0, 0, 0, 0])
    weights = torch.zeros(pages, Hkv, 16, device="cuda")

    def load(b):
        k.fill_(math.nan), v.fill_(math.nan)
        k[:b.n_pages], v[:b.n_pages] = b.k.cuda(), b.v.cuda()
        table.fill_(-1)
        table[:, :b.table.shape[1]] = b.table.cuda()
        n.copy_(i32(b.lens)), cu.copy_(i32(b.cu))
        q[:b.q.shape[0]] = b.q.cuda()

    def run():
        out, lse = slope.kv_attn(q, cache, table, n, cu_q=cu, out_dtype=torch.float32)
        slope.kv_attn_weights(q, cache, table, n, lse, weights, cu_q=cu, accumulate=False)
        return out, lse

    load(batches[0])
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = run()
    for b in batches + batches[:1]:
        load(b)
        graph.replay()
        torch.cuda.synchronize()
        T = b.cu[-1]
        check(out[:T], lse[:, :T], ko.attention(b))
        check_weights(b, weights[:b.n_pages], lse[:, :T].cpu())


def test_a_captured_decode_step():
    """Store, attention, weights and eviction of a growing sequence, all in one graph."""
    H, Hkv, d, page = 8, 2, 64, 16
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn(40, Hkv, d, generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(40, H, d, generator=g).to(torch.bfloat16)
    cache = slope.KVCache(8, page, Hkv, d, d)
    cache.k.fill_(math.nan), cache.v.fill_(math.nan)
    weights = torch.full((8, Hkv, page), math.nan, device="cuda")
    table = i32([[3, 1, 6]])
    n, now = i32([0]), dict(q=q[:1].cuda(), k=k[:1].cuda(), v=v[:1].cuda(), slot=i32([0]))
    kept = i32(torch.zeros(1, Hkv, 32))

    def step():
        slope.kv_write(cache, now["k"], now["v"], now["slot"], weights=weights)
        n.add_(1)
        out, lse = slope.kv_attn(now["q"], cache, table, n, out_dtype=torch.float32)
        slope.kv_attn_weights(now["q"], cache, table, n, lse, weights)
        slope.kv_evict(cache, weights, table, n, 32, recent=4, kept=kept, out_lens=n)
        return out

    slots = [int(table[0, t // page]) * page + t % page for t in range(33)]
    now["slot"].fill_(slots[0])
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    n.zero_()
    with torch.cuda.graph(graph):
        out = step()
    n.zero_()
    alive = [list(range(0)) for _ in range(Hkv)]  # tokens of each head
    w = [dict() for _ in range(Hkv)]
    for i in range(40):
        now["q"].copy_(q[i:i + 1]), now["k"].copy_(k[i:i + 1]), now["v"].copy_(v[i:i + 1])
        now["slot"].fill_(slots[min(i, 32)])
        graph.replay()
        torch.cuda.synchronize()
        for h in range(Hkv):
            alive[h].append(i)
            w[h][i] = 0.0
            for j in range(H // Hkv):
                head = h * (H // Hkv) + j
                s = k[alive[h], h].double() @ q[i, head].double() * d ** -0.5
                p = torch.softmax(s, 0)
                want = p @ v[alive[h], h].double()
                off = (2.0 ** -8 + 2.0 ** -13) * (p @ v[alive[h], h].double().abs())
                assert ((out[0, head].cpu().double() - want).abs() <= off).all(), (i, h)
                for t, x in zip(alive[h], p.tolist()):
                    w[h][t] += x
            if len(alive[h]) > 32:
                # the weights of the random scores are far enough apart for their order to be the same
                stay = ko.choose(torch.tensor([w[h][t] for t in alive[h]], dtype=torch.float64), 32, 0, 4)
                assert kept[0, h].tolist() == stay
                alive[h] = [alive[h][t] for t in stay]
        assert n.item() == min(i + 1, 32)


def test_arguments_made_by_the_kernel_before():
    """The calls' kernels may start early, but read nothing before the kernels ahead of them are done."""
    batch = ko.Batch([700, 90], [1, 1], 8, 2, 64, 64, 16, seed=7)
    cache, table, n, _ = on_gpu(batch)
    q, ref = batch.q.cuda(), ko.attention(batch)
    lse0 = ref[1].float().cuda()
    ek, ew = evict_case([700, 90], 2, 64, 64, 16, seed=7)
    ecache, etable, en, _ = on_gpu(ek)
    rows = torch.randn(300, 2, 64, device="cuda").to(torch.bfloat16)
    slots = torch.randperm(cache.n_pages * 16, device="cuda")[:300].int()
    for _ in range(5):
        out = torch.empty(2, 8, 64, device="cuda")
        bad_q, bad_n, bad_t = torch.zeros_like(q), torch.zeros_like(n), torch.full_like(table, -1)
        torch.cuda._sleep(300000)
        bad_q.copy_(q), bad_t.copy_(table), bad_n.copy_(n)
        _, lse = slope.kv_attn(bad_q, cache, bad_t, bad_n, out=out)
        check(out, lse, ref)
        w, late = torch.full((batch.n_pages, 2, 16), math.nan, device="cuda"), torch.zeros_like(lse0)
        bad_n.zero_()
        torch.cuda._sleep(300000)
        late.copy_(lse0), bad_n.copy_(n)
        slope.kv_attn_weights(q, cache, table, bad_n, late, w, accumulate=False)
        check_weights(batch, w, lse0.cpu())
        k, v, wg = ek.k.cuda(), ek.v.cuda(), torch.zeros_like(ew).cuda()
        c = slope.KVCache(ek.n_pages, 16, 2, 64, 64, k=k, v=v)
        bad_n, good = torch.zeros_like(en), ew.cuda()
        torch.cuda._sleep(300000)
        wg.copy_(good), bad_n.copy_(en)
        got = slope.kv_evict(c, wg, etable, bad_n, 64, out_lens=bad_n)
        check_evict(ek, ew, 64, 0, 0, got, [(ek.k, k), (ek.v, v), (ew, wg)])
        c = slope.KVCache(cache.n_pages, 16, 2, 64, 64)
        late = torch.zeros_like(rows)
        torch.cuda._sleep(300000)
        late.copy_(rows)
        slope.kv_write(c, late, late, slots)
        at = slots.long()
        assert torch.equal(c.k[at // 16, :, at % 16], rows) and torch.equal(c.v[at // 16, :, at % 16], rows)


@pytest.mark.parametrize("heads", [(8, 2, 64, 64), (2, 2, 192, 128)], ids=str)
def test_memory_farther_apart_than_32_bits(heads):
    """Pages 2^31 elements apart, in the caches and in the weights."""
    H, Hkv, dqk, dv = heads
    page, far = 64, 2 ** 31 + 64
    batch = ko.Batch([130, 40], [20, 1], H, Hkv, dqk, dv, page, seed=8, extra_pages=0)
    assert batch.n_pages == 4

    def spread(x):
        room = torch.empty((batch.n_pages - 1) * far + x[0].numel(), dtype=x.dtype, device="cuda")
        y = room.as_strided(x.shape, (far, *x.stride()[1:]))
        y.copy_(x)
        return y

    k, v = spread(batch.k), spread(batch.v)
    cache = slope.KVCache(batch.n_pages, page, Hkv, dqk, dv, k=k, v=v)
    q, table, n, cu = batch.q.cuda(), batch.table.cuda(), i32(batch.lens), i32(batch.cu)
    out, lse = slope.kv_attn(q, cache, table, n, cu_q=cu)
    check(out, lse, ko.attention(batch))
    w = spread(torch.zeros(batch.n_pages, Hkv, page))
    slope.kv_attn_weights(q, cache, table, n, lse, w, cu_q=cu)
    check_weights(batch, w.contiguous(), lse.cpu())
    before = [x.contiguous().cpu() for x in (k, v, w)]
    got = slope.kv_evict(cache, w, table, n, 50, first=1, recent=9)
    check_evict(batch, before[2], 50, 1, 9, got, list(zip(before, (x.contiguous() for x in (k, v, w)))))
    rows = [torch.randn(2, Hkv, d, device="cuda").to(torch.bfloat16) for d in (dqk, dv)]
    slope.kv_write(cache, *rows, i32([3 * page + 63, 70]), weights=w)
    for x, r in zip((k, v), rows):
        assert torch.equal(x[3, :, 63], r[0]) and torch.equal(x[1, :, 6], r[1])
    assert (w[3, :, 63] == 0).all() and (w[1, :, 6] == 0).all()


def test_token_major_weights_and_eviction():
    batch, w = evict_case([100, 55], 3, 64, 64, 32, seed=9)
    k, v = (x.transpose(1, 2).contiguous().cuda().transpose(1, 2) for x in (batch.k, batch.v))
    cache = slope.KVCache(batch.n_pages, 32, 3, 64, 64, k=k, v=v)
    wide = torch.full((batch.n_pages, 3, 50), 7.0, device="cuda")  # rows with room behind them
    wg = wide[:, :, :32]
    wg.copy_(w)
    got = slope.kv_evict(cache, wg, batch.table.cuda(), i32(batch.lens), 40, recent=3)
    check_evict(batch, w, 40, 0, 3, got, [(batch.k, k.contiguous()), (batch.v, v.contiguous()), (w, wg.contiguous())])
    assert (wide[:, :, 32:] == 7).all()


def test_outputs_and_workspaces_given():
    batch = ko.Batch([2000, 3], [2, 2], 8, 2, 64, 64, 16, seed=10)
    cache, table, n, _ = on_gpu(batch)
    q = batch.q.cuda()
    ref = ko.attention(batch)
    size = slope.kv_attn_workspace_size(4, 8, cache, 2)
    most = max(size, slope.kv_attn_weights_workspace_size(4, 8, cache, 2), slope.kv_evict_workspace_size(2, cache, 100))
    guard = torch.full((most + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    room = torch.full((4, 10, 72), 3.0, device="cuda")
    out, lse = room[:, 1:9, 4:68], torch.full((4, 16), 3.0, device="cuda").t()[::2, :]
    got = slope.kv_attn(q, cache, table, n, q_len=2, out=out, lse=lse, workspace=guard[256:256 + size])
    assert got[0] is out and got[1] is lse
    check(out, lse, ref)
    assert (guard[:256] == 0xA5).all() and (guard[256 + size:] == 0xA5).all()
    assert (room[:, 0] == 3).all() and (room[:, 9] == 3).all() and (room[:, :, :4] == 3).all() and (room[:, :, 68:] == 3).all()
    assert slope.kv_attn(q, cache, table, n, q_len=2, want_lse=False)[1] is None
    with pytest.raises(slope.SlopeError):
        slope.kv_attn(q, cache, table, n, q_len=2, workspace=guard[256:256 + size - 1])
    wsize = slope.kv_attn_weights_workspace_size(4, 8, cache, 2)
    w = torch.zeros(batch.n_pages, 2, 16, device="cuda")
    slope.kv_attn_weights(q, cache, table, n, lse.contiguous(), w, q_len=2, workspace=guard[256:256 + wsize])
    check_weights(batch, w, lse.cpu())
    esize = slope.kv_evict_workspace_size(2, cache, 100)
    guard.fill_(0xA5)
    slope.kv_evict(cache, w, table, n, 100, workspace=guard[256:256 + esize])
    torch.cuda.synchronize()
    assert (guard[:256] == 0xA5).all() and (guard[256 + esize:] == 0xA5).all()


def test_a_cache_whose_memory_moves():
    batch = ko.Batch([50], [1], 4, 2, 64, 64, 16, seed=11)
    cache, table, n, _ = on_gpu(batch)
    ref = ko.attention(batch)
    check(*slope.kv_attn(batch.q.cuda(), cache, table, n), ref)
    moved = cache.k.clone()
    cache.k.set_(moved)
    check(*slope.kv_attn(batch.q.cuda(), cache, table, n), ref)
    cache.k.untyped_storage().resize_(16)
    with pytest.raises(ValueError):
        slope.kv_attn(batch.q.cuda(), cache, table, n)


def test_long_sequences_of_many_pieces():
    """Cuts of many lengths: what a piece ends on, and how many there are of a pair, changes nothing."""
    for lens, new, heads in (([20000], [1], (8, 1, 64, 64)), ([20000, 3], [64, 3], (4, 1, 64, 64)),
                             ([9000] * 3, [1] * 3, (8, 8, 64, 64)), ([6000], [300], (2, 2, 192, 128)),
                             ([15000], [2], (6, 1, 128, 128))):
        batch = ko.Batch(lens, new, *heads, 64, seed=sum(lens))
        cache, table, n, cu = on_gpu(batch)
        out, lse = slope.kv_attn(batch.q.cuda(), cache, table, n, cu_q=cu, out_dtype=torch.float32)
        check(out, lse, ko.attention(batch))
        w = torch.zeros(batch.n_pages, heads[1], 64, device="cuda")
        slope.kv_attn_weights(batch.q.cuda(), cache, table, n, lse, w, cu_q=cu)
        check_weights(batch, w, lse.cpu())


def ragged(n, longest, most, seed):
    gen = torch.Generator().manual_seed(seed)
    lens = torch.randint(0, longest + 1, (n,), generator=gen).tolist()
    return lens, [min(a, int(torch.randint(0, most + 1, (1,), generator=gen))) for a in lens]


@pytest.mark.parametrize("lens, new, heads, window", [
    ([1500, 1490], [640, 640], (32, 4, 64, 64), 0),          # more pairs than CTAs: full rounds, then shares
    ([900] * 8, [600] * 8, (8, 4, 128, 128), 0),             # the same with two Q tiles, the last block half empty
    ([2600, 2600, 400], [520, 300, 90], (5, 1, 64, 64), 700),
    (*ragged(70, 1500, 60, 1), (5, 1, 64, 64), 0),           # more than two warps' lanes of sequences
    (*ragged(70, 1500, 60, 2), (10, 2, 64, 64), 200),
    (*ragged(45, 900, 300, 3), (4, 2, 192, 128), 0),
    (*ragged(530, 300, 3, 4), (4, 1, 64, 64), 0),            # two launches
    (*ragged(40, 5000, 1, 5), (8, 4, 64, 64), 0),
], ids=["rounds", "two_tiles", "window", "many", "many_window", "wide", "two_launches", "decode"])
def test_shares_of_many_pairs(lens, new, heads, window):
    """Where the work is dealt out in full rounds of whole pairs and equal shares of the rest, every pair is there once."""
    batch = ko.Batch(lens, new, *heads, 16, seed=len(lens))
    cache, table, n, cu = on_gpu(batch)
    out, lse = slope.kv_attn(batch.q.cuda(), cache, table, n, cu_q=cu, window=window, out_dtype=torch.float32)
    check(out, lse, ko.attention(batch, window=window))


def test_a_graph_replayed_beside_thousands_of_calls():
    """A recorded call keeps the counter that its CTAs claim their work from; calls on streams never come round to it."""
    batch = ko.Batch([700, 90, 1500], [1, 1, 1], 16, 2, 64, 64, 16, seed=21)
    cache, table, n, _ = on_gpu(batch)
    q = batch.q.cuda()
    out, lse = slope.kv_attn(q, cache, table, n, q_len=1)
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        got = [slope.kv_attn(q, cache, table, n, q_len=1) for _ in range(4)]
    mine = torch.zeros_like(out)
    work = torch.empty(slope.kv_attn_workspace_size(3, 16, cache, 1), dtype=torch.uint8, device="cuda")
    side.wait_stream(torch.cuda.current_stream())
    for i in range(4500):
        if i % 20 == 0:
            graph.replay()
        slope.kv_attn(q, cache, table, n, q_len=1, out=mine, want_lse=False, workspace=work, stream=side)
        if i % 500 == 499:
            torch.cuda.synchronize()
            assert (mine == out).all()
            for o, l in got:
                assert (o == out).all() and (l == lse).all()
                o.zero_(), l.zero_()
            mine.zero_()
            torch.cuda.synchronize()
    assert slope.device_status() == (0, 0)
