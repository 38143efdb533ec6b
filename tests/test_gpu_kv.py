"""The calls on the 16-bit paged cache against plain forms in 64 bits (tests/kv_oracle.py, which says how far fp32 and the
one bf16 rounding of the weights may be off).  An output's own rounding to bf16 is off by at most 2^-8 of the value, to fp32 by 2^-24."""
import math

import pytest
import torch

import kv_oracle as ko
import ring_attention_slope_gb300 as slope

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


@pytest.fixture(scope="module", autouse=True)
def _built():
    slope.build()
    slope.load()
    assert slope.device_status() == (0, 0)
    yield
    torch.cuda.synchronize()
    assert slope.device_status() == (0, 0)


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def on_gpu(batch):
    """(cache, block table, lengths, cu_q) of a batch."""
    k, v = batch.k.cuda(), batch.v.cuda()
    if batch.token_major:
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    cache = slope.KVCache(batch.n_pages, batch.page, batch.Hkv, batch.dqk, batch.dv, k=k, v=v)
    return cache, batch.table.cuda(), i32(batch.lens), i32(batch.cu)


def check(out, lse, ref):
    want, want_lse, off, lse_off = ref
    out, lse = out.cpu(), lse.cpu()
    bad = (out.double() - want).abs() > off + HALF[out.dtype] * want.abs() + 1e-30
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist(), float((out.double() - want).abs().max()))
    assert not out.isnan().any()
    none = want_lse == -math.inf
    assert torch.equal(lse == -math.inf, none)
    bad = ((lse.double() - want_lse).abs() > lse_off)[~none]
    assert not bad.any(), float((lse.double() - want_lse)[~none].abs().max())


HEADS = [(8, 1, 64, 64), (5, 1, 64, 64), (6, 2, 128, 128), (3, 3, 192, 128), (4, 2, 64, 128), (12, 1, 128, 64),
         (2, 1, 192, 64)]
LENS = {
    "one_token": ([1, 16, 127, 128, 129, 700], [1] * 6),
    "none": ([0, 5, 0], [1, 1, 2]),
    "chunks": ([300, 257, 40], [300, 130, 3]),
    "mixed": ([513, 64, 1, 999], [200, 1, 1, 0]),
    "more_new_than_cached": ([3, 100], [9, 140]),
    "long": ([5000], [1]),
    "long_chunk": ([3001], [70]),
}


@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("heads", HEADS, ids=str)
def test_attention(heads, lens):
    batch = ko.Batch(*LENS[lens], *heads, 16 if heads[0] % 2 else 64, seed=len(lens))
    cache, table, n, cu = on_gpu(batch)
    out, lse = slope.kv_attn(batch.q.cuda(), cache, table, n, cu_q=cu, out_dtype=torch.float32)
    check(out, lse, ko.attention(batch))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 1024])
@pytest.mark.parametrize("token_major", [False, True])
def test_attention_pages(page, token_major):
    batch = ko.Batch([1500, 77, 640], [33, 1, 128], 16, 2, 64, 64, page, token_major=token_major, seed=page)
    cache, table, n, cu = on_gpu(batch)
    out, lse = slope.kv_attn(batch.q.cuda(), cache, table, n, cu_q=cu)
    assert out.dtype == torch.bfloat16
    check(out, lse, ko.attention(batch))


@pytest.mark.parametrize("window", [1, 100, 128, 1000])
@pytest.mark.parametrize("heads", [(8, 1, 64, 64), (2, 2, 192, 128)], ids=str)
def test_attention_window(heads, window):
    batch = ko.Batch([900, 300, 1], [1, 290, 1], *heads, 16, seed=window)
    cache, table, n, cu = on_gpu(batch)
    out, lse = slope.kv_attn(batch.q.cuda(), cache, table, n, cu_q=cu, window=window, scale=0.2)
    check(out, lse, ko.attention(batch, window=window, scale=0.2))


@pytest.mark.parametrize("q_len", [1, 4, 33])
def test_attention_equal_runs(q_len):
    batch = ko.Batch([1000, 40, 333], [q_len] * 3, 8, 2, 64, 64, 32, seed=q_len)
    cache, table, n, cu = on_gpu(batch)
    q = batch.q.cuda()
    out, lse = slope.kv_attn(q, cache, table, n, q_len=q_len)
    check(out, lse, ko.attention(batch))
    again, lse2 = slope.kv_attn(q, cache, table, n, cu_q=cu)
    assert torch.equal(out, again) and torch.equal(lse, lse2)


def test_attention_large_group():
    """More query heads to a key head than a tile has rows."""
    batch = ko.Batch([200, 31], [3, 1], 131, 1, 64, 64, 16, seed=3)
    cache, table, n, cu = on_gpu(batch)
    out, lse = slope.kv_attn(batch.q.cuda(), cache, table, n, cu_q=cu)
    check(out, lse, ko.attention(batch))


def test_attention_many_sequences():
    """More sequences than a launch takes, among them empty ones."""
    lens = [(7 * i) % 50 for i in range(1100)]
    batch = ko.Batch(lens, [1 + i % 2 for i in range(1100)], 4, 1, 64, 64, 16, seed=4)
    cache, table, n, cu = on_gpu(batch)
    out, lse = slope.kv_attn(batch.q.cuda(), cache, table, n, cu_q=cu)
    check(out, lse, ko.attention(batch))


def test_attention_missing_pages():
    batch = ko.Batch([600, 600, 40], [1, 90, 2], 8, 1, 64, 64, 16, seed=5)
    gone = {(0, 3): -1, (0, 20): 10 ** 6, (1, 0): -5, (1, 30): batch.n_pages, (2, 0): -1, (2, 1): -1, (2, 2): 2 ** 31 - 1}
    for (b, e), p in gone.items():
        batch.table[b, e] = p

    def missing(b):
        page = torch.arange(batch.lens[b]) // batch.page
        return torch.tensor([(b, int(e)) in gone for e in page])

    cache, table, n, cu = on_gpu(batch)
    out, lse = slope.kv_attn(batch.q.cuda(), cache, table, n, cu_q=cu)
    check(out, lse, ko.attention(batch, missing=missing))


def test_attention_leaves_other_rows():
    batch = ko.Batch([100, 50], [4, 2], 4, 2, 64, 64, 16, seed=6)
    cache, table, n, _ = on_gpu(batch)
    q = torch.cat((torch.full((3, 4, 64), math.nan), batch.q.float(), torch.full((2, 4, 64), math.nan))).to(torch.bfloat16).cuda()
    out = torch.full((11, 4, 64), 5.0, device="cuda")
    lse = torch.full((4, 11), 5.0, device="cuda")
    slope.kv_attn(q, cache, table, n, cu_q=i32([3, 7, 9]), out=out, lse=lse)
    check(out[3:9], lse[:, 3:9], ko.attention(batch))
    for x in (out[:3], out[9:], lse[:, :3], lse[:, 9:]):
        assert (x == 5).all()
    # bounds out of range are cut off, and lengths too
    out.fill_(5.0)
    slope.kv_attn(q[3:9], cache, table, i32([100, 50]), cu_q=i32([-9, 4, 10 ** 9]), out=out[3:9], lse=lse[:, 3:9])
    check(out[3:9], lse[:, 3:9], ko.attention(batch))
    slope.kv_attn(q[3:9], cache, table, i32([-3, 10 ** 9]), cu_q=i32([5, 2, 6]), out=out[3:9], lse=lse[:, 3:9])
    assert slope.device_status() == (0, 0)


# ---------------------------------------------------------------- the store

@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("heads", [(1, 64, 64), (3, 192, 128), (2, 64, 128), (9, 128, 64)], ids=str)
@pytest.mark.parametrize("T", [1, 2, 3, 37, 400])
def test_write(T, heads, dtype):
    H, dqk, dv = heads
    g = torch.Generator().manual_seed(T)
    pages, page = 30, 16
    k, v = (torch.randn(T, H, d + 8, generator=g).to(dtype)[..., :d] for d in (dqk, dv))  # rows with gaps
    slots = torch.randperm(pages * page, generator=g)[:T].int()
    slots[T // 2:T // 2 + 1] = -1
    slots[:1] = pages * page if T > 2 else slots[:1]
    pools = [torch.randn(pages, H, page, d, generator=g).to(torch.bfloat16) for d in (dqk, dv)]
    weights = torch.rand(pages, H, page, generator=g)
    got = [x.cuda() for x in (*pools, weights)]
    cache = slope.KVCache(pages, page, H, dqk, dv, k=got[0], v=got[1])
    slope.kv_write(cache, *(torch.randn(T, H, d + 8, dtype=torch.float32).to(dtype).cuda()[..., :d].copy_(x)
                            for x, d in ((k, dqk), (v, dv))), slots.cuda(), weights=got[2])
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < pages * page:
            for pool, x in zip(pools, (k, v)):
                pool[s // page, :, s % page] = x[t].to(torch.bfloat16)
            weights[s // page, :, s % page] = 0
    for x, y in zip(got, (*pools, weights)):
        assert torch.equal(x.cpu(), y)


def test_write_token_major_and_one_buffer():
    """Keys and values as slices of one token-major buffer; without weights."""
    pages, page, H, d = 5, 16, 2, 64
    both = torch.zeros(pages, 2, page, H, d, dtype=torch.bfloat16, device="cuda")
    cache = slope.KVCache(pages, page, H, d, d, k=both[:, 0].transpose(1, 2), v=both[:, 1].transpose(1, 2))
    k, v = (torch.randn(20, H, d, device="cuda").to(torch.bfloat16) for _ in range(2))
    slots = torch.arange(3, 63, 3, dtype=torch.int32, device="cuda")
    slope.kv_write(cache, k, v, slots)
    flat = both.transpose(1, 2).reshape(pages * page, 2, H, d)
    assert torch.equal(flat[slots.long(), 0], k) and torch.equal(flat[slots.long(), 1], v)
    assert int((both != 0).any(-1).sum()) == 20 * 2 * H


# ---------------------------------------------------------------- weights

def weights_of(batch, pool, b):
    """[Hkv, tokens] of a sequence, out of a [pages, Hkv, page] pool."""
    t = torch.arange(batch.lens[b])
    return pool[batch.table[b].long()[t // batch.page], :, t % batch.page].t()


def check_weights(batch, got, lse, before=None, **how):
    got = got.cpu()
    touched = torch.zeros(got.shape, dtype=torch.bool)
    for b, (w, off) in enumerate(ko.token_weights(batch, lse, **how)):
        if before is not None:
            w = w + weights_of(batch, before, b).double()
        bad = (weights_of(batch, got, b).double() - w).abs() > off + 2.0 ** -23 * w.abs() + 1e-30
        assert not bad.any(), (b, bad.nonzero()[0].tolist(), float((weights_of(batch, got, b).double() - w).abs().max()))
        t = torch.arange(batch.lens[b])
        touched[batch.table[b].long()[t // batch.page], :, t % batch.page] = True
    return touched


@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("heads", HEADS, ids=str)
def test_weights(heads, lens):
    batch = ko.Batch(*LENS[lens], *heads, 16 if heads[0] % 2 else 64, seed=len(lens))
    cache, table, n, cu = on_gpu(batch)
    lse = ko.attention(batch)[1].float()
    start = torch.rand(batch.n_pages, batch.Hkv, batch.page)
    for accumulate in (False, True):
        got = start.cuda()
        assert slope.kv_attn_weights(batch.q.cuda(), cache, table, n, lse.cuda(), got, cu_q=cu,
                                     accumulate=accumulate) is got
        touched = check_weights(batch, got, lse, start if accumulate else None)
        assert torch.equal(got.cpu()[~touched], start[~touched])


@pytest.mark.parametrize("window", [1, 100, 129, 1000])
@pytest.mark.parametrize("heads", [(8, 1, 64, 64), (2, 2, 192, 128), (131, 1, 64, 64)], ids=str)
def test_weights_window(heads, window):
    batch = ko.Batch([900, 300, 1], [1, 290, 1], *heads, 16, seed=window)
    cache, table, n, cu = on_gpu(batch)
    lse = ko.attention(batch, window=window, scale=0.2)[1].float()
    got = torch.zeros(batch.n_pages, batch.Hkv, batch.page, device="cuda")
    slope.kv_attn_weights(batch.q.cuda(), cache, table, n, lse.cuda(), got, cu_q=cu, window=window, scale=0.2,
                          accumulate=False)
    check_weights(batch, got, lse, window=window, scale=0.2)
    # each row's weights are a probability distribution
    total = sum(float(weights_of(batch, got.cpu(), b).double().sum()) for b in range(3))
    assert abs(total - batch.cu[-1] * heads[0]) < 1e-3 * batch.cu[-1] * heads[0]


def test_weights_many_rows_and_sequences():
    """Pieces that are joined (few keys, many rows); more sequences than a launch takes."""
    batch = ko.Batch([700, 600], [700, 400], 16, 1, 64, 64, 64, seed=8)
    cache, table, n, cu = on_gpu(batch)
    lse = ko.attention(batch)[1].float()
    got = torch.zeros(batch.n_pages, 1, 64, device="cuda")
    for _ in range(2):
        slope.kv_attn_weights(batch.q.cuda(), cache, table, n, lse.cuda(), got, cu_q=cu)
    check_weights(batch, got / 2, lse)
    lens = [(7 * i) % 50 for i in range(1100)]
    batch = ko.Batch(lens, [1] * 1100, 4, 1, 64, 64, 16, seed=9)
    cache, table, n, _ = on_gpu(batch)
    lse = ko.attention(batch)[1].float()
    got = torch.zeros(batch.n_pages, 1, 16, device="cuda")
    slope.kv_attn_weights(batch.q.cuda(), cache, table, n, lse.cuda(), got)
    check_weights(batch, got, lse)


def test_weights_of_hidden_values():
    """What masked places hold, NaN and infinities too, reaches no weight; rows that saw nothing add nothing."""
    batch = ko.Batch([300], [60], 5, 1, 64, 64, 16, seed=10)
    cache, table, n, _ = on_gpu(batch)
    lse = ko.attention(batch)[1].float()
    q = torch.cat((batch.q, torch.full((70, 5, 64), math.nan).to(torch.bfloat16))).cuda()  # rows of no sequence
    lse_all = torch.cat((lse, torch.full((5, 70), math.nan)), 1).cuda()
    lse_all[:, 50:60] = -math.inf  # the last ten rows add nothing
    got = torch.zeros(batch.n_pages, 1, 16, device="cuda")
    slope.kv_attn_weights(q, cache, table, n, lse_all, got, cu_q=i32([0, 60]), accumulate=False)
    check_weights(batch, got, lse_all[:, :60].cpu())
    # a row that is not finite spoils the keys that it sees, and no others
    q[20] = math.inf
    slope.kv_attn_weights(q, cache, table, n, lse_all, got, cu_q=i32([0, 60]), accumulate=False)
    w = weights_of(batch, got.cpu(), 0)
    assert w[:, :261].isnan().all() and not w[:, 261:].isnan().any()


def test_weights_without_rows():
    batch = ko.Batch([40, 3], [0, 0], 4, 2, 64, 64, 16, seed=11)
    cache, table, n, cu = on_gpu(batch)
    got = torch.ones(batch.n_pages, 2, 16, device="cuda")
    q, lse = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(4, 0, device="cuda")
    slope.kv_attn_weights(q, cache, table, n, lse, got, cu_q=cu)
    assert (got == 1).all()
    slope.kv_attn_weights(q, cache, table, n, lse, got, cu_q=cu, accumulate=False)
    assert int((got == 0).sum()) == 2 * 43


# ---------------------------------------------------------------- eviction

def evict_case(lens, Hkv, dqk, dv, page, seed, ties=False):
    batch = ko.Batch(lens, [0] * len(lens), Hkv, Hkv, dqk, dv, page, seed=seed)
    g = torch.Generator().manual_seed(seed)
    w = torch.randn(batch.n_pages, Hkv, page, generator=g).exp()
    if ties:
        w = (w * 2).round() / 2
    return batch, w


def check_evict(batch, w, keep, first, recent, got, pools, out_table=None):
    """pools: keys, values, weights before and after."""
    kept, left = (x.cpu() for x in got)
    want = [x.clone() for x, _ in pools]
    assert left.tolist() == [min(n, keep) for n in batch.lens]
    for b, n in enumerate(batch.lens):
        here = weights_of(batch, w, b)
        for h in range(batch.Hkv):
            stay = ko.choose(here[h], keep, first, recent)
            assert kept[b, h].tolist() == stay + [-1] * (keep - len(stay))
            if not stay:
                continue
            old, new = torch.tensor(stay), torch.arange(len(stay))
            row, to = batch.table[b].long(), (batch.table if out_table is None else out_table)[b].long()
            for x, (before, _) in zip(want, pools):
                x[to[new // batch.page], h, new % batch.page] = before[row[old // batch.page], h, old % batch.page]
    for x, (_, after) in zip(want, pools):
        assert torch.equal(x.view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32),
                           after.cpu().view(torch.int16 if x.dtype == torch.bfloat16 else torch.int32))


EVICT = [
    ([1, 2, 0, 40], 3, 0, 0),
    ([100, 33, 32, 31], 32, 0, 0),
    ([100, 33], 32, 4, 8),
    ([700, 64, 500], 64, 0, 64),
    ([700], 64, 64, 0),
    ([700], 64, 30, 34),
    ([3000, 2999], 1500, 1, 16),
    ([20000, 100, 9000], 5000, 4, 512),
    ([20000], 19999, 0, 0),
    ([20000], 1, 0, 0),
]


@pytest.mark.parametrize("ties", [False, True])
@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("case", EVICT, ids=str)
def test_evict(case, apart, ties):
    lens, keep, first, recent = case
    heads = [(2, 64, 64), (1, 192, 128), (3, 128, 64), (1, 64, 128)][len(lens) % 4 if sum(lens) < 5000 else 0]
    batch, w = evict_case(lens, *heads, 16 if keep % 2 else 64, seed=keep, ties=ties)
    out_table = None
    if apart:  # into pages of their own
        need = -(-keep // batch.page)
        more = len(lens) * need
        out_table = (batch.n_pages + torch.randperm(more)).view(len(lens), need).int()
        grow = lambda x: torch.cat((x, torch.full((more, *x.shape[1:]), 7.0, dtype=x.dtype)))  # noqa: E731
        batch.k, batch.v, w = grow(batch.k), grow(batch.v), grow(w)
        batch.n_pages += more
    cache, table, n, _ = on_gpu(batch)
    wg = w.cuda()
    got = slope.kv_evict(cache, wg, table, n, keep, first=first, recent=recent,
                         out_table=None if out_table is None else out_table.cuda())
    check_evict(batch, w, keep, first, recent, got, [(batch.k, cache.k), (batch.v, cache.v), (w, wg)], out_table)


def test_evict_special_weights():
    """NaN below -inf, -0 as 0, equal infinities by position."""
    batch, w = evict_case([64], 1, 64, 64, 16, seed=1)
    vals = [math.nan, -math.inf, math.inf, 0.0, -0.0, -1.0, 1e-45, 3e38]
    here = torch.tensor([vals[i % 8] for i in range(64)])
    for t in range(64):
        w[int(batch.table[0, t // 16]), 0, t % 16] = here[t]
    for keep in (1, 8, 9, 16, 20, 30, 35, 55, 60):
        cache, table, n, _ = on_gpu(batch)
        wg = w.cuda()
        got = slope.kv_evict(cache, wg, table, n, keep)
        check_evict(batch, w, keep, 0, 0, got, [(batch.k, cache.k), (batch.v, cache.v), (w, wg)])


def test_evict_missing_pages():
    """Tokens without a page are the last to be chosen; rows there are neither read nor written."""
    batch, w = evict_case([300, 300], 2, 64, 64, 16, seed=2)
    cache, table, n, _ = on_gpu(batch)
    table[0, 2] = -1
    table[1, 1] = batch.n_pages
    wg = w.cuda()
    kept, left = slope.kv_evict(cache, wg, table, n, 270, first=3, recent=20)
    kept = kept.cpu()
    assert left.tolist() == [270, 270] and slope.device_status() == (0, 0)
    for b, e in ((0, 2), (1, 1)):
        here = weights_of(batch, w, b).clone()
        here[:, 16 * e:16 * e + 16] = math.nan  # no number in these cases is a NaN
        for h in range(2):
            assert kept[b, h].tolist() == ko.choose(here[h], 270, 3, 20)


def test_evict_lengths_in_place():
    batch, w = evict_case([50, 7, 30], 4, 64, 64, 16, seed=3)
    cache, table, n, _ = on_gpu(batch)
    wg = w.cuda()
    got = slope.kv_evict(cache, wg, table, n, 20, out_lens=n)
    assert got[1] is n
    check_evict(batch, w, 20, 0, 0, got, [(batch.k, cache.k), (batch.v, cache.v), (w, wg)])


# ---------------------------------------------------------------- as a server runs them

def test_a_prompt_in_chunks_then_decoding_with_eviction():
    """Two prompts come in chunks beside one another's decoding; then each keeps half of its tokens, and decoding goes
    on over those."""
    Hq, Hkv, d, page = 8, 2, 64, 16
    g = torch.Generator().manual_seed(12)
    rnd = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)  # noqa: E731
    total = [330, 150]
    q, k, v = ([rnd(n, h, d) for n in total] for h in (Hq, Hkv, Hkv))
    cache = slope.KVCache(60, page, Hkv, d, d)
    cache.k.fill_(math.nan), cache.v.fill_(math.nan)
    weights = torch.full((60, Hkv, page), math.nan, device="cuda")
    table = torch.randperm(60, generator=g)[:50].view(2, 25).int()
    done, sums = [0, 0], [torch.zeros(Hkv, n, dtype=torch.float64) for n in total]
    for step in ((200, 120), (129, 1), (1, 29)):
        now = [x + s for x, s in zip(done, step)]
        rows = [slice(a, e) for a, e in zip(done, now)]
        slots = torch.cat([table[b].long()[torch.arange(r.start, r.stop) // page] * page + torch.arange(r.start, r.stop) % page
                           for b, r in enumerate(rows)]).int()
        pick = lambda x: torch.cat([y[r] for y, r in zip(x, rows)]).cuda()  # noqa: E731
        slope.kv_write(cache, pick(k), pick(v), slots.cuda(), weights=weights)
        how = dict(cu_q=i32([0, step[0], sum(step)]))
        out, lse = slope.kv_attn(pick(q), cache, table.cuda(), i32(now), **how)
        slope.kv_attn_weights(pick(q), cache, table.cuda(), i32(now), lse, weights, **how)
        batch = ko.Batch([0, 0], [0, 0], Hq, Hkv, d, d, page)
        batch.lens, batch.new, batch.cu = now, list(step), [0, step[0], sum(step)]
        batch.q, batch.keys, batch.values = pick(q).cpu(), [x[:n] for x, n in zip(k, now)], [x[:n] for x, n in zip(v, now)]
        check(out, lse, ko.attention(batch))
        for b, (w, _) in enumerate(ko.token_weights(batch, lse.cpu())):
            sums[b][:, :now[b]] += w
        done = now
    t = [torch.arange(n) for n in total]
    have = [weights.cpu()[table[b].long()[t[b] // page], :, t[b] % page].t() for b in range(2)]
    for x, y in zip(have, sums):
        assert (x.double() - y).abs().max() <= 2.0 ** -14 * y.max()
    kept, left = slope.kv_evict(cache, weights, table.cuda(), i32(total), 160, first=2, recent=30)
    assert left.tolist() == [160, 150]
    # the next token of each, over the tokens that stayed
    nq, nk, nv = (rnd(2, h, d) for h in (Hq, Hkv, Hkv))
    slope.kv_write(cache, nk.cuda(), nv.cuda(), i32([int(table[b, n // page]) * page + n % page for b, n in enumerate(left.tolist())]))
    out, lse = slope.kv_attn(nq.cuda(), cache, table.cuda(), left + 1)
    for b in range(2):
        for h in range(Hkv):
            m = int(left[b])
            stay = kept[b, h].cpu().long()[:m]
            assert stay.tolist() == ko.choose(have[b][h], 160, 2, 30)
            kk, vv = (torch.cat((x[b][stay, h], y[b:b + 1, h])).double() for x, y in ((k, nk), (v, nv)))
            for i in range(4):
                s = kk @ nq[b, 4 * h + i].double() * d ** -0.5
                p = torch.softmax(s, 0)
                tol = (2.0 ** -8 + 2.0 ** -13) * (p @ vv.abs()) + 2.0 ** -8 * (p @ vv).abs()
                assert ((out[b, 4 * h + i].cpu().double() - p @ vv).abs() <= tol).all()
