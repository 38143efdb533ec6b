"""Eviction from the 16-bit paged cache where its work takes other ways than in a short batch: many sequences, long ones."""
import math

import pytest
import torch

import kv_oracle as ko
import ring_attention_slope_gb300 as slope
from test_gpu_kv import check_evict, evict_case, on_gpu, weights_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    slope.build()
    slope.load()
    assert slope.device_status() == (0, 0)
    yield
    torch.cuda.synchronize()
    assert slope.device_status() == (0, 0)


def test_evict_tens_of_thousands_of_sequences():
    """More launches than 64: each has a ticket of its own."""
    lens = [(5 * i) % 23 + 1 for i in range(32768 + 300)]
    batch, w = evict_case(lens, 1, 64, 64, 16, seed=31)
    cache, table, n, _ = on_gpu(batch)
    wg = w.cuda()
    got = slope.kv_evict(cache, wg, table, n, 6, first=1, recent=2)
    check_evict(batch, w, 6, 1, 2, got, [(batch.k, cache.k), (batch.v, cache.v), (w, wg)])


def grown(batch, w, out_pages):
    """Room for out_pages pages behind a case's own, and a table of those."""
    grow = lambda x: torch.cat((x, torch.full((out_pages.numel(), *x.shape[1:]), 7.0, dtype=x.dtype)))  # noqa: E731
    batch.k, batch.v, w = grow(batch.k), grow(batch.v), grow(w)
    table = (batch.n_pages + out_pages).int()
    batch.n_pages += out_pages.numel()
    return w, table


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("lens, keep, first, recent, heads", [
    ([1 + (13 * i) % 70 for i in range(1100)], 20, 2, 5, (2, 64, 64)),   # three launches
    ([40000, 37, 33000], 9000, 4, 100, (2, 64, 64)),                     # clusters of eight
    ([40000], 39999, 0, 0, (1, 128, 128)),
    ([340000, 20], 50001, 16, 3000, (1, 64, 64)),                        # more keys than a CTA holds
    ([340000], 2, 0, 1, (1, 64, 64)),
], ids=["many", "long", "all_but_one", "longer", "two"])
def test_evict_many_and_long(lens, keep, first, recent, heads, apart):
    batch, w = evict_case(lens, *heads, 64, seed=keep, ties=keep == 9000)
    out_table = None
    if apart:
        need = -(-keep // 64)
        order = torch.randperm(len(lens) * need, generator=torch.Generator().manual_seed(1)).view(len(lens), need)
        w, out_table = grown(batch, w, order)
    cache, table, n, _ = on_gpu(batch)
    wg = w.cuda()
    got = slope.kv_evict(cache, wg, table, n, keep, first=first, recent=recent,
                         out_table=None if out_table is None else out_table.cuda())
    check_evict(batch, w, keep, first, recent, got, [(batch.k, cache.k), (batch.v, cache.v), (w, wg)], out_table)


@pytest.mark.parametrize("apart", [False, True])
def test_evict_leaves_pages_that_are_missing_alone(apart):
    """Where a token's old or new page is missing, nothing is read or written; all else moves as it should."""
    batch, w = evict_case([300, 300], 2, 64, 64, 16, seed=2)
    out_table = None
    if apart:
        w, out_table = grown(batch, w, torch.randperm(34).view(2, 17))
    cache, table, n, _ = on_gpu(batch)
    wg = w.cuda()
    before = [x.clone() for x in (batch.k, batch.v, w)]
    gone = {(0, 2): -1, (1, 1): batch.n_pages, (1, 18): 2 ** 31 - 1}
    for (b, e), p in gone.items():
        table[b, e] = p
    to_table = table.clone() if out_table is None else out_table.cuda()
    if apart:
        to_table[0, 5] = -1
    keep, first, recent = 270, 3, 20
    kept, left = slope.kv_evict(cache, wg, table, n, keep, first=first, recent=recent, out_table=to_table if apart else None)
    kept = kept.cpu()
    assert left.tolist() == [270, 270] and slope.device_status() == (0, 0)
    want = [x.clone() for x in before]
    rows, to = table.cpu().long(), to_table.cpu().long()
    for b in range(2):
        here = weights_of(batch, w, b).clone()
        for e in [e for c, e in gone if c == b]:
            here[:, 16 * e:16 * e + 16] = math.nan  # no number in these cases is a NaN
        for h in range(2):
            stay = ko.choose(here[h], keep, first, recent)
            assert kept[b, h].tolist() == stay
            old, new = torch.tensor(stay), torch.arange(keep)
            src, dst = rows[b][old // 16], to[b][new // 16]
            there = (src >= 0) & (src < batch.n_pages) & (dst >= 0) & (dst < batch.n_pages)
            assert not there.all()
            old, new, src, dst = (x[there] for x in (old, new, src, dst))
            for x, y in zip(want, before):
                x[dst, h, new % 16] = y[src, h, old % 16]
    for x, y in zip(want, (cache.k, cache.v, wg)):
        kind = torch.int16 if x.dtype == torch.bfloat16 else torch.int32
        assert torch.equal(x.view(kind), y.cpu().view(kind))


def test_evict_sequences_that_share_a_prefix():
    """Two sequences over the same pages, each into pages of its own."""
    batch, w = evict_case([200, 90, 200], 2, 64, 128, 16, seed=5)
    batch.table[2, :10] = batch.table[0, :10]
    batch.table[1] = batch.table[0]
    w, out_table = grown(batch, w, torch.randperm(15).view(3, 5))
    cache, table, n, _ = on_gpu(batch)
    wg = w.cuda()
    got = slope.kv_evict(cache, wg, table, n, 70, first=1, recent=8, out_table=out_table.cuda())
    check_evict(batch, w, 70, 1, 8, got, [(batch.k, cache.k), (batch.v, cache.v), (w, wg)], out_table)
