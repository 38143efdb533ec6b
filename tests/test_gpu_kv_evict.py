"""Eviction from the 16-bit paged cache where its work takes other ways than in a short batch: many sequences, long ones."""
import pytest
import torch

import ring_attention_slope_gb300 as slope
from test_gpu_kv import check_evict, evict_case, i32, on_gpu

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
