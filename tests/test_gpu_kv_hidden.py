"""What rows and keys that do not count may hold in the calls on the 16-bit paged cache."""
import math

import pytest
import torch

import kv_oracle as ko
import ring_attention_slope_gb300 as slope
from test_gpu_kv import check_weights, i32, on_gpu, weights_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    slope.build()
    slope.load()
    assert slope.device_status() == (0, 0)
    yield
    torch.cuda.synchronize()
    assert slope.device_status() == (0, 0)


@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("lens, new, heads", [
    ([300], [60], (5, 1, 64, 64)),       # few row tiles, of 125 rows
    ([700, 90], [1, 1], (8, 1, 64, 64)),    # single tokens
    ([1500, 640], [700, 200], (8, 2, 64, 64)),  # many
    ([900], [300], (4, 2, 128, 128)),
    ([600], [9], (131, 1, 64, 64)),      # a group in parts
], ids=str)
def test_a_row_whose_lse_is_minus_infinity_adds_nothing(lens, new, heads, what):
    """Whatever its query holds."""
    batch = ko.Batch(lens, new, *heads, 16, seed=sum(lens))
    cache, table, n, cu = on_gpu(batch)
    lse = ko.attention(batch)[1].float()
    T = batch.cu[-1]
    out = torch.zeros(T, dtype=torch.bool)
    out[::3] = True
    out[-1] = True
    rows = torch.nonzero(out)[:, 0]
    lse[:, rows] = -math.inf
    lse[::2, 0] = -math.inf  # of some heads only
    q = batch.q.clone()
    q[rows] = what
    q[0, ::2] = what
    batch.q[rows] = 0  # the oracle's rows, which count for nothing
    batch.q[0, ::2] = 0
    got = torch.full((batch.n_pages, heads[1], 16), 7.0, device="cuda")
    slope.kv_attn_weights(q.cuda(), cache, table, n, lse.cuda(), got, cu_q=cu, accumulate=False)
    assert not any(weights_of(batch, got.cpu(), b).isnan().any() for b in range(len(lens)))
    check_weights(batch, got, lse)


@pytest.mark.parametrize("heads", [(8, 1, 64, 64), (2, 2, 192, 128)], ids=str)
def test_scores_that_are_all_minus_infinity(heads):
    """A row of them gives 0 and -inf, as one that sees nothing, alone or joined from pieces; and adds no weight."""
    H, Hkv, dqk, dv = heads
    batch = ko.Batch([3000, 60], [1, 3], *heads, 16, seed=12)
    q, k = torch.zeros_like(batch.q), batch.k.clone()
    q[..., 0] = 1.0
    k[..., 0] = -math.inf  # all keys: every score is -inf
    cache = slope.KVCache(batch.n_pages, 16, Hkv, dqk, dv, k=k.nan_to_num(nan=0.0, neginf=-math.inf).cuda(), v=batch.v.cuda())
    table, n, cu = batch.table.cuda(), i32(batch.lens), i32(batch.cu)
    out, lse = slope.kv_attn(q.cuda(), cache, table, n, cu_q=cu)
    assert (out == 0).all() and (lse == -math.inf).all()
    w = torch.full((batch.n_pages, Hkv, 16), 2.0, device="cuda")
    slope.kv_attn_weights(q.cuda(), cache, table, n, lse, w, cu_q=cu)
    assert (w == 2).all()


def test_a_key_that_is_not_finite_spoils_its_own_weight_alone():
    batch = ko.Batch([500], [40], 5, 1, 64, 64, 16, seed=13)
    lse = ko.attention(batch)[1].float()
    page, at = int(batch.table[0, 3]), 5
    batch.k[page, 0, at] = math.nan
    cache, table, n, cu = on_gpu(batch)
    got = torch.zeros(batch.n_pages, 1, 16, device="cuda")
    slope.kv_attn_weights(batch.q.cuda(), cache, table, n, lse.cuda(), got, cu_q=cu)
    assert got[page, 0, at].isnan()
    got[page, 0, at] = 0
    batch.keys[0][3 * 16 + at] = -1e4  # (in the oracle a key without weight)
    w, off = ko.token_weights(batch, lse)[0]
    have = weights_of(batch, got.cpu(), 0)
    keep = torch.arange(500) != 3 * 16 + at
    assert ((have.double() - w).abs() <= off + 2.0 ** -23 * w)[:, keep].all()
