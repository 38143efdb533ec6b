"""The counters that recorded launches of the calls on the 16-bit paged cache claim their work from."""
import time

import pytest
import torch

import kv_oracle as ko
import ring_attention_slope_gb300 as slope
from test_gpu_kv import check, on_gpu

pytestmark = pytest.mark.gpu

COUNTERS = 65536  # SLOPE_KV_COUNTERS


@pytest.fixture(scope="module", autouse=True)
def _built():
    slope.build()
    slope.load()
    assert slope.device_status() == (0, 0)
    yield
    torch.cuda.synchronize()
    assert slope.device_status() == (0, 0)


class Call:
    """A call on given outputs and workspace, and how often its result was another one."""

    def __init__(self, lens, seed):
        batch = ko.Batch(lens, [1] * len(lens), 16, 2, 64, 64, 64, seed=seed)
        self.cache, self.table, self.n, _ = on_gpu(batch)
        self.q = batch.q.cuda()
        self.work = torch.empty(slope.kv_attn_workspace_size(len(lens), 16, self.cache, 1), dtype=torch.uint8, device="cuda")
        self.out = torch.zeros(len(lens), 16, 64, device="cuda")
        self()
        check(self.out, slope.kv_attn(self.q, self.cache, self.table, self.n)[1], ko.attention(batch))
        self.want, self.bad = self.out.clone(), torch.zeros((), dtype=torch.int64, device="cuda")
        torch.cuda.synchronize()

    def __call__(self, stream=None):
        slope.kv_attn(self.q, self.cache, self.table, self.n, out=self.out, want_lse=False, workspace=self.work, stream=stream)

    def look(self):
        self.bad.add_((self.out != self.want).sum())
        self.out.zero_()

    def recorded(self, times=1, look=True):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(times):
                self()
            if look:
                self.look()
        return graph


def test_a_graph_beside_more_calls_than_there_are_counters():
    """Calls on streams go once round their counters while a recorded call runs."""
    long, short = Call([40000, 30000, 35000], 1), Call([700], 2)
    graph, side = long.recorded(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for i in range(COUNTERS + 200):
        if i % 4 == 0:
            graph.replay()
        short(side)
        if i % 64 == 63:
            with torch.cuda.stream(side):
                short.look()
        if i % 1024 == 1023:
            torch.cuda.synchronize()
            assert int(long.bad) == 0 and int(short.bad) == 0, i
    torch.cuda.synchronize()
    assert int(long.bad) == 0 and int(short.bad) == 0


def test_counters_of_graphs_that_are_gone_come_again():
    """A recorded call keeps its counter while others are recorded and dropped, more of them than there are counters; where
    all are kept, a further recording is refused; and they are there again once the graphs are gone."""
    one, two = Call([40000, 30000], 3), Call([35000, 20000, 9000], 4)
    first = one.recorded()
    for _ in range(COUNTERS // 1024 + 2):
        two.recorded(1024, look=False)
    second = two.recorded()

    def together(*graphs):
        streams = [torch.cuda.Stream() for _ in graphs]
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for _ in range(100):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        assert int(one.bad) == 0 and int(two.bad) == 0

    together(first, second)
    kept = []
    with pytest.raises(slope.SlopeError):
        for _ in range(COUNTERS // 1024 + 2):
            kept.append(two.recorded(1024, look=False))
    assert len(kept) <= COUNTERS // 1024
    together(first, second)
    two()  # calls on streams have counters of their own
    two.look()
    kept.clear()
    for _ in range(100):  # (a graph's end is told by another thread)
        try:
            third = two.recorded()
            break
        except slope.SlopeError:
            time.sleep(0.1)
    together(first, third)
