"""Several captured serving steps of one cache."""

import pytest
import torch

from quantized_paged_kv_tile_b200 import build, kvq
from quantized_paged_kv_tile_b200.paged import DecodeStepGraph

from test_gpu_evict import config, filled, rows

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()
    return kvq.load_library()


@pytest.mark.parametrize("track", [True, False])
def test_a_graph_keeps_the_workspace_it_recorded(track):
    """A second graph with more splits needs a larger workspace; the first one's
    replays still run in the buffer that the first one recorded."""
    cfg = config()
    cache, twin = (filled(cfg, [3000, 700], 61, track=track, extra=512) for _ in range(2))
    kept = cache.workspace
    small = DecodeStepGraph(cache, num_splits=1)
    mid = DecodeStepGraph(cache, num_splits=900)
    large = DecodeStepGraph(cache, num_splits=3000)
    assert cache.workspace is kept
    assert large.workspace.numel() > mid.workspace.numel() > kept.numel()
    assert len({g.workspace.data_ptr() for g in (small, mid, large)}) == 3
    sizes = [kept.numel(), mid.workspace.numel(), large.workspace.numel()]
    others = [torch.full((n,), 123, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    for i, graph in enumerate([small, large, mid, small, mid]):
        q, k, v = rows(cfg, 2, 600 + i)
        graph.new_k.copy_(k)
        graph.new_v.copy_(v)
        graph.q.copy_(q)
        out = graph.replay()
        twin.append(k, v)
        assert torch.equal(out, twin.decode(q, num_splits=graph.num_splits))
        if track:
            assert torch.equal(cache.mass, twin.mass)
    assert all(bool((x == 123).all()) for x in others)
    assert cache.status() == 0
