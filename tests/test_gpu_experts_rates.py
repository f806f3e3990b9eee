"""Rates that a type must not lose."""
import pytest
import torch

from tests.routekit import log

pytestmark = pytest.mark.gpu

experts = pytest.importorskip("latent_projection_top_amd.experts")


def least_time(call, passes=8):
    """The least of some passes' times in a graph, ms."""
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
        call()
    times = []
    for _ in range(passes):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        graph.replay()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    return min(times)


def test_gather_of_wide_types():
    """FP32 rows are twice BF16's bytes, both bound by memory: 2.2 times their
    time as it is, 4.7 where halves of lines go to memory apart."""
    log("gather rates")
    rows, topk, width = 2048, 16, 3584
    place = torch.randperm(rows * topk, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(rows, topk)
    place = place.cuda()
    times = {}
    for dtype in (torch.bfloat16, torch.float32):
        x = torch.ones(rows, width, dtype=dtype, device="cuda")
        xs = torch.empty(rows * topk, width, dtype=dtype, device="cuda")
        plan = experts.CombinePlan(rows, topk, width, dtype=dtype)
        times[dtype] = least_time(lambda: experts.gather(plan, x, place, xs))
    assert times[torch.float32] <= 3.3 * times[torch.bfloat16], times
