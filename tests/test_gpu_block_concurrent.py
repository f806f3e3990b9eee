"""Calls of the few-row products that overlap in time on two streams, in the
shapes whose split sums are joined by the last block of each column tile: the
arrival counters and the exchange of sums between blocks of one launch are what
concurrent calls could disturb."""
import pytest
import torch

from tests import blockkit as kit
from tests.routekit import log

pytestmark = pytest.mark.gpu

block = pytest.importorskip("latent_projection_top_amd.block")

BF = torch.bfloat16
INPUTS, CALLS = 4, 24
COUNTERS = 131072  # bytes at the start of a workspace


def make(op, rows, k, n, seed):
    """A plan's call as call(input, output, workspace, stream), its inputs and
    the shape of its output. Each stream has its own weights."""
    if op == "gated":
        cases = [kit.GatedCase(rows, k, n, "silu", BF, seed=100 * seed + i) for i in range(INPUTS)]
        plan, c = block.GatedPlan(rows, k, n), cases[0]
        return (plan, [i.x for i in cases], n,
                lambda x, out, ws, s: block.gated(plan, x, c.wg, c.wu, out, ws, stream=s))
    cases = [kit.LinearCase(rows, k, n, "none", BF, seed=100 * seed + i) for i in range(INPUTS)]
    plan, c = block.LinearPlan(rows, k, n, training=op == "dx"), cases[0]
    if op == "linear":
        return (plan, [i.x for i in cases], n,
                lambda x, out, ws, s: block.linear(plan, x, c.w, out, ws, bias=c.bias, residual=c.residual, stream=s))
    return (plan, [i.dy for i in cases], k,
            lambda dy, out, ws, s: block.linear_backward(plan, dy, c.x, c.w, None, out, None, None, ws, stream=s))


@pytest.mark.parametrize("op,rows,k,n", [("gated", 1, 3584, 2048), ("gated", 4, 3584, 2048), ("gated", 3, 1001, 333),
                                         ("linear", 8, 2048, 7168), ("linear", 1, 7168, 520), ("dx", 8, 2048, 7168),
                                         ("dx", 5, 777, 2001)])
def test_two_streams_with_changing_inputs(op, rows, k, n):
    """Two streams, a workspace each, the inputs different from call to call:
    every output has the bits of the same call alone, and the counters are zero
    afterwards."""
    log(f"two streams {op} {rows}x{k}x{n}")
    sides = [make(op, rows, k, n, seed) for seed in (1, 2)]
    want = []
    for plan, inputs, width, call in sides:
        ws = plan.new_workspace()
        want.append([torch.empty(rows, width, dtype=BF, device="cuda") for _ in inputs])
        for x, out in zip(inputs, want[-1]):
            call(x, out, ws, None)
    torch.cuda.synchronize()
    assert not torch.equal(want[0][0], want[0][1])
    spaces = [side[0].new_workspace() for side in sides]
    outs = [[torch.empty(rows, side[2], dtype=BF, device="cuda") for _ in range(CALLS)] for side in sides]
    streams = [torch.cuda.Stream() for _ in sides]
    torch.cuda.synchronize()
    for i in range(CALLS):
        for (plan, inputs, width, call), ws, out, s in zip(sides, spaces, outs, streams):
            call(inputs[i % INPUTS], out[i], ws, s)
    torch.cuda.synchronize()
    for w, out, ws in zip(want, outs, spaces):
        for i in range(CALLS):
            assert torch.equal(out[i], w[i % INPUTS]), i
        assert not ws[:COUNTERS].any()
