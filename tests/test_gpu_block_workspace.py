"""Workspaces as a C caller sees them: the size that the library names is the
size that its calls accept."""
import pytest
import torch

from tests import blockkit as kit
from tests.routekit import log

pytestmark = pytest.mark.gpu

block = pytest.importorskip("latent_projection_top_amd.block")
from latent_projection_top_amd import route  # noqa: E402

BF, FP = torch.bfloat16, torch.float32


@pytest.mark.parametrize("width,dtype", [(64, BF), (7168, BF), (16384, BF), (20000, BF), (8192, FP), (9001, FP)])
def test_norm_backward_takes_the_size_it_asks_for(width, dtype):
    """Rows that registers hold and rows that they do not: exactly
    block_norm_workspace_bytes bytes, allocated as a C program would."""
    log(f"norm workspace {width} {dtype}")
    c = kit.NormCase(5, width, dtype, seed=1)
    plan = block.NormPlan(5, width, dtype=dtype)
    size = int(block.LIB.block_norm_workspace_bytes(plan.handle))
    assert plan.workspace_bytes == size
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    dx = torch.empty_like(c.x)
    m, r = torch.empty(5, device="cuda"), torch.empty(5, device="cuda")
    dw = torch.empty(width, device="cuda")
    block.layer_norm(plan, c.x, c.weight, c.bias, dx, m, r)
    st = block.LIB.block_norm_backward(
        plan.handle, c.dy.data_ptr(), width, c.x.data_ptr(), width, c.weight.data_ptr(), m.data_ptr(), r.data_ptr(),
        dx.data_ptr(), width, dw.data_ptr(), None, ws.data_ptr() or None, 5,
        torch.cuda.current_stream().cuda_stream or None)
    torch.cuda.synchronize()
    assert st == route.OK
    ref = c.reference()
    kit.check(dx, *ref["dx"], dtype, "dx")
    kit.check(dw, *ref["dweight"], FP, "dweight")


def test_split_sums_take_what_a_plan_can_use():
    """A decode plan's workspace holds its counters, the split sums of at most
    a block per CU (four splits of 56 column tiles) and a copy of x; a training
    plan of few rows also 64 column tiles' worth for dx (two splits of 32)."""
    pad = 8 * 256
    plan = block.LinearPlan(8, 2048, 7168)
    assert plan.workspace_bytes <= block.WORKSPACE_ZEROED + 4 * 8 * 7168 * 4 + 8 * 2048 * 2 + pad
    # dw has one step of 32 rows: never split
    plan = block.LinearPlan(20, 7168, 2048, training=True)
    splits = max(16 * 20 * 2048, 2 * 20 * 7168) * 4  # forward: 16 column tiles; dx: 112
    rest = 20 * 2048 * 2 + 20 * 2048 * 4 + 20 * 7168 * 2  # dz, the rows of dbias's sums, x
    assert plan.workspace_bytes <= block.WORKSPACE_ZEROED + splits + rest + pad


SHAPES = [(1, 3584, 2048), (5, 777, 1001), (20, 7168, 2048), (64, 4096, 512), (333, 1001, 777), (700, 512, 128)]


@pytest.mark.parametrize("rows,k,n", SHAPES)
def test_only_the_counters_have_to_be_zero(rows, k, n):
    """The same bits from a workspace whose other bytes are all ones (NaN in
    every type) as from one of zeros."""
    log(f"workspace of ones {rows}x{k}x{n}")
    g = kit.GatedCase(rows, k, n, "silu", BF, seed=1)
    c = kit.LinearCase(rows, k, n, "gelu", BF, seed=2)
    norm = kit.NormCase(rows, n, BF, seed=3)
    plans = (block.GatedPlan(rows, k, n, training=True), block.LinearPlan(rows, k, n, "gelu", training=True),
             block.NormPlan(rows, n))
    results = []
    for fill in (0, 255):
        gw, lw, nw = (torch.full((p.workspace_bytes,), fill, dtype=torch.uint8, device="cuda") for p in plans)
        for ws in (gw, lw):
            ws[:block.WORKSPACE_ZEROED] = 0
        o = {i: torch.empty(rows, n, dtype=BF, device="cuda") for i in ("h", "dg", "du", "y", "s", "ny", "ndx")}
        o.update({i: torch.empty(k, n, dtype=BF, device="cuda") for i in ("wg", "wu", "w")})
        o.update({i: torch.empty(rows, k, dtype=BF, device="cuda") for i in ("x1", "x2")})
        o["b"] = torch.empty(n, dtype=BF, device="cuda")
        o.update({i: torch.empty(rows, device="cuda") for i in ("m", "r")})
        o.update({i: torch.empty(n, device="cuda") for i in ("nw", "nb")})
        block.gated(plans[0], g.x, g.wg, g.wu, o["h"], gw, o["dg"], o["du"])
        block.gated_backward(plans[0], g.dh, g.x, g.wg, g.wu, o["dg"], o["du"], o["x1"], o["wg"], o["wu"], gw)
        block.linear(plans[1], c.x, c.w, o["y"], lw, c.bias, c.residual, o["s"])
        block.linear_backward(plans[1], c.dy, c.x, c.w, o["s"], o["x2"], o["w"], o["b"], lw)
        block.layer_norm(plans[2], norm.x, norm.weight, norm.bias, o["ny"], o["m"], o["r"])
        block.layer_norm_backward(plans[2], norm.dy, norm.x, norm.weight, o["m"], o["r"], o["ndx"], o["nw"], o["nb"],
                                  nw)
        torch.cuda.synchronize()
        results.append(o)
    for name, t in results[0].items():
        assert bool(torch.isfinite(t).all()) and torch.equal(t, results[1][name]), name
