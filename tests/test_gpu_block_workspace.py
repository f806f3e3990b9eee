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
