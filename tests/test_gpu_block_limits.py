"""Products at the documented limits of their sizes."""
import pytest
import torch

from tests import blockkit as kit
from tests.routekit import log

pytestmark = pytest.mark.gpu

block = pytest.importorskip("latent_projection_top_amd.block")

BF = torch.bfloat16


def test_padded_copy_of_the_most_rows():
    """2^20 rows of 32761 inputs: their padded copy has 2^32 pieces of eight
    values, more than one launch has threads. x and the copy take 69 GB each.
    All rows are zero but for sampled ones, on both sides of the middle."""
    rows, k, n = 1 << 20, 32761, 8
    if torch.cuda.mem_get_info()[0] < 160 << 30:
        pytest.skip("needs 160 GB of free device memory")
    log(f"linear {rows}x{k}x{n}")
    at = torch.tensor([0, 1, 12345, rows // 2 - 1, rows // 2, rows - 2, rows - 1], device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.zeros(rows, k, dtype=BF, device="cuda")
    x[at] = torch.randn(len(at), k, generator=gen, device="cuda").to(BF)
    w = (torch.randn(k, n, generator=gen, device="cuda") * k ** -0.5).to(BF)
    plan = block.LinearPlan(rows, k, n)
    ws = plan.new_workspace()
    y = torch.full((rows, n), float("nan"), dtype=BF, device="cuda")
    try:
        block.linear(plan, x, w, y, ws)
        torch.cuda.synchronize()
        ref = x[at].double() @ w.double()
        kit.check(y[at], ref, (k + 8) * kit.E * (x[at].double().abs() @ w.double().abs()), ref.abs(), BF, "y")
        y[at] = 0
        assert int((y != 0).sum()) == 0
    finally:
        del x, ws
        torch.cuda.empty_cache()
