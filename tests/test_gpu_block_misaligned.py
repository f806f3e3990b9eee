"""Weights whose rows are a multiple of 8 long at an address that is no multiple
of 16 (the 64 x 64 kernel, forward and dx), with x and the gradients aligned or
not (dw always takes the tile kernel), in both types, against FP64."""
import pytest
import torch

from tests import blockkit as kit
from tests.routekit import log

pytestmark = pytest.mark.gpu

block = pytest.importorskip("latent_projection_top_amd.block")

BF, HF = torch.bfloat16, torch.float16


def shifted(w, offset):
    buf = torch.empty(offset + w.numel(), dtype=w.dtype, device="cuda")
    buf[offset:].copy_(w.flatten())
    return buf[offset:].view_as(w)


def nan(*shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


@pytest.mark.parametrize("dtype", (BF, HF))
@pytest.mark.parametrize("rows,k,n,offset,odd_rows", [(33, 8, 64, 1, False), (40, 264, 72, 4, True), (129, 101, 136, 2, False),
                                                     (300, 264, 520, 7, True), (300, 520, 264, 4, False)])
def test_products(rows, k, n, offset, odd_rows, dtype):
    log(f"misaligned {rows}x{k}x{n} +{offset} {dtype}")
    xs, ys = (k + 3, n + 5) if odd_rows else (0, 0)
    g = kit.GatedCase(rows, k, n, "silu", dtype, seed=1, xs=xs, hs=ys)
    g.wg, g.wu = shifted(g.wg, offset), shifted(g.wu, offset)
    c = kit.LinearCase(rows, k, n, "gelu_tanh", dtype, seed=2, xs=xs, ys=ys)
    c.w = shifted(c.w, offset)
    assert g.wg.data_ptr() % 16 != 0 and c.w.data_ptr() % 16 != 0
    plan = block.GatedPlan(rows, k, n, "silu", dtype, training=True)
    ws = plan.new_workspace()
    out = {i: nan(rows, n, dtype=dtype) for i in ("h", "d_gate", "d_up")}
    out.update(dx=nan(rows, k, dtype=dtype), dw_gate=nan(k, n, dtype=dtype), dw_up=nan(k, n, dtype=dtype))
    block.gated(plan, g.x, g.wg, g.wu, out["h"], ws, out["d_gate"], out["d_up"])
    block.gated_backward(plan, g.dh, g.x, g.wg, g.wu, out["d_gate"], out["d_up"], out["dx"], out["dw_gate"],
                         out["dw_up"], ws)
    torch.cuda.synchronize()
    ref = g.reference()
    for name, t in out.items():
        kit.check(t, *ref[name], dtype, name)
    plan = block.LinearPlan(rows, k, n, "gelu_tanh", dtype, training=True)
    ws = plan.new_workspace()
    out = {"y": nan(rows, n, dtype=dtype), "slope": nan(rows, n, dtype=dtype), "dx": nan(rows, k, dtype=dtype),
           "dw": nan(k, n, dtype=dtype), "dbias": nan(n, dtype=dtype)}
    block.linear(plan, c.x, c.w, out["y"], ws, c.bias, c.residual, out["slope"])
    block.linear_backward(plan, c.dy, c.x, c.w, out["slope"], out["dx"], out["dw"], out["dbias"], ws)
    torch.cuda.synchronize()
    ref = c.reference()
    for name, t in out.items():
        kit.check(t, *ref[name], dtype, name)
