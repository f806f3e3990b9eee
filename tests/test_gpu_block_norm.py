"""Layer norm against its FP64 definition: every type, widths and row counts
where tiles, vectors and loops end, strides and offsets, missing parameters,
rows that hold infinities or NaNs, empty calls, and refusals."""
import numpy as np
import pytest
import torch

from tests import blockkit as kit
from tests.routekit import log

pytestmark = pytest.mark.gpu

block = pytest.importorskip("latent_projection_top_amd.block")
from latent_projection_top_amd import route  # noqa: E402

BF, HF, FP = torch.bfloat16, torch.float16, torch.float32


def run(c, backward=True):
    plan = block.NormPlan(c.rows + 3, c.width, dtype=c.dtype, param_dtype=c.pdt, eps=c.eps)
    ws = plan.new_workspace()
    dev = c.x.device
    got = {k: torch.full((c.rows, c.width), float("nan"), dtype=c.dtype, device=dev) for k in ("y", "dx")}
    for k in ("mean", "rstd"):
        got[k] = torch.full((c.rows,), float("nan"), device=dev)
    for k in ("dweight", "dbias"):
        got[k] = torch.full((c.width,), float("nan"), dtype=c.pdt, device=dev)
    block.layer_norm(plan, c.x, c.weight, c.bias, got["y"], got["mean"], got["rstd"])
    if backward:
        block.layer_norm_backward(plan, c.dy, c.x, c.weight, got["mean"], got["rstd"], got["dx"],
                                  got["dweight"], got["dbias"], ws)
    torch.cuda.synchronize()
    return got


def compare(c, got):
    for name, (ref, bound, scale) in c.reference().items():
        kit.check(got[name], ref, bound, scale, got[name].dtype, name)


WIDTHS = (1, 2, 3, 63, 64, 65, 127, 256, 500, 512, 1000, 1019, 1024, 2047, 2048, 3584, 4096, 5000, 7168, 8192,
          9001, 16384, 20000, 40001)


@pytest.mark.parametrize("dtype", (BF, HF, FP))
@pytest.mark.parametrize("width", WIDTHS)
def test_widths(width, dtype):
    rows = 37 if width < 9000 else 5
    log(f"norm {rows}x{width} {dtype}")
    c = kit.NormCase(rows, width, dtype, seed=width)
    compare(c, run(c))


@pytest.mark.parametrize("rows,width", [(1, 7168), (2, 7168), (1, 1), (1, 64), (255, 96), (256, 96), (257, 96),
                                        (1025, 72), (4099, 130), (2049, 1024), (700, 3584), (20011, 8)])
def test_rows(rows, width):
    log(f"norm {rows}x{width}")
    c = kit.NormCase(rows, width, BF, seed=rows)
    compare(c, run(c))


@pytest.mark.parametrize("pdt", (BF, HF, FP))
@pytest.mark.parametrize("weight,bias", [(True, False), (False, True), (False, False), (True, True)])
def test_parameters(pdt, weight, bias):
    c = kit.NormCase(70, 520, BF, param_dtype=pdt, weight=weight, bias=bias, seed=5)
    compare(c, run(c))


@pytest.mark.parametrize("dtype", (BF, FP))
@pytest.mark.parametrize("width,stride,offset", [(512, 520, 0), (512, 513, 0), (512, 512, 1), (3584, 7168, 3),
                                                 (100, 999, 5), (8, 8, 1), (1024, 1032, 4)])
def test_strides(width, stride, offset, dtype):
    """Rows inside a wider buffer of NaNs, at every alignment: nothing of the
    buffer leaks in, nothing is written beside the rows."""
    c = kit.NormCase(19, width, dtype, stride=stride, offset=offset, seed=3)
    plan = block.NormPlan(19, width, dtype=dtype, eps=c.eps)
    got = run(c)
    compare(c, got)
    for src, dst in ((c.x, "y"), (c.dy, "dx")):
        out, buf = kit.rows_like(torch.zeros_like(src), dtype, stride, offset, fill=7.0)
        if dst == "y":
            block.layer_norm(plan, c.x, c.weight, c.bias, out)
        else:
            block.layer_norm_backward(plan, c.dy, c.x, c.weight, got["mean"], got["rstd"], out, None, None,
                                      plan.new_workspace())
        torch.cuda.synchronize()
        assert torch.equal(out, got[dst])
        out.fill_(7.0)
        assert (buf == 7.0).all()


def test_far_mean_and_constant_rows():
    """Rows whose mean is large against their spread, and rows of one value
    (variance 0: y is the bias)."""
    c = kit.NormCase(16, 3584, FP, shift=1000.0, seed=8)
    compare(c, run(c))
    c = kit.NormCase(4, 3584, BF, seed=8)
    c.x[1].fill_(3.0)
    c.x[2].fill_(0.0)
    got = run(c)
    assert torch.equal(got["y"][1], c.bias.to(BF)) and torch.equal(got["y"][2], c.bias.to(BF))
    np.testing.assert_allclose(got["rstd"][1:3].cpu().numpy(), c.eps ** -0.5, rtol=1e-6)


def test_nonfinite_rows_stay_alone():
    c = kit.NormCase(33, 1000, BF, seed=2)
    clean = run(c)
    c.x[4, 17] = float("nan")
    c.x[9, 999] = float("inf")
    c.x[20, 0] = float("-inf")
    got = run(c)
    keep = torch.ones(33, dtype=torch.bool, device="cuda")
    keep[[4, 9, 20]] = False
    assert torch.equal(got["y"][keep], clean["y"][keep]) and torch.equal(got["dx"][keep], clean["dx"][keep])
    assert torch.isnan(got["y"][~keep]).all()
    assert torch.isnan(got["dweight"]).all() and torch.equal(got["dbias"], clean["dbias"])


@pytest.mark.parametrize("width", (64, 1000, 9001))
def test_empty_and_partial_calls(width):
    c = kit.NormCase(9, width, BF, seed=1)
    plan = block.NormPlan(9, width)
    ws = plan.new_workspace()
    empty = c.x[:0]
    y = torch.full((9, width), 7.0, dtype=BF, device="cuda")
    block.layer_norm(plan, empty, c.weight, c.bias, y)
    dw, db = (torch.full((width,), 7.0, device="cuda") for _ in range(2))
    m = torch.empty(0, device="cuda")
    block.layer_norm_backward(plan, empty, empty, c.weight, m, m, empty, dw, db, ws)
    torch.cuda.synchronize()
    assert (y == 7.0).all() and (dw == 0).all() and (db == 0).all()
    # fewer rows than the plan and the tensors hold
    block.layer_norm(plan, c.x, c.weight, c.bias, y, rows=4)
    torch.cuda.synchronize()
    assert (y[4:] == 7.0).all() and torch.equal(y[:4], run(c, backward=False)["y"][:4])


def test_each_gradient_alone():
    c = kit.NormCase(50, 640, BF, seed=4)
    full = run(c)
    plan = block.NormPlan(50, 640)
    ws = plan.new_workspace()
    for want in ("dx", "dweight", "dbias"):
        out = {k: torch.full_like(full[k], 7.0) if k == want else None for k in ("dx", "dweight", "dbias")}
        block.layer_norm_backward(plan, c.dy, c.x, c.weight, full["mean"], full["rstd"], out["dx"],
                                  out["dweight"], out["dbias"], ws)
        torch.cuda.synchronize()
        assert torch.equal(out[want], full[want])


def test_gradient_against_differences():
    """The kernel's gradients along random directions against central
    differences of the FP64 forward definition; FP32 tensors. With a step of
    2^-10 the differences' own error is below 1e-5 of the values here."""
    c = kit.NormCase(6, 300, FP, seed=11)
    got = run(c)
    gen = torch.Generator(device="cuda").manual_seed(1)

    def loss(x, w, b):
        m = x.mean(1, keepdim=True)
        v = (x - m).square().mean(1, keepdim=True)
        return (((x - m) / torch.sqrt(v + c.eps) * w + b) * c.dy.double()).sum()

    base = [t.double() for t in (c.x, c.weight, c.bias)]
    for i, name in enumerate(("dx", "dweight", "dbias")):
        d = torch.randn(base[i].shape, generator=gen, device="cuda", dtype=torch.float64)
        h = 2.0 ** -10
        hi, lo = (loss(*[t + s * h * d if j == i else t for j, t in enumerate(base)]) for s in (1, -1))
        num = float((hi - lo) / (2 * h))
        ana = float((got[name].double() * d).sum())
        scale = float((got[name].double() * d).square().sum().sqrt())
        assert abs(num - ana) <= 1e-4 * scale, (name, num, ana)


def test_repeatable_and_in_a_graph():
    """The same bits on every call, on another stream and from a graph that is
    replayed with new inputs and other work between the replays."""
    c = kit.NormCase(600, 1000, BF, seed=6)
    plan = block.NormPlan(600, 1000, eps=c.eps)
    ws = plan.new_workspace()
    got = run(c)
    names = ("y", "mean", "rstd", "dx", "dweight", "dbias")
    buf = {k: torch.empty_like(got[k]) for k in names}
    x, dy = c.x.clone(), c.dy.clone()

    def step():
        block.layer_norm(plan, x, c.weight, c.bias, buf["y"], buf["mean"], buf["rstd"])
        block.layer_norm_backward(plan, dy, x, c.weight, buf["mean"], buf["rstd"], buf["dx"], buf["dweight"],
                                  buf["dbias"], ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    assert all(torch.equal(buf[k], got[k]) for k in names)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (21, 22, 23):
        n = kit.NormCase(600, 1000, BF, seed=seed)
        n.weight, n.bias = c.weight, c.bias
        x.copy_(n.x)
        dy.copy_(n.dy)
        graph.replay()
        torch.cuda.synchronize()
        ref = run(n)
        assert all(torch.equal(buf[k], ref[k]) for k in names)


def test_refusals():
    c = kit.NormCase(8, 64, BF, seed=1)
    plan = block.NormPlan(8, 64)
    ws = plan.new_workspace()
    y = torch.empty(8, 64, dtype=BF, device="cuda")
    m = torch.empty(8, device="cuda")

    def fwd(status, p=plan, **kw):
        a = dict(x=c.x, weight=c.weight, bias=c.bias, y=y)
        a.update(kw)
        with pytest.raises(status):
            block.layer_norm(p, **a)

    fwd(TypeError, x=c.x.float())
    fwd(TypeError, weight=c.weight.to(BF))
    fwd(ValueError, x=c.x.cpu())
    fwd(ValueError, x=c.x.t())
    fwd(ValueError, x=c.x[:, :32])
    fwd(ValueError, x=c.x[:1].expand(8, 64))
    fwd(ValueError, y=y[:4])
    fwd(ValueError, bias=c.bias[:10])
    fwd(ValueError, mean=m[:3], rstd=m)
    for kw, st in ((dict(rows=-1), route.E_ROWS), (dict(mean=m), route.E_ARG)):
        with pytest.raises(route.RouteError) as e:
            block.layer_norm(plan, c.x, c.weight, c.bias, y, **kw)
        assert e.value.status == st
    small = block.NormPlan(7, 64)
    with pytest.raises(route.RouteError) as e:
        block.layer_norm(small, c.x, c.weight, c.bias, y)
    assert e.value.status == route.E_ROWS
    with pytest.raises(route.RouteError) as e:
        block.layer_norm_backward(plan, c.dy, c.x, c.weight, m, m, None, None, None, ws)
    assert e.value.status == route.E_ARG
    with pytest.raises(ValueError):
        block.layer_norm_backward(plan, c.dy, c.x, c.weight, m, m, y, None, None, ws[:100])
    # raw calls: strides, alignment, NULL
    s = torch.cuda.current_stream().cuda_stream or None
    px, py, pm = c.x.data_ptr(), y.data_ptr(), m.data_ptr()
    call = block.LIB.block_norm
    assert call(plan.handle, px, 63, None, None, py, 64, None, None, 8, s) == route.E_SHAPE
    assert call(plan.handle, px, 64, None, None, py, block.MAX_STRIDE + 1, None, None, 8, s) == route.E_SHAPE
    assert call(plan.handle, px + 1, 64, None, None, py, 64, None, None, 8, s) == route.E_ALIGN
    assert call(plan.handle, px, 64, None, None, py, 64, pm + 2, pm, 8, s) == route.E_ALIGN
    assert call(plan.handle, None, 64, None, None, py, 64, None, None, 8, s) == route.E_ARG
    back = block.LIB.block_norm_backward
    assert back(plan.handle, px, 64, px, 64, None, pm, pm, py, 64, None, None, ws.data_ptr() + 16, 8,
                s) == route.E_ALIGN
    assert back(plan.handle, px, 64, px, 64, None, pm, pm, py, 64, None, None, None, 8, s) == route.E_ARG
