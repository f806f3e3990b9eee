"""Gather, combine and their gradients against FP64."""
import pytest
import torch

from tests import blockkit as bk
from tests import expertskit as kit
from tests.routekit import log

pytestmark = pytest.mark.gpu

experts = pytest.importorskip("latent_projection_top_amd.experts")
from latent_projection_top_amd import route  # noqa: E402

BF, HF, FP = kit.BF, kit.HF, kit.FP


def same(got, ref, dtype, what):
    """Equal to the reference rounded once (no sum: nothing else to round)."""
    assert torch.equal(got, ref.to(dtype)), what


def run(c, stride=0, offset=0, residual=True):
    """All four calls; outputs in buffers that hold 3 before."""
    plan = experts.CombinePlan(c.rows, c.topk, c.width, dtype=c.dtype)

    def buffer(rows):
        return bk.rows_like(torch.full((rows, c.width), 3.0, device="cuda").to(c.dtype), c.dtype, stride, offset)[0]

    xs, dys, dx, y = buffer(c.capacity), buffer(c.capacity), buffer(c.rows), buffer(c.rows)
    dw = torch.full((c.rows, c.topk), 3.0, device="cuda")
    experts.gather(plan, c.x, c.place, xs)
    experts.gather_backward(plan, c.dxs, c.place, dx)
    experts.combine(plan, c.ys, c.place, c.weights, y, residual=c.residual if residual else None)
    experts.combine_backward(plan, c.dy, c.ys, c.place, c.weights, dys, dw)
    torch.cuda.synchronize()
    return xs, dx, y, dys, dw


def check(c, **kw):
    xs, dx, y, dys, dw = run(c, **kw)
    fill = torch.full((c.capacity, c.width), 3.0, device="cuda")
    same(xs, c.spread(fill, rows=c.x), c.dtype, "xs")
    bk.check(dys, c.spread(fill, c.weights, c.dy), kit.E * c.spread(fill, c.weights, c.dy).abs(), None, c.dtype, "dys")
    bk.check(dx, *c.collect(c.dxs), None, c.dtype, "dx")
    residual = c.residual if kw.get("residual", True) else None
    bk.check(y, *c.collect(c.ys, c.weights, residual), None, c.dtype, "y")
    bk.check(dw, *c.dweights(), None, FP, "dweights")


SIZES = [(1, 1, 1, 4, 4), (1, 16, 3584, 896, 896), (2, 3, 7, 8, 4), (8, 16, 7168, 896, 896), (20, 16, 7168, 896, 112),
         (33, 8, 1000, 64, 64), (333, 6, 1001, 64, 32), (64, 64, 264, 128, 128), (1024, 2, 64, 8, 1),
         (513, 17, 2049, 300, 100), (5, 4, 20001, 16, 16), (2500, 16, 72, 40, 20)]


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("rows,topk,width,total,count", SIZES)
def test_forward_and_gradients(rows, topk, width, total, count, dtype):
    log(f"rows {rows}x{topk}x{width} {count}/{total} {dtype}")
    check(kit.RowsCase(rows, topk, width, total, count, dtype, first=total - count, seed=rows))


@pytest.mark.parametrize("dtype", [BF, HF, FP])
@pytest.mark.parametrize("width,stride,offset", [(64, 72, 0), (65, 65, 1), (1001, 1003, 3), (512, 513, 1), (7, 9, 5)])
def test_strides_and_alignment(width, stride, offset, dtype):
    log(f"rows strides {width}/{stride}+{offset} {dtype}")
    check(kit.RowsCase(70, 5, width, 12, 9, dtype, seed=3, stride=stride, offset=offset), stride=stride,
          offset=offset)


@pytest.mark.parametrize("rows,topk,width", [(3, 16, 7168), (100, 7, 1001), (700, 16, 256)])
def test_sums_that_are_exact(rows, topk, width):
    """Integers whose products and sums FP32 holds: no term lost or doubled."""
    log(f"rows exact {rows}x{topk}x{width}")
    c = kit.RowsCase(rows, topk, width, 64, 48, FP, seed=5, whole=True)
    xs, dx, y, dys, dw = run(c)
    assert torch.equal(dx.double(), c.collect(c.dxs)[0])
    assert torch.equal(y.double(), c.collect(c.ys, c.weights, c.residual)[0])
    assert torch.equal(dw.double(), c.dweights()[0])


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("capacity", [0, 1, 300, 1000])
def test_capacity(capacity, dtype):
    """Sorted buffers that do not hold every choice: the rest are dropped."""
    log(f"rows capacity {capacity} {dtype}")
    check(kit.RowsCase(130, 6, 200, 16, 16, dtype, seed=6, capacity=capacity))


@pytest.mark.parametrize("dtype", [BF, HF, FP])
def test_nothing_of_a_dropped_choice_is_read(dtype):
    """Weights of dropped choices hold infinities and NaN, the spare rows of
    the sorted buffers NaN; rows with nothing left are the residual, or 0."""
    log(f"rows dropped {dtype}")
    c = kit.RowsCase(90, 4, 333, 64, 8, dtype, seed=7)
    gone = c.place < 0
    assert gone.all(1).any() and not gone.all()
    c.weights[gone] = float("nan")
    c.weights[gone & (torch.arange(4, device="cuda") % 2 == 0)] = float("inf")
    kept = int(c.offsets[-1])
    c.ys[kept:] = float("nan")
    c.dxs[kept:] = float("nan")
    check(c)
    xs, dx, y, dys, dw = run(c, residual=False)
    empty = gone.all(1)
    assert (y[empty] == 0).all() and (dx[empty] == 0).all() and (dw[gone] == 0).all()


def test_places_that_no_buffer_has():
    """place is not trusted: entries outside the buffer count as dropped."""
    log("rows foreign places")
    c = kit.RowsCase(50, 4, 100, 16, 16, BF, seed=8)
    c.place[::3, 1] = 200
    c.place[1::3, 2] = 2 ** 31 - 1
    c.place[2::3, 0] = -2 ** 31
    check(c)


def test_infinities_and_nan_come_through():
    log("rows infinities")
    c = kit.RowsCase(4, 2, 16, 4, 4, BF, seed=9)
    c.ys[c.place[1, 0].long(), 3] = float("inf")
    c.ys[c.place[2, 1].long(), 5] = float("nan")
    _, _, y, _, dw = run(c)
    assert torch.isinf(y[1, 3]) and torch.isnan(y[2, 5])
    assert int((~torch.isfinite(y.float())).sum()) == 2
    assert torch.isnan(dw[2, 1]) and not torch.isfinite(dw[1, 0])
    assert int((~torch.isfinite(dw)).sum()) == 2


def test_each_gradient_alone_and_in_place_residual():
    log("rows parts")
    c = kit.RowsCase(70, 6, 500, 16, 12, BF, seed=10)
    plan = experts.CombinePlan(c.rows, c.topk, c.width)
    _, _, y, dys, dw = run(c)
    dys2, dw2 = torch.full_like(dys, 3.0), torch.full_like(dw, 3.0)
    experts.combine_backward(plan, c.dy, c.ys, c.place, None, None, dw2)
    experts.combine_backward(plan, c.dy, None, c.place, c.weights, dys2, None)
    y2 = c.residual.clone()
    experts.combine(plan, c.ys, c.place, c.weights, y2, residual=y2)
    torch.cuda.synchronize()
    assert torch.equal(dys, dys2) and torch.equal(dw, dw2) and torch.equal(y, y2)


def test_gradients_against_differences():
    """The directional derivative of sum(dy * y) along (ys, weights), and of
    sum(dxs * xs) along x, in FP32: both forms are linear in each argument, so
    the differences have no truncation error, only the sums' rounding."""
    log("rows differences")
    c = kit.RowsCase(40, 6, 128, 16, 12, FP, seed=11, whole=True)
    plan = experts.CombinePlan(c.rows, c.topk, c.width, dtype=FP)
    _, dx, y, dys, dw = run(c)
    live = c.live()
    on = live >= 0

    def forward(ys, weights):
        out = torch.empty_like(y)
        experts.combine(plan, ys, c.place, weights, out, residual=c.residual)
        return (out.double() * c.dy.double()).sum()

    gen = torch.Generator(device="cuda").manual_seed(1)
    d = torch.randint(-2, 3, c.ys.shape, generator=gen, device="cuda").float()
    # dys is left alone where no choice is placed: take those out of the direction
    placed = torch.zeros(c.ys.shape[0], 1, device="cuda")
    placed[live[on]] = 1
    d *= placed
    assert forward(c.ys + d, c.weights) - forward(c.ys, c.weights) == (d.double() * (dys * placed).double()).sum()
    d = torch.randint(-2, 3, c.weights.shape, generator=gen, device="cuda").float()
    assert forward(c.ys, c.weights + d) - forward(c.ys, c.weights) == (d.double() * dw.double()).sum()
    d = torch.randint(-2, 3, c.x.shape, generator=gen, device="cuda").float()
    out = torch.zeros_like(c.dxs)
    experts.gather(plan, c.x + d, c.place, out)
    xs = torch.zeros_like(c.dxs)
    experts.gather(plan, c.x, c.place, xs)
    assert ((out - xs).double() * c.dxs.double()).sum() == (d.double() * dx.double()).sum()


def test_no_rows_and_fewer_rows_than_the_plan():
    log("rows few")
    plan = experts.CombinePlan(50, 4, 64)
    c = kit.RowsCase(9, 4, 64, 8, 8, BF, seed=12)
    y = torch.full((12, 64), 3.0, dtype=BF, device="cuda")
    experts.combine(plan, c.ys, c.place, c.weights, y, rows=9)
    ref, bound = c.collect(c.ys, c.weights)
    torch.cuda.synchronize()
    bk.check(y[:9], ref, bound, None, BF, "y")
    assert (y[9:] == 3).all()
    none = torch.empty(0, 64, dtype=BF, device="cuda")
    places, weights = c.place[:0], c.weights[:0]
    experts.gather(plan, none, places, none)
    experts.gather_backward(plan, none, places, none)
    experts.combine(plan, none, places, weights, none)
    experts.combine_backward(plan, none, none, places, weights, none, weights)
    torch.cuda.synchronize()


def test_offsets_past_32_bits():
    """Sorted rows of which the last begin beyond 2^32 bytes, and the places
    that reach them."""
    log("rows 64-bit")
    width, cap = 7168, 310000  # 4.4 GB
    rows, topk = 3, 2
    ys = torch.zeros(cap, width, dtype=BF, device="cuda")
    place = torch.tensor([[cap - 1, 0], [cap - 2, cap - 3], [5, -1]], dtype=torch.int32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(3)
    at = [cap - 1, cap - 2, cap - 3, 0, 5]
    ys[at] = torch.randn(5, width, generator=gen, device="cuda").to(BF)
    weights = torch.rand(rows, topk, generator=gen, device="cuda")
    plan = experts.CombinePlan(rows, topk, width)
    y, x = torch.empty(rows, width, dtype=BF, device="cuda"), torch.randn(rows, width, device="cuda").to(BF)
    dw = torch.empty(rows, topk, device="cuda")
    experts.combine(plan, ys, place, weights, y)
    experts.combine_backward(plan, x, ys, place, weights, None, dw)
    torch.cuda.synchronize()
    want = torch.zeros(rows, width, dtype=torch.float64, device="cuda")
    for r in range(rows):
        for j in range(topk):
            if place[r, j] >= 0:
                v = ys[int(place[r, j])].double()
                want[r] += weights[r, j].double() * v
                dot = (v * x[r].double())
                assert abs(float(dw[r, j]) - float(dot.sum())) <= (width + 3) * kit.E * float(dot.abs().sum())
    size = want.abs().max()
    bk.check(y, want, 4 * kit.E * (want.abs() + size), None, BF, "y")
    experts.gather(plan, x, place, ys)
    torch.cuda.synchronize()
    assert torch.equal(ys[cap - 1], x[0]) and torch.equal(ys[0], x[0]) and torch.equal(ys[cap - 2], x[1])
    assert torch.equal(ys[cap - 3], x[1]) and torch.equal(ys[5], x[2]) and (ys[6:cap - 3] == 0).all()


def test_refusals():
    plan = experts.CombinePlan(4, 2, 8)
    x, xs = torch.zeros(4, 8, dtype=BF, device="cuda"), torch.zeros(8, 8, dtype=BF, device="cuda")
    place = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    w = torch.zeros(4, 2, device="cuda")
    y = torch.zeros_like(x)
    experts.combine(plan, xs, place, w, y)
    for call, kind in (
            (lambda: experts.gather(plan, x.half(), place, xs), TypeError),
            (lambda: experts.gather(plan, x, place.long(), xs), TypeError),
            (lambda: experts.combine(plan, xs, place, w.double(), y), TypeError),
            (lambda: experts.gather(plan, x[:, :4], place, xs), ValueError),
            (lambda: experts.gather(plan, x, place[:3], xs), ValueError),
            (lambda: experts.gather(plan, x, place, xs.cpu()), ValueError),
            (lambda: experts.combine(plan, xs.t(), place, w, y), ValueError),
            (lambda: experts.combine(plan, xs, place, w, y, residual=x[:2]), ValueError),
            (lambda: experts.combine(plan, xs[:1].expand(8, 8), place, w, y), ValueError),
            (lambda: experts.combine_backward(plan, x, xs, place, w, xs[:7].clone(), w), ValueError),
            (lambda: experts.combine_backward(plan, x, xs, place, w, None, None), route.RouteError),
            (lambda: experts.combine_backward(plan, x, xs, place, None, xs.clone(), None), route.RouteError),
            (lambda: experts.combine(plan, xs, torch.zeros(5, 2, dtype=torch.int32, device="cuda"),
                                     torch.zeros(5, 2, device="cuda"), torch.zeros(5, 8, dtype=BF, device="cuda")),
             route.RouteError)):
        with pytest.raises(kind):
            call()
    lib, stream = experts.LIB.experts_combine, None
    args = [plan.handle, xs.data_ptr(), 8, place.data_ptr(), w.data_ptr(), None, 8, y.data_ptr(), 8, 8, 4, stream]
    for i, value, status in ((1, None, route.E_ARG), (3, None, route.E_ARG), (4, None, route.E_ARG),
                             (7, None, route.E_ARG), (2, 7, route.E_SHAPE), (8, 1 << 21, route.E_SHAPE),
                             (9, -1, route.E_ROWS), (9, experts.MAX_CHOICES + 1, route.E_ROWS), (10, 5, route.E_ROWS),
                             (10, -1, route.E_ROWS), (1, xs.data_ptr() + 1, route.E_ALIGN),
                             (4, w.data_ptr() + 2, route.E_ALIGN)):
        bad = list(args)
        bad[i] = value
        assert lib(*bad) == status, (i, value)
    torch.cuda.synchronize()
