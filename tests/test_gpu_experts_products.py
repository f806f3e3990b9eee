"""The 8-bit products against FP64: the integers are decided exactly, so the
bound is that of a few FP32 operations and one rounding."""
import pytest
import torch

from tests import blockkit as bk
from tests import expertskit as kit
from tests.routekit import log

pytestmark = pytest.mark.gpu

experts = pytest.importorskip("latent_projection_top_amd.experts")
from latent_projection_top_amd import route  # noqa: E402

BF, HF, FP = kit.BF, kit.HF, kit.FP

DENSE = [(1, 64, 16), (1, 1, 1), (2, 3, 5), (7, 100, 33), (15, 130, 260), (16, 256, 48), (17, 257, 47), (31, 1019, 777),
         (32, 512, 512), (33, 640, 300), (48, 1000, 264), (64, 2048, 256), (65, 63, 255), (100, 200, 257),
         (129, 321, 130), (200, 777, 513), (256, 64, 512), (300, 1001, 600), (517, 1019, 777), (1, 7168, 7168),
         (8, 2048, 7168), (20, 3584, 2048), (700, 512, 2000), (2048, 640, 1024)]


@pytest.mark.parametrize("planes,act,bias,residual", [(1, "none", False, True), (1, "gelu", True, False),
                                                      (2, "silu", False, False)])
@pytest.mark.parametrize("rows,k,n", DENSE)
def test_dense(rows, k, n, planes, act, bias, residual):
    log(f"dense {planes} {rows}x{k}x{n} {act}")
    kit.ProductCase(planes, k, n, act, BF, rows=rows, bias=bias, residual=residual, seed=rows + k).check(
        experts, f"{rows}x{k}x{n}")


COUNTS = [[0, 3, 0, 17, 1, 0], [1] * 40, [5, 0, 64, 65, 1, 200], [0, 0, 0, 700], [16, 32, 48, 33, 31, 15, 17],
          [256, 257, 1, 255, 512], [2], [40] * 9 + [0] * 50 + [7]]


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("planes,act,tokens", [(1, "gelu_tanh", 0), (2, "silu", 50), (2, "relu", 0), (1, "silu", 3)])
@pytest.mark.parametrize("counts", COUNTS, ids=[f"c{i}" for i in range(len(COUNTS))])
@pytest.mark.parametrize("k,n", [(192, 256), (1019, 333)])
def test_by_expert(k, n, counts, planes, act, tokens, dtype):
    log(f"experts {planes} {counts} {k}x{n} {act} {tokens} {dtype}")
    kit.ProductCase(planes, k, n, act, dtype, counts=counts, tokens=tokens, bias=planes == 1, residual=planes == 1,
                    seed=k + len(counts), spare=9).check(experts, f"{counts}")


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("rows", [5, 40, 300])
def test_activations(act, rows):
    log(f"acts {act} {rows}")
    kit.ProductCase(1, 256, 320, act, HF, rows=rows, bias=True, residual=True, seed=1).check(experts, act)
    if act != "none":
        kit.ProductCase(2, 256, 320, act, BF, rows=rows, seed=2).check(experts, act)


@pytest.mark.parametrize("rows", [3, 20, 70, 260])
@pytest.mark.parametrize("xs,ys,offset", [(200, 100, 0), (203, 97, 1), (264, 128, 3)])
def test_strides_and_alignment(rows, xs, ys, offset):
    log(f"product strides {rows} {xs} {ys} {offset}")
    for planes, act in ((1, "silu"), (2, "gelu")):
        kit.ProductCase(planes, 199, 95, act, BF, rows=rows, bias=True, residual=planes == 1, seed=4, xs=xs, ys=ys,
                        offset=offset).check(experts, "strided", ys=ys, offset=offset)


@pytest.mark.parametrize("rows,k", [(1, 131071), (40, 131071), (5, 100000), (300, 40000)])
def test_long_sums_of_the_largest_integers(rows, k):
    """Every weight -128 or 127 and every row's values of one size: the sums
    reach 2^31 of what 32 bits hold."""
    log(f"long {rows}x{k}")
    c = kit.ProductCase(1, k, 40, "none", BF, rows=rows, seed=5, extreme=True)
    c.x.copy_(torch.where(c.w[0][0, :, :1].t() > 0, 1.5, -1.5).to(BF).expand(rows, k))
    c.w[0][0, :, 1] = -128
    c.x[rows // 2:] = 2.0
    c.check(experts, "long")


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("rows", [4, 50, 300])
def test_values_on_the_borders(rows, dtype):
    """Rows whose values lie on the borders between two integers: multiples of
    half a step, where nearest-even decides."""
    log(f"borders {rows} {dtype}")
    c = kit.ProductCase(1, 254, 64, "none", dtype, rows=rows, seed=6)
    steps = torch.arange(-127, 127, device="cuda") + 0.5  # x = a (n + 1/2) / 127
    for r in range(rows):
        a = 127.0 * 2.0 ** (r % 7 - 3)
        c.x[r] = (steps * a / 127).to(dtype)
        c.x[r, 0] = a
    c.check(experts, "borders")


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("rows", [6, 50, 300])
def test_rows_of_extreme_values(rows, dtype):
    """Zeros, the smallest subnormal, the largest number, one value alone."""
    log(f"extremes {rows} {dtype}")
    c = kit.ProductCase(1, 200, 64, "none", dtype, rows=rows, seed=7)
    info = torch.finfo(dtype)
    small = 2.0 ** -133 if dtype is BF else 2.0 ** -24
    c.x[0] = 0
    c.x[1] = small
    c.x[2] = (torch.randint(-3, 4, (200,), device="cuda") * small).to(dtype)
    c.x[3] = info.max
    c.x[3, ::2] = -info.max
    c.x[4] = 0
    c.x[4, 199] = 1.0
    c.x[5] = info.tiny
    c.scale[0].fill_(2.0 ** -10)  # the largest rows stay finite in FP32
    plan = c.plan(experts)
    y = torch.empty(rows, 64, dtype=dtype, device="cuda")
    c.run(experts, plan, experts.pack(plan, *c.w), y, plan.new_workspace())
    torch.cuda.synchronize()
    ref, bound = c.reference()
    # scales below FP32's smallest normal number, and products with them, are
    # rounded to multiples of 2^-149 by half of it each: times the integers'
    # sum and the channel's scale
    bound = bound + 2.0 ** -150 * (2 + 200 * 127 * 128 * 2.0 ** -10)
    over = ref.abs() > float(info.max)  # rounds to infinity
    assert torch.isinf(y[over]).all()
    bk.check(torch.where(over, 0, y), torch.where(over, 0, ref), bound, None, dtype, "extremes")
    assert (y[0] == 0).all()


@pytest.mark.parametrize("rows", [4, 50, 300])
def test_rows_that_are_not_finite(rows):
    """An infinity or NaN makes its own row NaN and no other."""
    log(f"not finite {rows}")
    for planes, act in ((1, "none"), (2, "silu")):
        c = kit.ProductCase(planes, 100, 70, act, BF, rows=rows, seed=8)
        c.x[1, 37], c.x[2, 99], c.x[rows - 1, 0] = float("nan"), float("inf"), -float("inf")
        plan = c.plan(experts)
        y = torch.empty(rows, 70, dtype=BF, device="cuda")
        c.run(experts, plan, experts.pack(plan, *c.w), y, plan.new_workspace())
        torch.cuda.synchronize()
        bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
        bad[[1, 2, rows - 1]] = True
        assert torch.isnan(y[bad]).all()
        ref, bound = c.reference()
        bk.check(y[~bad], ref[~bad], bound[~bad], None, BF, "other rows")


@pytest.mark.parametrize("dtype", [BF, HF])
def test_quantised_weights(dtype):
    """quantize: the integers and scales of 16-bit weights, channel by channel."""
    log(f"quantize {dtype}")
    gen = torch.Generator(device="cuda").manual_seed(9)
    for e, k, n in ((3, 100, 50), (1, 1, 1), (2, 7, 300), (1, 1000, 17)):
        w = torch.randn(e, k, n, generator=gen, device="cuda").to(dtype)
        w[0, :, 0] = 0
        plan = experts.Linear8Plan(1, k, n, experts=e, dtype=dtype)
        w8, scale = experts.quantize(plan, w)
        torch.cuda.synchronize()
        for i in range(e):
            q, s = kit.quantised(w[i].t())
            assert torch.equal(w8[i].double(), q.t())
            assert ((scale[i].double() - s[:, 0]).abs() <= kit.E * s[:, 0]).all()
        gated = experts.Gated8Plan(1, k, n, experts=e, dtype=dtype)
        again, _ = experts.quantize(gated, w)
        assert torch.equal(again, w8)
    w = torch.ones(1, 8, 4, dtype=dtype, device="cuda")
    w[0, 3, 1], w[0, 0, 2] = float("nan"), float("inf")
    _, scale = experts.quantize(experts.Linear8Plan(1, 8, 4, dtype=dtype), w)
    assert torch.isnan(scale[0]).tolist() == [False, True, True, False]


@pytest.mark.parametrize("offsets", [[0, 9, 3, 20, 40], [-5, 4, 4, 1 << 30, 33], [40, 0, 40, 0, 40],
                                     [7, 7, 7, 7, 7], [0, 2 ** 31 - 1, -2 ** 31, 5, 12]])
def test_offsets_that_make_no_sense(offsets):
    """offsets are not trusted: cut to the rows there are, no access leaves the
    buffers (guards around them keep their values); a row that no range has is
    left alone."""
    log(f"offsets {offsets}")
    rows, k, n = 33, 70, 40
    for planes in (1, 2):
        c = kit.ProductCase(planes, k, n, "silu", BF, counts=[rows, 0, 0, 0], seed=10)
        plan = c.plan(experts)
        c.offsets = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        buf = torch.full((rows + 8, n), 7.0, dtype=BF, device="cuda")
        y = buf[4:4 + rows]
        c.run(experts, plan, experts.pack(plan, *c.w), y, plan.new_workspace())
        torch.cuda.synchronize()
        assert (buf[:4] == 7).all() and (buf[4 + rows:] == 7).all()
        covered = torch.zeros(rows, dtype=torch.bool)
        cut = [min(max(o, 0), rows) for o in offsets]
        for a, b in zip(cut, cut[1:]):
            covered[a:max(a, b)] = True
        assert (y[~covered.cuda()] == 7).all()


def test_tokens_that_no_row_has():
    log("foreign tokens")
    c = kit.ProductCase(1, 64, 32, "none", BF, counts=[5, 30], tokens=10, seed=11)
    want = c.token.clamp(0, 9)
    c.token[3], c.token[20], want[3], want[20] = -1, 2 ** 31 - 1, 0, 9
    plan = c.plan(experts)
    y, y2 = (torch.empty(35, 32, dtype=BF, device="cuda") for _ in range(2))
    packed = experts.pack(plan, *c.w)
    c.run(experts, plan, packed, y, plan.new_workspace())
    c.token = want
    c.run(experts, plan, packed, y2, plan.new_workspace())
    torch.cuda.synchronize()
    assert torch.equal(y, y2)


def test_no_rows_and_fewer_rows_than_the_plan():
    log("product few rows")
    c = kit.ProductCase(1, 128, 64, "none", BF, rows=300, seed=12)
    plan = c.plan(experts)
    packed, ws = experts.pack(plan, *c.w), plan.new_workspace()
    ref, bound = c.reference()
    for rows in (300, 0, 1, 40, 299):
        y = torch.full((300, 64), 7.0, dtype=BF, device="cuda")
        c.run(experts, plan, packed, y, ws, rows=rows)
        torch.cuda.synchronize()
        bk.check(y[:rows], ref[:rows], bound[:rows], None, BF, f"{rows} rows")
        assert (y[rows:] == 7).all()
    many = kit.ProductCase(2, 128, 64, "silu", BF, counts=[10, 20], tokens=7, seed=13)
    plan = many.plan(experts)
    packed = experts.pack(plan, *many.w)
    none = torch.empty(0, 64, dtype=BF, device="cuda")
    many.x = many.x[:0]
    many.run(experts, plan, packed, none, plan.new_workspace(), rows=0)
    torch.cuda.synchronize()


def test_refusals():
    c = kit.ProductCase(1, 64, 32, "none", BF, counts=[2, 2], tokens=3, bias=True, seed=14)
    plan = c.plan(experts)
    packed, ws = experts.pack(plan, *c.w), plan.new_workspace()
    y = torch.zeros(4, 32, dtype=BF, device="cuda")

    def call(**kw):
        a = dict(x=c.x, packed=packed, scale=c.scale[0], y=y, workspace=ws, offsets=c.offsets, token=c.token,
                 bias=c.bias)
        a.update(kw)
        experts.linear8(plan, **a)

    call()
    for bad in (dict(x=c.x.half()), dict(scale=c.scale[0].double()), dict(offsets=c.offsets.long()),
                dict(bias=c.bias.float())):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in (dict(packed=packed[:-1]), dict(scale=c.scale[0][:1]), dict(offsets=c.offsets[:2]),
                dict(token=c.token[:3]), dict(y=y[:, :16]), dict(workspace=ws[:-1]), dict(x=c.x.cpu())):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(offsets=None), dict(x=c.x[:0]),
                dict(x=torch.zeros(4, 64, dtype=BF, device="cuda"))):
        with pytest.raises((route.RouteError, ValueError)):
            call(**bad)
    with pytest.raises(ValueError):
        experts.pack(plan, c.w[0], c.w[0])
    with pytest.raises(TypeError):
        experts.pack(plan, c.w[0].to(BF))
    lib = experts.LIB.experts_linear8
    args = [plan.handle, c.x.data_ptr(), 64, packed.data_ptr(), c.scale[0].data_ptr(), c.offsets.data_ptr(),
            c.token.data_ptr(), c.bias.data_ptr(), None, 32, y.data_ptr(), 32, ws.data_ptr(), 3, 4, None]
    for i, value, status in ((1, None, route.E_ARG), (3, None, route.E_ARG), (4, None, route.E_ARG),
                             (5, None, route.E_ARG), (10, None, route.E_ARG), (12, None, route.E_ARG),
                             (6, None, route.E_ROWS), (13, 0, route.E_ROWS), (13, 4, route.E_ROWS),
                             (14, 5, route.E_ROWS), (14, -1, route.E_ROWS), (2, 63, route.E_SHAPE),
                             (11, 31, route.E_SHAPE), (11, 1 << 21, route.E_SHAPE), (1, c.x.data_ptr() + 1, route.E_ALIGN),
                             (3, packed.data_ptr() + 128, route.E_ALIGN), (12, ws.data_ptr() + 16, route.E_ALIGN),
                             (6, c.token.data_ptr() + 2, route.E_ALIGN)):
        bad = list(args)
        bad[i] = value
        assert lib(*bad) == status, (i, value)
    torch.cuda.synchronize()
