"""The gated feed-forward and linear products against their FP64 definitions:
every activation and type, sizes on both sides of every tile and vector,
strides, offsets, shared buffers, rows with infinities or NaNs, empty calls,
graphs, gradients against differences, and refusals."""
import pytest
import torch

from tests import blockkit as kit
from tests.routekit import log

pytestmark = pytest.mark.gpu

block = pytest.importorskip("latent_projection_top_amd.block")
from latent_projection_top_amd import route  # noqa: E402

BF, HF = torch.bfloat16, torch.float16


def nan(*shape, dtype):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def run_gated(c, training=True, plan=None, ws=None, rows=None):
    plan = plan or block.GatedPlan(c.rows + 5, c.k, c.n, c.act, c.dtype, training=training)
    ws = plan.new_workspace() if ws is None else ws
    got = {"h": nan(c.rows, c.n, dtype=c.dtype)}
    if not training:
        block.gated(plan, c.x, c.wg, c.wu, got["h"], ws, rows=rows)
    else:
        got.update(d_gate=nan(c.rows, c.n, dtype=c.dtype), d_up=nan(c.rows, c.n, dtype=c.dtype),
                   dx=nan(c.rows, c.k, dtype=c.dtype), dw_gate=nan(c.k, c.n, dtype=c.dtype),
                   dw_up=nan(c.k, c.n, dtype=c.dtype))
        block.gated(plan, c.x, c.wg, c.wu, got["h"], ws, got["d_gate"], got["d_up"], rows=rows)
        block.gated_backward(plan, c.dh, c.x, c.wg, c.wu, got["d_gate"], got["d_up"], got["dx"],
                             got["dw_gate"], got["dw_up"], ws, rows=rows)
    torch.cuda.synchronize()
    return got


def run_linear(c, training=True, plan=None, ws=None):
    plan = plan or block.LinearPlan(c.rows + 5, c.k, c.n, c.act, c.dtype, training=training)
    ws = plan.new_workspace() if ws is None else ws
    got = {"y": nan(c.rows, c.n, dtype=c.dtype)}
    if not training:
        block.linear(plan, c.x, c.w, got["y"], ws, c.bias, c.residual)
    else:
        got.update(dx=nan(c.rows, c.k, dtype=c.dtype), dw=nan(c.k, c.n, dtype=c.dtype),
                   dbias=nan(c.n, dtype=c.dtype))
        if c.act != "none":
            got["slope"] = nan(c.rows, c.n, dtype=c.dtype)
        block.linear(plan, c.x, c.w, got["y"], ws, c.bias, c.residual, got.get("slope"))
        block.linear_backward(plan, c.dy, c.x, c.w, got.get("slope"), got["dx"], got["dw"], got["dbias"], ws)
    torch.cuda.synchronize()
    return got


def compare(c, got):
    ref = c.reference()
    for name, t in got.items():
        r, bound, scale = ref[name]
        kit.check(t, r, bound, scale, c.dtype, name)


SIZES = [  # rows, K, N
    (1, 1, 1), (1, 7, 5), (2, 8, 16), (3, 64, 8), (1, 3584, 512), (7, 1000, 24), (16, 512, 128),
    (17, 33, 65), (20, 256, 130), (32, 1024, 264), (33, 136, 1000), (63, 200, 72), (64, 64, 64), (65, 100, 72),
    (100, 2048, 520), (129, 1001, 257), (128, 128, 128), (192, 96, 384), (257, 264, 520), (300, 512, 384),
    (333, 1001, 777), (512, 1024, 768), (520, 776, 1032), (1111, 328, 600), (1024, 2048, 1024)]


@pytest.mark.parametrize("dtype", (BF, HF))
@pytest.mark.parametrize("rows,k,n", SIZES)
def test_gated_sizes(rows, k, n, dtype):
    log(f"gated {rows}x{k}x{n} {dtype}")
    c = kit.GatedCase(rows, k, n, "silu", dtype, seed=rows + k + n)
    got = run_gated(c)
    compare(c, got)
    serve = run_gated(c, training=False)
    assert torch.equal(serve["h"], got["h"])


@pytest.mark.parametrize("dtype", (BF, HF))
@pytest.mark.parametrize("rows,k,n", SIZES)
def test_linear_sizes(rows, k, n, dtype):
    log(f"linear {rows}x{k}x{n} {dtype}")
    c = kit.LinearCase(rows, k, n, "gelu", dtype, seed=rows + k + n)
    got = run_linear(c)
    compare(c, got)
    serve = run_linear(c, training=False)
    assert torch.equal(serve["y"], got["y"])


# one long side: many rows, a long reduction, a wide output
LONG = [(9000, 64, 96), (12289, 40, 24), (5, 20000, 64), (40, 131072, 8), (6, 16, 131072), (3, 24, 99999),
        (260, 16384, 264)]


@pytest.mark.parametrize("rows,k,n", LONG)
def test_long_sides(rows, k, n):
    log(f"long {rows}x{k}x{n}")
    c = kit.GatedCase(rows, k, n, "silu", BF, seed=1)
    compare(c, run_gated(c))
    c = kit.LinearCase(rows, k, n, "none", BF, seed=1)
    compare(c, run_linear(c))


@pytest.mark.parametrize("act", list(block.ACTIVATIONS))
@pytest.mark.parametrize("rows", (5, 150, 600))
def test_activations(act, rows):
    log(f"activation {act} rows {rows}")
    if act != "none":
        c = kit.GatedCase(rows, 264, 520, act, BF, seed=3, scale=3.0)
        compare(c, run_gated(c))
    for bias, residual in ((True, True), (True, False), (False, True), (False, False)):
        c = kit.LinearCase(rows, 264, 520, act, BF, bias=bias, residual=residual, seed=4)
        compare(c, run_linear(c))


# x's row stride, the outputs' row stride, and an offset that no vector load likes
STRIDES = [(5, 256, 264, 264, 272, 0), (5, 256, 264, 257, 265, 0), (40, 256, 256, 256, 256, 1),
           (150, 128, 320, 999, 333, 3), (300, 264, 520, 272, 528, 0), (300, 264, 520, 264, 520, 4),
           (600, 520, 264, 7168, 1024, 0), (19, 72, 1032, 80, 2000, 7), (1, 520, 264, 0, 0, 1)]


@pytest.mark.parametrize("rows,k,n,xs,ys,offset", STRIDES)
def test_strides(rows, k, n, xs, ys, offset):
    """Rows inside wider buffers of NaNs, at several alignments."""
    log(f"strides {rows}x{k}x{n} {xs} {ys} {offset}")
    c = kit.GatedCase(rows, k, n, "silu", BF, seed=5, xs=xs, hs=ys, offset=offset)
    compare(c, run_gated(c))
    c = kit.LinearCase(rows, k, n, "silu", BF, seed=5, xs=xs, ys=ys, offset=offset)
    compare(c, run_linear(c))


@pytest.mark.parametrize("rows,k,n,xs,ys,offset", STRIDES)
def test_outputs_stay_in_their_rows(rows, k, n, xs, ys, offset):
    c = kit.LinearCase(rows, k, n, "silu", BF, seed=6)
    ref = run_linear(c)
    plan = block.LinearPlan(rows, k, n, "silu", BF, training=True)
    ws = plan.new_workspace()
    y, ybuf = kit.rows_like(torch.zeros(rows, n, dtype=BF, device="cuda"), BF, ys, offset, fill=7.0)
    dx, dbuf = kit.rows_like(torch.zeros(rows, k, dtype=BF, device="cuda"), BF, xs, offset, fill=7.0)
    dwbuf = torch.full((k * n + 16,), 7.0, dtype=BF, device="cuda")
    dw = dwbuf[8:8 + k * n].view(k, n)
    block.linear(plan, c.x, c.w, y, ws, c.bias, c.residual)
    block.linear_backward(plan, c.dy, c.x, c.w, ref["slope"], dx, dw, None, ws)
    torch.cuda.synchronize()
    for got, want in ((y, ref["y"]), (dx, ref["dx"]), (dw, ref["dw"])):
        kit.check(got, want.double(), 2 * kit.UNIT[BF] * want.double().abs().max() * torch.ones_like(want.double()),
                  None, BF, "strided output")
    for got, buf in ((y, ybuf), (dx, dbuf), (dw, dwbuf)):
        got.fill_(7.0)
        assert (buf == 7.0).all()


@pytest.mark.parametrize("rows", (4, 40, 300))
def test_residual_in_place(rows):
    c = kit.LinearCase(rows, 264, 520, "none", BF, seed=7)
    want = run_linear(c, training=False)["y"]
    plan = block.LinearPlan(rows, 264, 520)
    y = c.residual.clone()
    block.linear(plan, c.x, c.w, y, plan.new_workspace(), bias=c.bias, residual=y)
    torch.cuda.synchronize()
    assert torch.equal(y, want)


@pytest.mark.parametrize("rows,k,n", [(6, 264, 264), (50, 264, 264), (300, 264, 264), (300, 261, 263)])
def test_nonfinite_rows_stay_alone(rows, k, n):
    """An infinity or NaN in a row of x changes that row of h and no other
    row; in a gradient row likewise for dx."""
    c = kit.GatedCase(rows, k, n, "silu", BF, seed=8)
    clean = run_gated(c)
    c.x[2, k - 1] = float("nan")
    c.x[rows - 1, 0] = float("inf")
    got = run_gated(c)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[[2, rows - 1]] = False
    assert torch.equal(got["h"][keep], clean["h"][keep]) and torch.equal(got["dx"][keep], clean["dx"][keep])
    assert torch.isnan(got["h"][2]).all() and not torch.isfinite(got["h"][rows - 1]).any()
    c = kit.LinearCase(rows, k, n, "none", BF, seed=8)
    clean = run_linear(c)
    c.dy[1, n - 1] = float("nan")
    got = run_linear(c)
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[1] = False
    assert torch.equal(got["dx"][keep], clean["dx"][keep]) and torch.isnan(got["dx"][1]).all()
    cols = torch.ones(n, dtype=torch.bool, device="cuda")
    cols[n - 1] = False
    assert torch.equal(got["dw"][:, cols], clean["dw"][:, cols])
    assert torch.equal(got["dbias"][cols], clean["dbias"][cols]) and torch.isnan(got["dbias"][n - 1])


def test_infinite_bias_and_residual():
    c = kit.LinearCase(9, 64, 40, "none", BF, seed=2)
    c.bias[3] = float("inf")
    c.residual[5, 7] = float("-inf")
    y = run_linear(c, training=False)["y"]
    assert (y[:, 3] == float("inf")).all() and y[5, 7] == float("-inf")
    assert int((~torch.isfinite(y)).sum()) == 10


def test_f16_overflow_is_infinite():
    x = torch.full((3, 64), 200.0, dtype=HF, device="cuda")
    w = torch.full((64, 16), 100.0, dtype=HF, device="cuda")
    plan = block.LinearPlan(3, 64, 16, dtype=HF)
    y = torch.empty(3, 16, dtype=HF, device="cuda")
    block.linear(plan, x, w, y, plan.new_workspace())
    torch.cuda.synchronize()
    assert (y == float("inf")).all()


@pytest.mark.parametrize("k,n", [(264, 136), (33, 65)])
def test_empty_calls(k, n):
    e = torch.empty(0, k, dtype=BF, device="cuda")
    en = torch.empty(0, n, dtype=BF, device="cuda")
    w = torch.ones(k, n, dtype=BF, device="cuda")
    plan = block.GatedPlan(4, k, n, training=True)
    ws = plan.new_workspace()
    dwg, dwu = torch.full_like(w, 7.0), torch.full_like(w, 7.0)
    block.gated(plan, e, w, w, en, ws, en, en)
    block.gated_backward(plan, en, e, w, w, en, en, e, dwg, dwu, ws)
    lplan = block.LinearPlan(4, k, n, "relu", training=True)
    lws = lplan.new_workspace()
    dw, db = torch.full_like(w, 7.0), torch.full((n,), 7.0, dtype=BF, device="cuda")
    block.linear(lplan, e, w, en, lws, residual=en, slope=en)
    block.linear_backward(lplan, en, e, w, en, e, dw, db, lws)
    torch.cuda.synchronize()
    for t in (dwg, dwu, dw, db):
        assert (t == 0).all()


@pytest.mark.parametrize("rows", (5, 40, 200, 520))
def test_fewer_rows_than_tensors(rows):
    """`rows` below the tensors' and the plan's: later rows keep their values
    and stay out of the weights' gradients."""
    c = kit.GatedCase(rows, 136, 264, "silu", BF, seed=9)
    big = kit.GatedCase(rows + 37, 136, 264, "silu", BF, seed=10)
    big.x[:rows], big.dh[:rows], big.wg, big.wu = c.x, c.dh, c.wg, c.wu
    got, ref = run_gated(big, rows=rows), run_gated(c)
    for k in ("h", "d_gate", "d_up", "dx"):
        assert torch.equal(got[k][:rows], ref[k]) and torch.isnan(got[k][rows:]).all()
    assert torch.equal(got["dw_gate"], ref["dw_gate"]) and torch.equal(got["dw_up"], ref["dw_up"])


@pytest.mark.parametrize("rows,k,n", [(6, 512, 264), (300, 264, 520)])
def test_each_gradient_alone(rows, k, n):
    c = kit.LinearCase(rows, k, n, "silu", BF, seed=12)
    full = run_linear(c)
    plan = block.LinearPlan(rows, k, n, "silu", training=True)
    ws = plan.new_workspace()
    for want in ("dx", "dw", "dbias"):
        out = {g: torch.full_like(full[g], 7.0) if g == want else None for g in ("dx", "dw", "dbias")}
        block.linear_backward(plan, c.dy, c.x, c.w, full["slope"], out["dx"], out["dw"], out["dbias"], ws)
        torch.cuda.synchronize()
        kit.check(out[want], full[want].double(), torch.zeros_like(full[want].double()), None, BF, want)
    g = kit.GatedCase(rows, k, n, "silu", BF, seed=12)
    full = run_gated(g)
    plan = block.GatedPlan(rows, k, n, training=True)
    ws = plan.new_workspace()
    dx = torch.full_like(full["dx"], 7.0)
    block.gated_backward(plan, g.dh, g.x, g.wg, g.wu, full["d_gate"], full["d_up"], dx, None, None, ws)
    dwg, dwu = torch.full_like(g.wg, 7.0), torch.full_like(g.wu, 7.0)
    block.gated_backward(plan, g.dh, g.x, g.wg, g.wu, full["d_gate"], full["d_up"], None, dwg, dwu, ws)
    torch.cuda.synchronize()
    assert torch.equal(dx, full["dx"]) and torch.equal(dwg, full["dw_gate"]) and torch.equal(dwu, full["dw_up"])


@pytest.mark.parametrize("rows,k,n", [(5, 96, 72), (150, 264, 136)])
def test_gradients_against_differences(rows, k, n):
    """The kernels' gradients along random directions against central
    differences of the FP64 forward definition. The directional derivative of
    a gradient g along d is off by at most 3 u sum |g_i d_i| through g's
    roundings, in the RMS 3 u sqrt(sum (g_i d_i)^2); eight of those are
    allowed, and the differences' own error with a step of 2^-10 is below."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    g = kit.GatedCase(rows, k, n, "gelu_tanh", HF, seed=13)
    ln = kit.LinearCase(rows, k, n, "gelu", HF, residual=False, seed=13)
    got_g, got_l = run_gated(g), run_linear(ln)

    def gated_loss(x, wg, wu):
        return (kit.ACT[g.act](x @ wg) * (x @ wu) * g.dh.double()).sum()

    def linear_loss(x, w, b):
        return (kit.ACT[ln.act](x @ w + b) * ln.dy.double()).sum()

    for loss, base, grads in (
            (gated_loss, (g.x, g.wg, g.wu), [got_g[i] for i in ("dx", "dw_gate", "dw_up")]),
            (linear_loss, (ln.x, ln.w, ln.bias), [got_l[i] for i in ("dx", "dw", "dbias")])):
        base = [t.double() for t in base]
        for i, grad in enumerate(grads):
            # each coordinate moves on its own scale
            d = torch.randn(base[i].shape, generator=gen, device="cuda", dtype=torch.float64) * base[i].std()
            h = 2.0 ** -10
            hi, lo = (loss(*[t + s * h * d if j == i else t for j, t in enumerate(base)]) for s in (1, -1))
            num = float((hi - lo) / (2 * h))
            ana = float((grad.double() * d).sum())
            scale = float((grad.double() * d).square().sum().sqrt())
            assert abs(num - ana) <= 8 * 3 * kit.UNIT[HF] * scale, (i, num, ana, scale)


@pytest.mark.parametrize("rows,k,n", [(1, 3584, 512), (20, 1024, 520), (150, 264, 520), (333, 101, 77),
                                      (600, 520, 776)])
def test_repeatable_and_in_a_graph(rows, k, n):
    """The same bits on every call, on another stream with a workspace of its
    own, and from a graph replayed with new inputs and other work between."""
    log(f"graph {rows}x{k}x{n}")
    c = kit.GatedCase(rows, k, n, "silu", BF, seed=14)
    lc = kit.LinearCase(rows, k, n, "silu", BF, seed=14)
    plan = block.GatedPlan(rows + 5, k, n, training=True)
    lplan = block.LinearPlan(rows + 5, k, n, "silu", training=True)
    ws, lws = plan.new_workspace(), lplan.new_workspace()
    first, lfirst = run_gated(c, plan=plan, ws=ws), run_linear(lc, plan=lplan, ws=lws)
    for _ in range(3):
        again, lagain = run_gated(c, plan=plan, ws=ws), run_linear(lc, plan=lplan, ws=lws)
        assert all(torch.equal(again[i], first[i]) for i in first)
        assert all(torch.equal(lagain[i], lfirst[i]) for i in lfirst)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        again = run_gated(c, plan=plan, ws=plan.new_workspace())
    assert all(torch.equal(again[i], first[i]) for i in first)
    x, dh = c.x.clone(), c.dh.clone()
    buf = {i: torch.empty_like(t) for i, t in first.items()}
    lbuf = {i: torch.empty_like(t) for i, t in lfirst.items()}
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block.gated(plan, x, c.wg, c.wu, buf["h"], ws, buf["d_gate"], buf["d_up"])
        block.gated_backward(plan, dh, x, c.wg, c.wu, buf["d_gate"], buf["d_up"], buf["dx"], buf["dw_gate"],
                             buf["dw_up"], ws)
        block.linear(lplan, x, lc.w, lbuf["y"], lws, lc.bias, lc.residual, lbuf["slope"])
        block.linear_backward(lplan, dh, x, lc.w, lbuf["slope"], lbuf["dx"], lbuf["dw"], lbuf["dbias"], lws)
    for seed in (31, 32, 33, 34):
        m = kit.GatedCase(rows, k, n, "silu", BF, seed=seed)
        m.wg, m.wu = c.wg, c.wu
        x.copy_(m.x)
        dh.copy_(m.dh)
        graph.replay()
        torch.cuda.synchronize()
        ref = run_gated(m, plan=plan, ws=ws)
        assert all(torch.equal(buf[i], ref[i]) for i in ref), seed
        lc.x, lc.dy = m.x, m.dh
        ref = run_linear(lc, plan=lplan, ws=lws)
        assert all(torch.equal(lbuf[i], ref[i]) for i in ref), seed


def test_refusals():
    c = kit.GatedCase(8, 64, 72, "silu", BF, seed=1)
    plan = block.GatedPlan(8, 64, 72)
    ws = plan.new_workspace()
    h = torch.empty(8, 72, dtype=BF, device="cuda")

    def fwd(err, **kw):
        a = dict(x=c.x, w_gate=c.wg, w_up=c.wu, h=h, workspace=ws)
        a.update(kw)
        with pytest.raises(err) as e:
            block.gated(plan, **a)
        return getattr(e.value, "status", None)

    fwd(TypeError, x=c.x.half())
    fwd(ValueError, x=c.x.cpu())
    fwd(ValueError, w_gate=c.wg.t())
    fwd(ValueError, w_up=c.wu[:, :64])
    fwd(ValueError, x=c.x.t().contiguous().t())
    fwd(ValueError, h=h[:7])
    fwd(ValueError, workspace=ws[:128])
    assert fwd(route.RouteError, d_gate=torch.empty_like(h)) == route.E_ARG
    assert fwd(route.RouteError, rows=-1) == route.E_ROWS
    big = kit.GatedCase(9, 64, 72, "silu", BF, seed=1)
    assert fwd(route.RouteError, x=big.x, h=torch.empty(9, 72, dtype=BF, device="cuda")) == route.E_ROWS
    # a forward-only plan has no backward
    with pytest.raises(route.RouteError) as e:
        block.gated_backward(plan, c.dh, c.x, c.wg, c.wu, h, h, c.x.clone(), None, None, ws)
    assert e.value.status == route.E_ARG
    lplan = block.LinearPlan(8, 64, 72, "silu", training=True)
    lws = lplan.new_workspace()
    lc = kit.LinearCase(8, 64, 72, "silu", BF, seed=1)
    for args in ((None, c.x.clone(), None, None), (h, None, None, None)):  # no slope; nothing asked for
        with pytest.raises(route.RouteError) as e:
            block.linear_backward(lplan, lc.dy, lc.x, lc.w, *args, lws)
        assert e.value.status == route.E_ARG
    s = torch.cuda.current_stream().cuda_stream or None
    px, pw, pu, ph, pws = (t.data_ptr() for t in (c.x, c.wg, c.wu, h, ws))
    call = block.LIB.block_gated
    assert call(plan.handle, px, 63, pw, pu, ph, 72, None, None, pws, 8, s) == route.E_SHAPE
    assert call(plan.handle, px, 64, pw, pu, ph, block.MAX_STRIDE + 1, None, None, pws, 8, s) == route.E_SHAPE
    assert call(plan.handle, px + 1, 64, pw, pu, ph, 72, None, None, pws, 8, s) == route.E_ALIGN
    assert call(plan.handle, px, 64, pw, pu, ph, 72, None, None, pws + 16, 8, s) == route.E_ALIGN
    assert call(plan.handle, None, 64, pw, pu, ph, 72, None, None, pws, 8, s) == route.E_ARG
    assert call(plan.handle, px, 64, pw, None, ph, 72, None, None, pws, 8, s) == route.E_ARG
