"""The layer's operators together (examples/latent_layer.py): a decode round
around the route and a training step, against FP64 compositions; workspaces
that are exactly as large as asked for, with guards around every buffer;
matrices whose offsets pass 32 bits."""
import importlib.util
import os

import pytest
import torch

from tests import blockkit as kit
from tests.routekit import log, weights_dev

pytestmark = pytest.mark.gpu

block = pytest.importorskip("latent_projection_top_amd.block")
from latent_projection_top_amd import route  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF, HF = torch.bfloat16, torch.float16


def example():
    spec = importlib.util.spec_from_file_location("latent_layer",
                                                  os.path.join(ROOT, "examples", "latent_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def norm64(x, p):
    m = x.mean(1, keepdim=True)
    return (x - m) / torch.sqrt((x - m).square().mean(1, keepdim=True) + 1e-5) * p["norm_w"].double() + \
        p["norm_b"].double()


def rel(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


@pytest.mark.parametrize("rows", (1, 8, 20))
def test_decode_round(rows):
    """Each BF16 step of the round (norm, latent, h, y) rounds once, with an
    RMS of at most 2^-8 / sqrt(3) of its values; the layer's share of y goes
    through four of them and products that carry a relative error through
    unchanged in the RMS: 4 x 2^-8 bounds it. The same round from a HIP graph
    gives the same bits."""
    ex = example()
    w, wr = weights_dev(0)
    p = ex.weights(route.LATENT, 1024, route.HIDDEN)
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x0 = torch.randn(rows, route.HIDDEN, generator=gen, device="cuda").to(BF)
    step = ex.DecodeRound(rows, 1024)
    x = x0.clone()
    step(x, w, wr, p)
    torch.cuda.synchronize()
    latent = norm64(x0.double(), p) @ w.double()
    g, u = latent @ p["w_gate"].double(), latent @ p["w_up"].double()
    add = (g * torch.sigmoid(g) * u) @ p["w_down"].double()
    assert rel(step.latent, latent) <= 2 * 2.0 ** -8
    err = (x.double() - (x0.double() + add)).norm()
    assert err <= 2.0 ** -8 * (4 * add.norm() + x0.double().norm())
    # the experts are those of the route on the normalised rows
    plan = route.Plan(route.MODE_DECODE, rows)
    ids, wts = torch.empty_like(step.ids), torch.empty_like(step.weights)
    route.fused(plan, step.xn, w, wr, torch.empty_like(step.latent), torch.empty_like(step.logits), ids, wts,
                plan.new_workspace())
    torch.cuda.synchronize()
    assert torch.equal(ids, step.ids) and torch.equal(wts, step.weights)
    graph = torch.cuda.CUDAGraph()
    buf = x0.clone()
    with torch.cuda.graph(graph):
        step(buf, w, wr, p)
    for _ in range(4):
        buf.copy_(x0)
        torch.relu(x0.float()).sum()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf, x)


def test_train_step():
    """Gradients of the composed step against autograd in FP64: a chain of at
    most six roundings on the way to dx (h, dh, dg and du through the saved
    derivatives, dxn, dx), 6 x 2^-8 in the RMS, and no more for the others."""
    ex = example()
    rows, inner = 96, 264
    p = ex.weights(route.HIDDEN, inner, route.HIDDEN, seed=3)
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn(rows, route.HIDDEN, generator=gen, device="cuda").to(BF)
    dy = torch.randn(rows, route.HIDDEN, generator=gen, device="cuda").to(BF)
    step = ex.TrainStep(rows, inner)
    y = step.forward(x, p)
    dx, grads = step.backward(x, dy, p)
    torch.cuda.synchronize()
    q = {k: v.double().requires_grad_() for k, v in p.items()}
    xd = x.double().requires_grad_()
    m = xd.mean(1, keepdim=True)
    xn = (xd - m) / torch.sqrt((xd - m).square().mean(1, keepdim=True) + 1e-5) * q["norm_w"] + q["norm_b"]
    g, u = torch.mm(xn, q["w_gate"]), torch.mm(xn, q["w_up"])
    ref = xd + torch.mm(g * torch.sigmoid(g) * u, q["w_down"])
    want = torch.autograd.grad(ref, [xd] + list(q.values()), dy.double())
    assert rel(y, ref.detach()) <= 6 * 2.0 ** -8
    assert rel(dx, want[0]) <= 6 * 2.0 ** -8
    for k, r in zip(q, want[1:]):
        assert rel(grads[k], r) <= 6 * 2.0 ** -8, k


def test_a_step_lowers_the_loss():
    """A step that the gradient says takes off 5 % of the loss takes off at
    least half of that (the rest is the loss's curvature)."""
    ex = example()
    rows, inner = 64, 128
    p = ex.weights(route.HIDDEN, inner, route.HIDDEN, seed=5)
    step = ex.TrainStep(rows, inner)
    gen = torch.Generator(device="cuda").manual_seed(6)
    x, t = (torch.randn(rows, route.HIDDEN, generator=gen, device="cuda").to(BF) for _ in range(2))
    before, after = (step.descend(x, t, p) for _ in range(2))
    log(f"loss {before} -> {after}")
    assert after <= 0.975 * before


def guarded(nbytes):
    """A zeroed workspace of exactly nbytes inside a buffer of 0xA5."""
    buf = torch.full((nbytes + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    ws = buf[2048:2048 + nbytes]
    assert ws.data_ptr() % 256 == 0
    ws.zero_()
    return ws, buf


def intact(buf, nbytes):
    return bool((buf[:2048] == 0xA5).all()) and bool((buf[2048 + nbytes:] == 0xA5).all())


@pytest.mark.parametrize("rows,k,n", [(1, 100, 36), (1, 4096, 1000), (8, 2048, 7168), (16, 264, 100), (31, 999, 333),
                                      (32, 3584, 512), (33, 1000, 264), (64, 4096, 512), (200, 777, 1001),
                                      (256, 4096, 512), (700, 512, 128), (40, 5, 3), (2, 3, 5)])
def test_workspace_is_enough(rows, k, n):
    """Every call stays inside the bytes its plan asks for, leaves its counters
    at zero, and gives the same bits in a workspace that held other calls."""
    log(f"workspace {rows}x{k}x{n}")
    g = kit.GatedCase(rows, k, n, "silu", BF, seed=1)
    c = kit.LinearCase(rows, k, n, "gelu", BF, seed=2)
    gp, lp = block.GatedPlan(rows, k, n, training=True), block.LinearPlan(rows, k, n, "gelu", training=True)
    results = []
    spaces = [(guarded(gp.workspace_bytes), guarded(lp.workspace_bytes))]
    for again in (False, True):
        (gw, gbuf), (lw, lbuf) = spaces[0]
        o = {i: torch.empty(rows, n, dtype=BF, device="cuda") for i in ("h", "dg", "du", "y", "s")}
        o.update({i: torch.empty(k, n, dtype=BF, device="cuda") for i in ("wg", "wu", "w")})
        o.update({i: torch.empty(rows, k, dtype=BF, device="cuda") for i in ("x1", "x2")})
        o["b"] = torch.empty(n, dtype=BF, device="cuda")
        if again:  # other row counts in between
            for r in {1, max(1, rows // 2)}:
                block.gated(gp, g.x, g.wg, g.wu, o["h"], gw, rows=r)
                block.linear(lp, c.x, c.w, o["y"], lw, rows=r)
        block.gated(gp, g.x, g.wg, g.wu, o["h"], gw, o["dg"], o["du"])
        block.gated_backward(gp, g.dh, g.x, g.wg, g.wu, o["dg"], o["du"], o["x1"], o["wg"], o["wu"], gw)
        block.linear(lp, c.x, c.w, o["y"], lw, c.bias, c.residual, o["s"])
        block.linear_backward(lp, c.dy, c.x, c.w, o["s"], o["x2"], o["w"], o["b"], lw)
        torch.cuda.synchronize()
        assert intact(gbuf, gp.workspace_bytes) and intact(lbuf, lp.workspace_bytes)
        assert not gw[:65536].any() and not lw[:65536].any()  # the counters
        results.append(o)
    for name, t in results[0].items():
        assert torch.equal(t, results[1][name]), name


@pytest.mark.parametrize("rows,width,dtype", [(1, 7168, BF), (5, 64, BF), (300, 1000, HF), (4096, 96, torch.float32),
                                              (1000, 16000, BF), (20, 20000, BF)])
def test_norm_workspace_is_enough(rows, width, dtype):
    c = kit.NormCase(rows, width, dtype, seed=1)
    plan = block.NormPlan(rows, width, dtype=dtype)
    ws, buf = guarded(plan.workspace_bytes)
    y, dx = torch.empty_like(c.x), torch.empty_like(c.x)
    m, r = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    dw, db = torch.empty(width, device="cuda"), torch.empty(width, device="cuda")
    block.layer_norm(plan, c.x, c.weight, c.bias, y, m, r)
    block.layer_norm_backward(plan, c.dy, c.x, c.weight, m, r, dx, dw, db, ws)
    torch.cuda.synchronize()
    assert intact(buf, plan.workspace_bytes)


def test_two_streams_at_once():
    """Calls that overlap in time, each stream with a workspace of its own."""
    c = [kit.GatedCase(12, 2048, 1024, "silu", BF, seed=s) for s in (1, 2)]
    plan = block.GatedPlan(12, 2048, 1024)
    want = []
    for i in range(2):
        h = torch.empty(12, 1024, dtype=BF, device="cuda")
        block.gated(plan, c[i].x, c[i].wg, c[i].wu, h, plan.new_workspace())
        want.append(h)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [plan.new_workspace() for _ in range(2)]
    out = [[torch.empty_like(want[0]) for _ in range(20)] for _ in range(2)]
    torch.cuda.synchronize()
    for k in range(20):
        for i in range(2):
            block.gated(plan, c[i].x, c[i].wg, c[i].wu, out[i][k], ws[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(t, want[i]) for t in out[i])


def sample_rows(rows):
    return torch.tensor([0, 1, rows // 3, rows // 2, rows - 2, rows - 1], device="cuda")


def test_offsets_past_32_bits():
    """x of 2^20 rows x 2056: 2.2 G elements, 4.3 GB. Rows on both sides of
    2^31 elements and 2^32 bytes against FP64; dw adds up all rows, so it is
    checked with rows that are zero but for the sampled ones."""
    rows, k, n = 1 << 20, 2056, 64
    at = torch.unique(torch.cat([sample_rows(rows), torch.tensor([(1 << 31) // k, (1 << 31) // k + 1,
                                                                  (1 << 30) // k], device="cuda")]))
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.zeros(rows, k, dtype=BF, device="cuda")
    x[at] = torch.randn(len(at), k, generator=gen, device="cuda").to(BF)
    w = (torch.randn(k, n, generator=gen, device="cuda") * k ** -0.5).to(BF)
    plan = block.LinearPlan(rows, k, n, training=True)
    ws = plan.new_workspace()
    y = torch.empty(rows, n, dtype=BF, device="cuda")
    block.linear(plan, x, w, y, ws)
    ref = x[at].double() @ w.double()
    bound = (k + 8) * kit.E * (x[at].double().abs() @ w.double().abs())
    kit.check(y[at], ref, bound, ref.abs(), BF, "y")
    assert int((y != 0).any(1).sum()) <= len(at)
    dw = torch.empty(k, n, dtype=BF, device="cuda")
    dx = torch.empty(rows, k, dtype=BF, device="cuda")
    block.linear_backward(plan, y, x, w, None, dx, dw, None, ws)
    torch.cuda.synchronize()
    rw = x[at].double().t() @ y[at].double()
    kit.check(dw, rw, (rows + 8) * kit.E * (x[at].double().abs().t() @ y[at].double().abs()), None, BF, "dw")
    rx = y[at].double() @ w.double().t()
    kit.check(dx[at], rx, (n + 8) * kit.E * (y[at].double().abs() @ w.double().abs().t()), None, BF, "dx")
    del dx
    norm = block.NormPlan(rows, k)
    out = torch.empty_like(x)
    block.layer_norm(norm, x, None, None, out)
    torch.cuda.synchronize()
    xs = x[at].double()
    m = xs.mean(1, keepdim=True)
    ref = (xs - m) / torch.sqrt((xs - m).square().mean(1, keepdim=True) + 1e-5)
    assert rel(out[at], ref) <= 2.0 ** -8
    assert int((out != 0).any(1).sum()) <= len(at)


@pytest.mark.parametrize("rows", (20, 300))
def test_widest_stride(rows):
    """Rows 2^20 elements apart: the last starts past 2^29 bytes."""
    k, n = 264, 136
    buf = torch.full((rows * block.MAX_STRIDE,), float("nan"), dtype=BF, device="cuda")
    x = buf.view(rows, block.MAX_STRIDE)[:, 8:8 + k]
    gen = torch.Generator(device="cuda").manual_seed(2)
    x.copy_(torch.randn(rows, k, generator=gen, device="cuda"))
    w = (torch.randn(k, n, generator=gen, device="cuda") * k ** -0.5).to(BF)
    plan = block.LinearPlan(rows, k, n, training=True)
    ws = plan.new_workspace()
    y, y2 = (torch.empty(rows, n, dtype=BF, device="cuda") for _ in range(2))
    block.linear(plan, x, w, y, ws)
    block.linear(plan, x.contiguous(), w, y2, ws)
    dw, dw2 = (torch.empty(k, n, dtype=BF, device="cuda") for _ in range(2))
    block.linear_backward(plan, y, x, w, None, None, dw, None, ws)
    block.linear_backward(plan, y, x.contiguous(), w, None, None, dw2, None, ws)
    torch.cuda.synchronize()
    assert torch.equal(y, y2) and torch.equal(dw, dw2) and torch.isfinite(dw).all()
