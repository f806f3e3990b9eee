"""The routed half of a layer together (examples/routed_layer.py): a serving
round behind the route, a training step with every gradient, HIP graphs, two
streams, other streams than the current one, and workspaces with guards."""
import importlib.util
import os

import pytest
import torch

from tests import expertskit as kit
from tests.routekit import log

pytestmark = pytest.mark.gpu

experts = pytest.importorskip("latent_projection_top_amd.experts")
from latent_projection_top_amd import route  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BF = torch.bfloat16


def example():
    spec = importlib.util.spec_from_file_location("routed_layer", os.path.join(ROOT, "examples", "routed_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def rel(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


def routed(rows, topk, total, seed):
    ids = kit.choices(rows, topk, total, seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.rand(rows, topk, generator=gen, device="cuda") + 0.1
    return ids, w / w.sum(1, keepdim=True)


def reference(x, ids, weights, residual, p, first):
    """FP64, with the one rounding that the 8-bit products start from: rows and
    channels as integers, h in BF16 between the two products."""
    q, s = kit.quantised(x)
    y = residual.double().clone()
    count = p["w_gate"].shape[0]
    mats = {}
    for k, v in p.items():
        mats[k] = []
        for e in range(count):
            wq, ws = kit.quantised(v[e].t())
            mats[k].append((wq * ws).t())
    for e in range(count):
        at = (ids == first + e).nonzero()
        r, j = at[:, 0], at[:, 1]
        if r.numel() == 0:
            continue
        xe = q[r] * s[r]
        g, u = torch.mm(xe, mats["w_gate"][e]), torch.mm(xe, mats["w_up"][e])
        hq, hs = kit.quantised((g * torch.sigmoid(g) * u).to(BF))
        y.index_add_(0, r, weights[r, j].double()[:, None] * torch.mm(hq * hs, mats["w_down"][e]))
    return y


@pytest.mark.parametrize("rows,topk,total,count,first", [(1, 16, 896, 896, 0), (8, 16, 896, 56, 112), (20, 16, 896, 112, 0),
                                                         (300, 6, 40, 20, 20), (700, 2, 3, 3, 0)])
def test_serving_round(rows, topk, total, count, first):
    """y's change goes through h (BF16, then integers: where h falls on the
    other side of a rounding, its integer moves by up to one of 127), ys and y,
    each off by at most 2^-8 of its values: 4 x 2^-8 of the change bounds them
    in the RMS, with y's own rounding. A HIP graph of the round gives the same
    bits at every replay, with changing inputs."""
    log(f"serving round {rows}x{topk} {count}/{total}")
    ex = example()
    k, inner, n = 320, 96, 384
    p = ex.matrices(count, k, inner, n)
    step = ex.RoutedRound(rows, topk, p, first)
    gen = torch.Generator(device="cuda").manual_seed(rows)

    def inputs(seed):
        ids, w = routed(rows, topk, total, seed)
        x = torch.randn(rows, k, generator=gen, device="cuda").to(BF)
        return x, ids, w, torch.randn(rows, n, generator=gen, device="cuda").to(BF)

    sets = [inputs(seed) for seed in (1, 2, 3)]
    want = []
    for x, ids, w, y0 in sets:
        y = y0.clone()
        step(x, ids, w, y)
        torch.cuda.synchronize()
        ref = reference(x, ids, w, y0, p, first)
        change = (ref - y0.double()).norm()
        assert (y.double() - ref).norm() <= 2.0 ** -8 * (4 * change + ref.norm())
        want.append(y)
    buf = [t.clone() for t in sets[0]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(*buf)
    for i in (0, 1, 2, 1, 0):
        for b, t in zip(buf, sets[i]):
            b.copy_(t)
        torch.relu(sets[i][0].float()).sum()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf[3], want[i]), i


def test_behind_the_route():
    """ids and weights as route.topk16 gives them, its 896 experts split over
    ranks: the ranks' shares add up to the whole layer, exactly as sorted."""
    log("behind the route")
    rows = 20
    plan = route.Plan(route.MODE_DECODE, rows)
    logits = torch.randn(rows, route.EXPERTS, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    ids = torch.empty(rows, route.TOPK, dtype=torch.int32, device="cuda")
    weights = torch.empty(rows, route.TOPK, device="cuda")
    route.topk16(plan, logits, ids, weights)
    kept = 0
    for ranks in (8, 16):
        _, share = route.RANK_SHARES[ranks]
        kept = 0
        for rank in range(ranks):
            s = experts.SortPlan(rows, route.TOPK, share, first=rank * share)
            offsets = torch.empty(share + 1, dtype=torch.int32, device="cuda")
            place, token = torch.empty_like(ids), torch.empty(ids.numel(), dtype=torch.int32, device="cuda")
            experts.sort(s, ids, offsets, place, token, s.new_workspace())
            torch.cuda.synchronize()
            kept += int(offsets[-1])
            mine = (ids >= rank * share) & (ids < (rank + 1) * share)
            assert torch.equal(place >= 0, mine)
        assert kept == ids.numel()


def test_training_step():
    """Every gradient against autograd in FP64: a chain of at most eight
    roundings on the way to dx (h, its saved derivative, ys, dys, dh, dg and
    du, dxs, dx), 8 x 2^-8 in the RMS, and no more for the others. An expert
    without rows gets zero gradients."""
    log("training step")
    ex = example()
    rows, topk, count, k, inner, n = 200, 3, 6, 264, 72, 200
    p = ex.matrices(count, k, inner, n, seed=2)
    step = ex.RoutedTraining(rows, topk, p, first=1)
    ids, w = routed(rows, topk, 9, 3)
    ids = torch.where(ids == 4, torch.full_like(ids, 8), ids)  # expert 4 - first has none
    gen = torch.Generator(device="cuda").manual_seed(4)
    x, res, dy = (torch.randn(rows, m, generator=gen, device="cuda").to(BF) for m in (k, n, n))
    y = step.forward(x, ids, w, res, p)
    dx, dw, grads = step.backward(dy, w, p)
    torch.cuda.synchronize()
    q = {i: v.double().requires_grad_() for i, v in p.items()}
    xd, wd = x.double().requires_grad_(), w.double().requires_grad_()
    out = res.double()
    for e in range(count):
        at = (ids == 1 + e).nonzero()
        r, j = at[:, 0], at[:, 1]
        g, u = torch.mm(xd[r], q["w_gate"][e]), torch.mm(xd[r], q["w_up"][e])
        out = out.index_add(0, r, wd[r, j][:, None] * torch.mm(g * torch.sigmoid(g) * u, q["w_down"][e]))
    want = torch.autograd.grad(out, [xd, wd] + list(q.values()), dy.double())
    assert rel(y, out.detach()) <= 4 * 2.0 ** -8
    assert rel(dx, want[0]) <= 8 * 2.0 ** -8
    assert rel(dw, want[1]) <= 4 * 2.0 ** -8
    for i, ref in zip(q, want[2:]):
        assert rel(grads[i], ref) <= 8 * 2.0 ** -8, i
        assert (grads[i][3] == 0).all()


def test_example_runs(capsys):
    log("example")
    example().main()
    out = capsys.readouterr().out
    assert "serving round" in out and "training step" in out


@pytest.mark.parametrize("rows,topk,total", [(8, 16, 896), (600, 6, 40)])
def test_two_streams(rows, topk, total):
    """Two streams with their own workspaces and changing inputs: the bits of
    the same calls alone; the zeroed parts are zero afterwards."""
    log(f"two streams {rows}")
    ex = example()
    k, inner, n = 256, 64, 128
    sides = []
    for seed in (1, 2):
        p = ex.matrices(total, k, inner, n, seed=seed)
        step = ex.RoutedRound(rows, topk, p)
        gen = torch.Generator(device="cuda").manual_seed(seed)
        sets = [(torch.randn(rows, k, generator=gen, device="cuda").to(BF), *routed(rows, topk, total, 10 * seed + i))
                for i in range(3)]
        want = []
        for x, ids, w in sets:
            y = torch.zeros(rows, n, dtype=BF, device="cuda")
            step(x, ids, w, y)
            want.append(y)
        sides.append((step, sets, want, [torch.zeros(rows, n, dtype=BF, device="cuda") for _ in range(12)],
                      torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i in range(12):
        for step, sets, _, outs, stream in sides:
            with torch.cuda.stream(stream):
                step(*sets[i % 3], outs[i])
    torch.cuda.synchronize()
    for step, _, want, outs, _ in sides:
        for i in range(12):
            assert torch.equal(outs[i], want[i % 3]), i
        for ws in step.ws[1:]:
            assert not ws[:experts.WORKSPACE_ZEROED].any()


@pytest.mark.parametrize("planes,rows,counts", [(1, 8, None), (2, 1, None), (1, 300, None), (2, 0, [3, 40, 0, 300]),
                                                (1, 0, [1] * 30)])
def test_workspaces_are_as_large_as_asked_for(planes, rows, counts):
    """Guards around the workspace; the same bits whatever its bytes hold
    beyond the zeroed part."""
    log(f"workspace {planes} {rows}")
    c = kit.ProductCase(planes, 1000, 264, "silu", BF, rows=rows, counts=counts, tokens=0, seed=1)
    plan = c.plan(experts)
    packed = experts.pack(plan, *c.w)
    outs = []
    for fill in (0, 255):
        buf = torch.full((plan.workspace_bytes + 512,), fill, dtype=torch.uint8, device="cuda")
        ws = buf[256:256 + plan.workspace_bytes]
        ws[:experts.WORKSPACE_ZEROED] = 0
        buf[:256], buf[256 + plan.workspace_bytes:] = 91, 91
        y = torch.empty(c.rows, c.n, dtype=BF, device="cuda")
        for _ in range(2):
            c.run(experts, plan, packed, y, ws)
        torch.cuda.synchronize()
        assert (buf[:256] == 91).all() and (buf[256 + plan.workspace_bytes:] == 91).all()
        assert not ws[:experts.WORKSPACE_ZEROED].any()
        outs.append(y)
    assert torch.equal(*outs)


@pytest.mark.parametrize("rows,topk,count", [(1, 16, 896), (3000, 16, 896)])
def test_sort_workspace_may_hold_anything(rows, topk, count):
    log(f"sort workspace {rows}")
    plan = experts.SortPlan(rows, topk, count)
    ids = kit.choices(rows, topk, count, seed=5)
    offsets, place, token = kit.sort_reference(ids, count)
    for fill in (0, 255, 17):
        buf = torch.full((plan.workspace_bytes + 512,), fill, dtype=torch.uint8, device="cuda")
        buf[:256], buf[-256:] = 91, 91
        out = [torch.empty(s, dtype=torch.int32, device="cuda") for s in ((count + 1,), (rows, topk), (rows * topk,))]
        for _ in range(2):
            experts.sort(plan, ids, *out, buf[256:-256])
        torch.cuda.synchronize()
        assert (buf[:256] == 91).all() and (buf[-256:] == 91).all()
        for got, want in zip(out, (offsets, place, token)):
            assert (got.cpu().numpy() == want).all()
