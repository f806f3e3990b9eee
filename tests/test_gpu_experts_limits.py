"""The routed half of a layer where sizes choose another way through the
kernels, past 32 bits and past one grid's threads, on streams and in graphs."""
import pytest
import torch

from tests import blockkit as bk
from tests import expertskit as kit
from tests.routekit import log

pytestmark = pytest.mark.gpu

experts = pytest.importorskip("latent_projection_top_amd.experts")

BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("planes,act,tokens,dtype", [(1, "none", 0, BF), (1, "gelu", 77, HF), (2, "silu", 400, BF)])
def test_weights_past_the_last_cache(planes, act, tokens, dtype):
    """More than 256 MB of them: short experts are streamed by a kernel of their
    own, the others are tiles."""
    log(f"large weights {planes}")
    counts = [0, 1, 17, 32, 33, 64, 65, 200, 0, 256, 257, 300, 16, 31, 0, 2]
    counts += [0] * ((66 if planes == 1 else 34) - len(counts) - 1) + [5]
    kit.ProductCase(planes, 2048, 2040, act, dtype, counts=counts, tokens=tokens, bias=planes == 1,
                    residual=planes == 1, seed=1, spare=5).check(experts, "large")


@pytest.mark.parametrize("planes,act,tokens", [(1, "silu", 0), (2, "gelu", 900)])
def test_many_rows_of_weights_past_the_last_cache(planes, act, tokens):
    """The same with more than 24 rows to an expert on average."""
    log(f"large weights, many rows {planes}")
    counts = [1, 0, 2, 31, 32, 33, 700, 17, 16, 1200, 0, 128, 129, 9, 600]
    counts += [0] * ((66 if planes == 1 else 34) - len(counts) - 1) + [60]
    kit.ProductCase(planes, 2048, 2040, act, BF, counts=counts, tokens=tokens, bias=planes == 1,
                    residual=planes == 1, seed=3, spare=5).check(experts, "large")


@pytest.mark.parametrize("counts", [[24], [5, 19, 0, 40], [16] * 32, [17] * 30, [0, 50] * 10, [24] * 20,
                                    [100] + [1] * 40, [513] + [0] * 30, [33, 65, 97, 129] + [0] * 20])
@pytest.mark.parametrize("k", [520, 2048, 2056])
def test_experts_of_few_rows_on_average(counts, k):
    """Some of them with more than an item's: they become several."""
    log(f"brief {counts} {k}")
    for planes, act in ((1, "none"), (2, "silu")):
        kit.ProductCase(planes, k, 72, act, BF, counts=counts, tokens=99, seed=k).check(experts, f"{counts}")


@pytest.mark.parametrize("planes,act", [(1, "relu"), (2, "gelu_tanh")])
def test_many_rows_of_small_experts(planes, act):
    """Enough rows for tiles: short experts follow them in the same launch."""
    log(f"together {planes}")
    counts = [0, 1, 32, 33, 64, 400, 2000, 257, 31, 0, 3, 1500, 700, 512, 513, 2300, 9, 0, 1900, 255, 20, 19, 1200, 17]
    kit.ProductCase(planes, 863, 368, act, BF, counts=counts, tokens=5000, residual=planes == 1, seed=2,
                    spare=7).check(experts, "together")


@pytest.mark.parametrize("counts", [[20], [30, 0], [9, 8, 0], [0, 25, 1], [32]])
@pytest.mark.parametrize("planes,act", [(1, "silu"), (2, "relu")])
def test_few_rows_of_few_experts(counts, planes, act):
    log(f"few of few {counts}")
    kit.ProductCase(planes, 1030, 200, act, HF, counts=counts, tokens=11, seed=3).check(experts, f"{counts}")


@pytest.mark.parametrize("rows,counts", [(1, None), (20, None), (40, None), (300, None), (1500, None),
                                         (0, [3, 0, 40, 300]), (0, [1] * 30), (0, [600, 700, 33, 2])])
def test_residual_is_the_output(rows, counts):
    """y += the product: the same bits as with a residual of its own."""
    log(f"in place {rows} {counts}")
    c = kit.ProductCase(1, 704, 536, "gelu", BF, rows=rows, counts=counts, residual=True, bias=True, seed=4)
    plan = c.plan(experts)
    packed, ws = experts.pack(plan, *c.w), plan.new_workspace()
    want, got = torch.empty_like(c.residual), c.residual.clone()
    c.run(experts, plan, packed, want, ws)
    c.residual = got
    c.run(experts, plan, packed, got, ws)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_packed_weights_past_32_bits():
    """4.7 GB of them: rows of the last experts."""
    log("packed 64-bit")
    k = n = 8192
    e = 70
    counts = [2] + [0] * (e - 4) + [0, 3, 40]
    c = kit.ProductCase(1, 64, 32, "none", BF, counts=counts, seed=5)  # (offsets, token and shapes)
    gen = torch.Generator(device="cuda").manual_seed(6)
    c.k, c.n = k, n
    c.x = torch.randn(c.rows, k, generator=gen, device="cuda").to(BF)
    c.w = [torch.randint(-128, 128, (e, k, n), generator=gen, device="cuda", dtype=torch.int8)]
    c.scale = [(torch.rand(e, n, generator=gen, device="cuda") + 0.5) / (74 * k ** 0.5)]
    c.check(experts, "64-bit")


def test_more_rows_than_one_grid_dimension():
    """A wave for each 512 columns makes more than 2^32 threads."""
    log("rows grid")
    rows, width = (1 << 18) + 1, 131072  # 69 GB
    x = torch.empty(rows, width, dtype=BF, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(7)
    x[0], x[-1] = (torch.randn(width, generator=gen, device="cuda").to(BF) for _ in range(2))
    place = torch.full((rows, 1), -1, dtype=torch.int32, device="cuda")
    place[0], place[-1] = 1, 0
    xs = torch.empty(2, width, dtype=BF, device="cuda")
    plan = experts.CombinePlan(rows, 1, width)
    experts.gather(plan, x, place, xs)
    torch.cuda.synchronize()
    assert torch.equal(xs[1], x[0]) and torch.equal(xs[0], x[-1])
    x.fill_(7)
    experts.gather_backward(plan, xs, place, x)
    torch.cuda.synchronize()
    assert torch.equal(xs[1], x[0]) and torch.equal(xs[0], x[-1])
    for part in x[1:-1].split(1 << 14):
        assert not part.any()
    del x, part
    torch.cuda.empty_cache()


def test_more_tokens_than_one_grid_dimension():
    """A block of 1024 threads for each row of x makes more than 2^32 threads."""
    log("tokens grid")
    k, rows, tokens = 8193, 40, (1 << 22) + 1  # 69 GB
    c = kit.ProductCase(1, k, 16, "none", BF, rows=rows, seed=8)
    plan = experts.Linear8Plan(rows, k, 16, tokens=tokens)
    token = torch.randint(1, tokens - 1, (rows,), generator=torch.Generator().manual_seed(9)).unique()
    assert token.numel() == rows
    token[0], token[-1] = 0, tokens - 1
    x = torch.empty(tokens, k, dtype=BF, device="cuda")
    x[token.cuda()] = c.x
    y = torch.empty(rows, 16, dtype=BF, device="cuda")
    experts.linear8(plan, x, experts.pack(plan, *c.w), c.scale[0], y, plan.new_workspace(),
                    token=token.to(torch.int32).cuda())
    torch.cuda.synchronize()
    ref, bound = c.reference()
    bk.check(y, ref, bound, None, BF, "tokens")
    del x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("planes,rows,k,n", [(1, 8, 8192, 40), (1, 30, 16384, 130), (2, 3, 7000, 24)])
def test_split_sums_on_two_streams(planes, rows, k, n):
    """Long reductions of few columns, whose parts several blocks add up: the
    bits of the calls alone, with other inputs from call to call, while another
    stream does the same in a workspace of its own."""
    log(f"split {planes} {rows}x{k}x{n}")
    sides = []
    for seed in (1, 2):
        c = kit.ProductCase(planes, k, n, "silu", BF, rows=rows, seed=seed)
        plan = c.plan(experts)
        packed, ws = experts.pack(plan, *c.w), plan.new_workspace()
        xs = [c.x, c.x.flip(0).contiguous(), (c.x.float() * 0.37).to(BF)]
        want = []
        for x in xs:
            c.x = x
            want.append(torch.empty(rows, n, dtype=BF, device="cuda"))
            c.run(experts, plan, packed, want[-1], ws)
        c.x = xs[0]
        ref, bound = c.reference()
        torch.cuda.synchronize()
        bk.check(want[0], ref, bound, None, BF, "alone")
        outs = [torch.empty_like(want[0]) for _ in range(24)]
        sides.append((c, plan, packed, ws, xs, want, outs, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for i in range(24):
        for c, plan, packed, ws, xs, _, outs, stream in sides:
            c.x = xs[i % 3]
            c.run(experts, plan, packed, outs[i], ws, stream=stream)
    torch.cuda.synchronize()
    for *_, want, outs, _ in sides:
        for i in range(24):
            assert torch.equal(outs[i], want[i % 3]), i


def test_training_calls_in_a_graph():
    """Sort, gather, combine and their gradients captured together: every replay,
    with other inputs and eager work in between, gives the eager bits."""
    log("graph of rows")
    rows, topk, width, total = 200, 3, 328, 11
    cases = [kit.RowsCase(rows, topk, width, total, total, BF, seed=s) for s in (1, 2, 3)]
    sort = experts.SortPlan(rows, topk, total)
    plan = experts.CombinePlan(rows, topk, width)
    ws = sort.new_workspace()
    offsets = torch.empty(total + 1, dtype=torch.int32, device="cuda")
    token = torch.empty(rows * topk, dtype=torch.int32, device="cuda")

    def step(ids, x, ys, w, res, dy, dxs):
        place = torch.empty_like(ids)
        xs, dys, y, dx = torch.zeros_like(ys), torch.zeros_like(ys), torch.empty_like(x), torch.empty_like(x)
        dw = torch.empty_like(w)
        experts.sort(sort, ids, offsets, place, token, ws)
        experts.gather(plan, x, place, xs)
        experts.combine(plan, ys, place, w, y, residual=res)
        experts.combine_backward(plan, dy, ys, place, w, dys, dw)
        experts.gather_backward(plan, dxs, place, dx)
        return place, xs, y, dys, dw, dx

    def inputs(c):
        return c.ids, c.x, c.ys, c.weights, c.residual, c.dy, c.dxs

    want = [step(*inputs(c)) for c in cases]
    torch.cuda.synchronize()
    buf = [t.clone() for t in inputs(cases[0])]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step(*buf)
    for i in (0, 1, 2, 0, 2):
        for b, t in zip(buf, inputs(cases[i])):
            b.copy_(t)
        torch.relu(cases[i].x.float()).sum()
        graph.replay()
        torch.cuda.synchronize()
        for g, t in zip(got, want[i]):
            assert torch.equal(g, t), i


def test_weights_made_on_another_stream():
    """quantize and pack with a stream: what they return is that stream's
    memory, which the current one does not hand out again while it is in use."""
    log("weights on a stream")
    gen = torch.Generator(device="cuda").manual_seed(10)
    w = torch.randn(3, 500, 264, generator=gen, device="cuda").to(BF)
    plan = experts.Linear8Plan(4, 500, 264, experts=3)
    w8, scale = experts.quantize(plan, w)
    packed = experts.pack(plan, w8)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    w8_s, scale_s = experts.quantize(plan, w, stream=stream)
    packed_s = experts.pack(plan, w8_s, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(w8, w8_s) and torch.equal(scale, scale_s) and torch.equal(packed, packed_s)
    at = packed_s.data_ptr()
    del packed_s
    assert torch.empty(plan.packed_bytes, dtype=torch.uint8, device="cuda").data_ptr() != at
    at = w8_s.data_ptr()
    del w8_s
    assert torch.empty_like(w8).data_ptr() != at


@pytest.mark.parametrize("rows,topk,experts_,first", [(32768, 16, 900, 0), (32769, 16, 900, 3), (40000, 16, 3000, 500),
                                                      (1 << 20, 16, 4096, 0)])
def test_sort_of_many_choices(rows, topk, experts_, first):
    """On both sides of where it takes more blocks, and the most choices."""
    log(f"sort {rows}x{topk} {experts_}")
    ids = torch.randint(0, 4096, (rows, topk), generator=torch.Generator().manual_seed(rows), dtype=torch.int32).cuda()
    plan = experts.SortPlan(rows, topk, experts_, first=first)
    capacity = rows * topk - 5
    out = [torch.empty(s, dtype=torch.int32, device="cuda") for s in ((experts_ + 1,), (rows, topk), (capacity,))]
    ws = plan.new_workspace()
    for _ in range(2):
        experts.sort(plan, ids, *out, ws)
    torch.cuda.synchronize()
    offsets, place, token = kit.sort_reference(ids, experts_, first, capacity)
    assert (out[0].cpu().numpy() == offsets).all() and (out[1].cpu().numpy() == place).all()
    assert (out[2].cpu().numpy()[:token.size] == token).all()


def test_graphs_that_share_a_workspace():
    """Calls of 8, 40 and 300 rows of one plan, captured into a graph each with
    the same workspace and replayed in turn, eager calls in between."""
    log("graphs, one workspace")
    c = kit.ProductCase(1, 8192, 136, "gelu", BF, rows=300, bias=True, residual=True, seed=11)
    plan = c.plan(experts)
    packed, ws = experts.pack(plan, *c.w), plan.new_workspace()
    ref, bound = c.reference()
    graphs = []
    for rows in (8, 40, 300):
        y = torch.zeros(300, 136, dtype=BF, device="cuda")
        c.run(experts, plan, packed, y, ws, rows=rows)
        torch.cuda.synchronize()
        bk.check(y[:rows], ref[:rows], bound[:rows], None, BF, f"{rows} rows")
        got = torch.zeros_like(y)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            c.run(experts, plan, packed, got, ws, rows=rows)
        graphs.append((graph, got, y))
    eager = torch.empty_like(y)
    for i in (0, 1, 2, 0, 0, 2, 1):
        graph, got, want = graphs[i]
        got.zero_()
        graph.replay()
        c.run(experts, plan, packed, eager, ws, rows=20)
        torch.cuda.synchronize()
        assert torch.equal(got, want), i
    assert not ws[:experts.WORKSPACE_ZEROED].any()


@pytest.mark.parametrize("counts,spare", [([3, 0, 9, 1], 20), ([30, 2, 0, 7] * 8, 1), ([30, 2, 0, 7] * 8, 3000),
                                          ([200, 0, 33, 300], 5000), ([0, 0, 0], 4000)])
def test_rows_behind_the_last_experts(counts, spare):
    """A rank's share of the choices: most rows are nobody's, whatever they and
    the workspace hold."""
    log(f"spare {counts} {spare}")
    for k, n in ((330, 90), (2100, 264)):
        c = kit.ProductCase(1, k, n, "silu", BF, counts=counts, bias=True, residual=True, seed=12, spare=spare)
        c.x[c.kept:] = float("nan")
        plan = c.plan(experts)
        packed, ws = experts.pack(plan, *c.w), plan.new_workspace()
        ws[experts.WORKSPACE_ZEROED:] = 255
        y = torch.full((c.rows, n), 7.0, dtype=BF, device="cuda")
        c.run(experts, plan, packed, y, ws)
        torch.cuda.synchronize()
        ref, bound = c.reference()
        bk.check(y[:c.kept], ref, bound, None, BF, "kept rows")
        assert (y[c.kept:] == 7).all()
