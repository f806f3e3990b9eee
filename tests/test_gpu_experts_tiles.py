"""The tile kernel of the 8-bit products: every body (64, 128, 192 and 256 rows,
with and without other row tiles of the same weights), reductions shorter than
its ring of stages and longer, and what its ending meets. Each test states the
way that the host's rules give its sizes."""
import pytest
import torch

from tests import blockkit as bk
from tests import expertskit as kit
from tests import waykit
from tests.routekit import log

pytestmark = pytest.mark.gpu

experts = pytest.importorskip("latent_projection_top_amd.experts")

BF, HF = torch.bfloat16, torch.float16

# rows and outputs: one row tile of each body, then several (2 x 160, 2 x 250,
# 4 x 224 and 134, 8 x 256 and 2)
DENSE = [(64, 50001), (100, 24995), (180, 16601), (250, 12603), (300, 10603), (500, 6403), (1030, 3203), (2050, 1603)]
INPUTS = [1, 64, 65, 130, 300, 520]  # 1 to 9 stages; a ring holds 5 to 8
LONG = [(64, 2048, 131071), (333, 1019, 20011), (2048, 2050, 3585)]
COUNTS = [40, 64, 100, 128, 180, 192, 250, 256, 300, 513, 0, 1, 32, 33, 20]


def dense_way(planes, rows, k, n):
    return waykit.way(planes, rows, k, n // planes | 1)


@pytest.mark.parametrize("rows,n", DENSE)
@pytest.mark.parametrize("k", INPUTS)
def test_dense(rows, n, k):
    """linear8 with everything in its ending, the types in turn."""
    assert dense_way(1, rows, k, n) == "together"
    log(f"tiles {rows}x{k}x{n}")
    dtype = (BF, HF)[(rows + k) % 2]
    kit.ProductCase(1, k, n, ("gelu", "none")[k % 2], dtype, rows=rows, bias=True, residual=True,
                    seed=rows + k).check(experts, f"{rows}x{k}x{n}")


@pytest.mark.parametrize("rows,n", DENSE)
@pytest.mark.parametrize("k", [1, 130, 520])
def test_dense_gated(rows, n, k):
    assert dense_way(2, rows, k, n) == "together"
    log(f"gated tiles {rows}x{k}x{n}")
    kit.ProductCase(2, k, n // 2 | 1, "silu", (BF, HF)[rows // 2 % 2], rows=rows, seed=rows + k).check(
        experts, f"{rows}x{k}x{n}")


@pytest.mark.parametrize("rows,k,n", LONG)
def test_long_reductions(rows, k, n):
    assert waykit.way(1, rows, k, n) == "together"
    log(f"tiles {rows}x{k}x{n}")
    kit.ProductCase(1, k, n, "silu", BF, rows=rows, bias=True, residual=True, seed=k).check(experts, "long")


@pytest.mark.parametrize("k", INPUTS + [1019])
@pytest.mark.parametrize("planes,act,tokens,dtype", [(1, "gelu_tanh", 0, HF), (1, "none", 777, BF),
                                                     (2, "gelu", 0, BF), (2, "relu", 777, HF)])
def test_by_expert(k, planes, act, tokens, dtype):
    """Every body in one launch, short experts behind them."""
    n = 4801 if planes == 1 else 2401
    assert waykit.way_of_counts(planes, COUNTS, k, n, 7) == "together"
    log(f"tiles by expert {planes} {k} {tokens}")
    kit.ProductCase(planes, k, n, act, dtype, counts=COUNTS, tokens=tokens, bias=planes == 1, residual=planes == 1,
                    seed=k, spare=7).check(experts, f"{k}")


@pytest.mark.parametrize("planes,act,dtype", [(1, "silu", HF), (2, "gelu_tanh", HF)])
def test_by_expert_past_the_last_cache(planes, act, dtype):
    """The tiles behind a launch of their own for the short experts."""
    counts = COUNTS + [0] * 50
    k, n = 2000, 2080 if planes == 1 else 1040
    assert waykit.way_of_counts(planes, counts, k, n, 7) == "apart"
    log(f"tiles apart {planes}")
    kit.ProductCase(planes, k, n, act, dtype, counts=counts, tokens=0 if planes == 1 else 500, bias=planes == 1,
                    residual=planes == 1, seed=3, spare=7).check(experts, "apart")


@pytest.mark.parametrize("rows,n", DENSE)
def test_residual_is_the_output(rows, n):
    """y += the product: the bits of a residual of its own."""
    k = 130
    assert dense_way(1, rows, k, n) == "together"
    log(f"tiles in place {rows}")
    c = kit.ProductCase(1, k, n, "gelu", BF, rows=rows, residual=True, bias=True, seed=4)
    plan = c.plan(experts)
    packed, ws = experts.pack(plan, *c.w), plan.new_workspace()
    want, got = torch.empty_like(c.residual), c.residual.clone()
    c.run(experts, plan, packed, want, ws)
    c.residual = got
    c.run(experts, plan, packed, got, ws)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("rows,n", [(64, 50001), (180, 16601), (300, 10603), (500, 6403)])
@pytest.mark.parametrize("xs,ys,offset", [(203, 4, 1), (264, 13, 3)])
def test_strides_and_alignment(rows, n, xs, ys, offset):
    """Row strides and pointers that no wider load is aligned to; ys: columns
    between the rows of y."""
    log(f"tiles strides {rows} {xs} {ys} {offset}")
    for planes, act in ((1, "silu"), (2, "gelu")):
        m = n // planes | 1
        assert waykit.way(planes, rows, 199, m) == "together"
        kit.ProductCase(planes, 199, m, act, BF, rows=rows, bias=True, residual=planes == 1, seed=5, xs=xs, ys=m + ys,
                        offset=offset).check(experts, "strided", ys=m + ys, offset=offset)


@pytest.mark.parametrize("rows,n", [(100, 24995), (500, 6403)])
@pytest.mark.parametrize("planes,act", [(1, "none"), (2, "silu")])
def test_rows_that_are_not_finite(rows, n, planes, act):
    """An infinity or NaN makes its own row NaN and no other."""
    log(f"tiles not finite {rows} {planes}")
    m = n // planes | 1
    assert waykit.way(planes, rows, 130, m) == "together"
    c = kit.ProductCase(planes, 130, m, act, BF, rows=rows, seed=6)
    c.x[1, 37], c.x[2, 129], c.x[rows - 1, 0] = float("nan"), float("inf"), -float("inf")
    plan = c.plan(experts)
    y = torch.empty(rows, m, dtype=BF, device="cuda")
    c.run(experts, plan, experts.pack(plan, *c.w), y, plan.new_workspace())
    torch.cuda.synchronize()
    bad = torch.zeros(rows, dtype=torch.bool, device="cuda")
    bad[[1, 2, rows - 1]] = True
    assert torch.isnan(y[bad]).all()
    ref, bound = c.reference()
    bk.check(y[~bad], ref[~bad], bound[~bad], None, BF, "other rows")


@pytest.mark.parametrize("rows,n", [(64, 50001), (500, 6403)])
def test_rows_of_zeros_and_of_one_value(rows, n):
    """Scales of 0 beside ordinary ones, and rows whose largest value is alone."""
    log(f"tiles zeros {rows}")
    assert dense_way(1, rows, 300, n) == "together"
    c = kit.ProductCase(1, 300, n, "none", HF, rows=rows, seed=7)
    c.x[::3] = 0
    c.x[1::3, 1:] = 0
    y = c.check(experts, "zeros")
    assert (y[::3] == 0).all()


@pytest.mark.parametrize("rows,k,n", [(520, 40000, 12811), (250, 131071, 12603)])
def test_long_sums_of_the_largest_integers(rows, k, n):
    """Weights of -128 and 127 against rows of one size: the first columns' sums
    reach 2^31 of what 32 bits hold. The weights are int8 of those two columns'
    patterns, repeated, so that the reference is that of 40 columns."""
    assert waykit.way(1, rows, k, n) == "together"
    log(f"tiles long {rows}x{k}")
    c = kit.ProductCase(1, k, 40, "none", BF, rows=rows, seed=8, extreme=True)
    c.x.copy_(torch.where(c.w[0][0, :, :1].t() > 0, 1.5, -1.5).to(BF).expand(rows, k))
    c.w[0][0, :, 1] = -128
    c.x[rows // 2:] = 2.0
    ref, bound = c.reference()
    times = (n + 39) // 40
    c.n = n
    c.w[0] = c.w[0].repeat(1, 1, times)[:, :, :n].contiguous()
    c.scale[0] = c.scale[0].repeat(1, times)[:, :n].contiguous()
    plan = c.plan(experts)
    y = torch.empty(rows, n, dtype=BF, device="cuda")
    c.run(experts, plan, experts.pack(plan, *c.w), y, plan.new_workspace())
    torch.cuda.synchronize()
    bk.check(y[:, :40], ref, bound, None, BF, "long")
    for at in range(40, n, 40):
        assert torch.equal(y[:, at:at + 40], y[:, :min(40, n - at)]), at
    del c, y
    torch.cuda.empty_cache()


def test_graph_of_tiles():
    """A captured product by expert, replayed with other rows and offsets and
    eager calls of the same workspace in between: the eager bits."""
    log("tiles graph")
    k, n = 300, 4801
    assert waykit.way_of_counts(1, COUNTS, k, n, 7) == "together"
    c = kit.ProductCase(1, k, n, "silu", BF, counts=COUNTS, bias=True, residual=True, seed=9, spare=7)
    plan = c.plan(experts)
    packed, ws = experts.pack(plan, *c.w), plan.new_workspace()
    xs = [c.x, c.x.flip(0).contiguous(), (c.x.float() * 0.37).to(BF)]
    turned = torch.tensor([0] + COUNTS[::-1], device="cuda").cumsum(0).to(torch.int32)
    offsets = [c.offsets.clone(), turned, c.offsets.clone()]
    want = []
    for x, o in zip(xs, offsets):
        c.x, c.offsets = x, o
        y = torch.full((c.rows, n), 7.0, dtype=BF, device="cuda")
        c.run(experts, plan, packed, y, ws)
        want.append(y)
    c.x, c.offsets = xs[0], offsets[0]
    ref, bound = c.reference()
    torch.cuda.synchronize()
    bk.check(want[0][:c.kept], ref, bound, None, BF, "eager")
    x, o, got = xs[0].clone(), offsets[0].clone(), torch.full_like(want[0], 7.0)
    c.x, c.offsets = x, o
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(experts, plan, packed, got, ws)
    eager = torch.empty_like(got)
    for i in (0, 1, 2, 0, 2, 1):
        x.copy_(xs[i])
        o.copy_(offsets[i])
        got.fill_(7.0)
        graph.replay()
        c.x, c.offsets = xs[1], offsets[1]
        c.run(experts, plan, packed, eager, ws)
        torch.cuda.synchronize()
        assert torch.equal(got, want[i]), i
