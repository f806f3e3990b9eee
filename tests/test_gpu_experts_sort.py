"""Choices sorted by expert: integers, equal to the definition."""
import numpy as np
import pytest
import torch

from tests import expertskit as kit
from tests.routekit import log

pytestmark = pytest.mark.gpu

experts = pytest.importorskip("latent_projection_top_amd.experts")
from latent_projection_top_amd import route  # noqa: E402

I32 = torch.int32


def run(ids, count, first=0, capacity=None, spare=3, plan=None, ws=None, **kw):
    """offsets, place, token of one call; buffers larger than needed."""
    rows, topk = ids.shape
    plan = plan or experts.SortPlan(max(rows, 1), topk, count, first=first)
    ws = plan.new_workspace() if ws is None else ws
    offsets = torch.full((count + 1,), -7, dtype=I32, device="cuda")
    place = torch.full((rows + spare, topk), -7, dtype=I32, device="cuda")
    token = torch.full((rows * topk + spare if capacity is None else capacity,), -7, dtype=I32, device="cuda")
    experts.sort(plan, ids, offsets, place, token, ws, rows=rows, **kw)
    torch.cuda.synchronize()
    return offsets.cpu().numpy(), place.cpu().numpy(), token.cpu().numpy()


def check(ids, count, first=0, capacity=None, **kw):
    offsets, place, token = run(ids, count, first, capacity, **kw)
    want_o, want_p, want_t = kit.sort_reference(ids, count, first, capacity)
    assert np.array_equal(offsets, want_o)
    assert np.array_equal(place[:ids.shape[0]], want_p)
    assert (place[ids.shape[0]:] == -7).all()
    assert np.array_equal(token[:want_t.size], want_t)
    assert (token[want_t.size:] == -7).all()  # left as they were


SIZES = [(1, 16, 896), (1, 1, 1), (2, 1, 3), (3, 2, 5), (8, 16, 896), (20, 16, 896), (63, 1, 64), (64, 1, 64),
         (65, 1, 64), (127, 6, 40), (128, 8, 128), (333, 6, 64), (1000, 16, 896), (2047, 16, 896), (4096, 16, 896),
         (5000, 7, 1023), (4097, 1, 4096), (9999, 3, 4096), (16384, 16, 896), (40000, 2, 2)]


@pytest.mark.parametrize("rows,topk,count", SIZES)
def test_all_experts(rows, topk, count):
    log(f"sort {rows}x{topk} of {count}")
    check(kit.choices(rows, topk, count, seed=rows), count)


@pytest.mark.parametrize("rows,topk,total,first,count", [
    (1, 16, 896, 0, 112), (8, 16, 896, 784, 112), (20, 16, 896, 112, 56), (333, 6, 64, 32, 32), (2047, 16, 896, 336, 112),
    (6000, 4, 300, 299, 1), (5000, 16, 896, 1, 894)])
def test_a_share_of_the_experts(rows, topk, total, first, count):
    log(f"sort {rows}x{topk} share {first}+{count} of {total}")
    check(kit.choices(rows, topk, total, seed=rows), count, first)


@pytest.mark.parametrize("rows", [1, 5, 700, 5000, 30000])
def test_ids_that_no_expert_has(rows):
    """Negative ids, ids past the last, the type's limits; rows with nothing
    left, and calls with nothing left at all."""
    log(f"sort foreign ids {rows}")
    gen = torch.Generator().manual_seed(rows)
    ids = torch.randint(-3, 12, (rows, 4), generator=gen, dtype=I32)
    ids[::3] = torch.tensor([-2 ** 31, 2 ** 31 - 1, -1, 8], dtype=I32)
    check(ids.cuda(), 8)
    check(ids.cuda(), 3, first=2)
    check(torch.full((rows, 4), -1, dtype=I32, device="cuda"), 8)
    check(torch.full((rows, 4), 2 ** 31 - 1, dtype=I32, device="cuda"), 8, first=2 ** 31 - 1)


@pytest.mark.parametrize("rows", [1, 64, 1000, 20000])
def test_one_expert_has_everything_and_repeats(rows):
    """Every choice the same expert, more than once in a row: stable."""
    log(f"sort one expert {rows}")
    check(torch.full((rows, 8), 5, dtype=I32, device="cuda"), 8)
    ids = torch.randint(0, 2, (rows, 8), generator=torch.Generator().manual_seed(1), dtype=I32) * 4000
    check(ids.cuda(), 4096)


@pytest.mark.parametrize("capacity", [0, 1, 100, 5000])
def test_capacity(capacity):
    """token holds what fits; offsets and place are whole."""
    log(f"sort capacity {capacity}")
    check(kit.choices(700, 8, 64, seed=1), 64, capacity=capacity)


def test_largest_share_of_ids():
    log("sort 2^20 rows")
    check(torch.randint(0, 896, (1 << 20, 2), generator=torch.Generator().manual_seed(2), dtype=I32).cuda(), 896)


def test_no_rows_and_fewer_rows_than_the_plan():
    log("sort few rows")
    plan = experts.SortPlan(5000, 16, 896)
    ws = plan.new_workspace()
    for rows in (0, 1, 300, 5000, 7):
        ids = kit.choices(max(rows, 1), 16, 896, seed=rows)[:rows]
        if rows:
            check(ids, 896, plan=plan, ws=ws)
        else:
            offsets, _, _ = run(ids, 896, plan=plan, ws=ws)
            assert (offsets == 0).all()


def test_refusals():
    plan = experts.SortPlan(4, 2, 8)
    ws = plan.new_workspace()
    ids = torch.zeros(4, 2, dtype=I32, device="cuda")
    offsets, place = torch.empty(9, dtype=I32, device="cuda"), torch.empty(4, 2, dtype=I32, device="cuda")
    token = torch.empty(8, dtype=I32, device="cuda")

    def call(**kw):
        a = dict(ids=ids, offsets=offsets, place=place, token=token, workspace=ws)
        a.update(kw)
        experts.sort(plan, **a)

    call()
    for bad in (dict(ids=ids.long()), dict(place=place.long())):
        with pytest.raises(TypeError):
            call(**bad)
    for bad in (dict(ids=ids.cpu()), dict(ids=ids[:, :1]), dict(offsets=offsets[:8]), dict(place=place[:3]),
                dict(token=place), dict(workspace=ws[:16]), dict(ids=torch.zeros(2, 4, dtype=I32, device="cuda").t())):
        with pytest.raises(ValueError):
            call(**bad)
    many = torch.zeros(5, 2, dtype=I32, device="cuda")
    with pytest.raises(route.RouteError) as e:
        call(ids=many, place=many.clone())
    assert e.value.status == route.E_ROWS
    lib = experts.LIB.experts_sort
    args = [plan.handle, ids.data_ptr(), offsets.data_ptr(), place.data_ptr(), token.data_ptr(), ws.data_ptr(), 8, 4,
            None]
    for i, value, status in ((1, None, route.E_ARG), (2, None, route.E_ARG), (3, None, route.E_ARG),
                             (4, None, route.E_ARG), (5, None, route.E_ARG), (6, -1, route.E_ROWS),
                             (6, experts.MAX_CHOICES + 1, route.E_ROWS), (7, -1, route.E_ROWS), (7, 5, route.E_ROWS),
                             (1, ids.data_ptr() + 2, route.E_ALIGN), (5, ws.data_ptr() + 4, route.E_ALIGN)):
        bad = list(args)
        bad[i] = value
        assert lib(*bad) == status, (i, value)
    torch.cuda.synchronize()
