"""Products by expert whose offsets a program got wrong, on every way through
the kernels."""
import pytest
import torch

from tests import blockkit as bk
from tests import expertskit as kit
from tests import waykit
from tests.routekit import log

pytestmark = pytest.mark.gpu

experts = pytest.importorskip("latent_projection_top_amd.experts")

BF = torch.bfloat16

# counts, K, N, rows that no expert has; the way that they take
CASES = {"fused": ([9, 8, 0], 330, 90, 9), "brief": ([30, 20, 0, 0, 0, 0, 0, 0], 2100, 264, 20),
         "few": ([40, 60, 0], 330, 90, 40), "together": ([600, 1400, 0, 900, 0], 863, 1368, 1400),
         "apart": ([700, 1200, 0, 1] + [0] * 62, 2048, 2040, 500)}


@pytest.mark.parametrize("planes,act", [(1, "silu"), (2, "gelu")])
@pytest.mark.parametrize("tokens", [0, 37])
@pytest.mark.parametrize("way", CASES)
def test_rows_behind_the_last_offset_are_nobodys(way, tokens, planes, act):
    """An expert's end past offsets[experts]: its rows there are left as they
    were, and what the workspace holds of earlier calls decides nothing."""
    counts, k, n, spare = CASES[way]
    assert waykit.way_of_counts(planes, counts, k, n, spare) == way
    log(f"ends {way} {tokens} {planes}")
    c = kit.ProductCase(planes, k, n, act, BF, counts=counts, tokens=tokens, bias=planes == 1,
                        residual=planes == 1, seed=1, spare=spare)
    # the second expert's range ends among the spare rows; the next begins there
    c.offsets[2] = c.kept + spare // 2
    if sum(counts[2:]) != 0:  # the others' rows are the second one's
        c.counts = [counts[0], c.kept - counts[0]] + [0] * (len(counts) - 2)
        c.offsets[2:-1] = c.kept + spare // 2
    plan = c.plan(experts)
    packed, ws = experts.pack(plan, *c.w), plan.new_workspace()
    outs = []
    for fill in (0, 85, 255):
        ws[experts.WORKSPACE_ZEROED:] = fill
        y = torch.full((c.rows, n), 7.0, dtype=BF, device="cuda")
        c.run(experts, plan, packed, y, ws)
        torch.cuda.synchronize()
        outs.append(y)
    ref, bound = c.reference()
    for y in outs:
        bk.check(y[:c.kept], ref, bound, None, BF, "kept rows")
        assert (y[c.kept:] == 7).all()
