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


def nonsense(experts_, rows):
    """Offsets of so many experts that no sort gives, by name."""
    def last(values):
        return (values + [rows] * (experts_ + 1))[:experts_] + [values[-1]]

    return {"decreasing": last([0, rows // 3, rows // 5, rows // 2, rows - 3]),
            "outside": last([-5, rows // 8, rows // 8, 1 << 30, rows]),
            "limits": last([0, 2 ** 31 - 1, -2 ** 31, rows // 7, rows // 2]),
            "nothing": [rows // 5] * (experts_ + 1), "negative": last([0, rows, -1, -2 ** 31]),
            "beyond": [0] + [2 ** 31 - 1] * experts_,
            "repeated": [0, rows] * (experts_ // 2) + [0] * (experts_ % 2) + [rows],
            "turns": [rows - 1 if e % 2 else e for e in range(experts_)] + [rows]}


@pytest.mark.parametrize("what", list(nonsense(4, 40)))
@pytest.mark.parametrize("way", CASES)
def test_offsets_that_make_no_sense(way, what):
    """No access leaves the buffers on any way: guards around y and the
    workspace keep their values; rows that no range has are left alone, and
    where ranges rise from 0 they hold their experts' results. Ranges that
    overlap make more items than the lists have room for."""
    counts, k, n, spare = CASES[way]
    rows = sum(counts) + spare
    for planes in (1, 2):
        assert waykit.way_of_counts(planes, counts, k, n, spare) == way
        log(f"offsets {way} {what} {planes}")
        c = kit.ProductCase(planes, k, n, "silu", BF, counts=[rows] + [0] * (len(counts) - 1), seed=2)
        offsets = nonsense(len(counts), rows)[what]
        assert len(offsets) == len(counts) + 1
        c.offsets = torch.tensor(offsets, dtype=torch.int32, device="cuda")
        plan = c.plan(experts)
        size = plan.workspace_bytes
        buf = torch.full((size + 512,), 91, dtype=torch.uint8, device="cuda")
        ws = buf[256:256 + size]
        ws[:experts.WORKSPACE_ZEROED] = 0
        full = torch.full((rows + 64, n), 7.0, dtype=BF, device="cuda")
        y = full[32:32 + rows]
        packed = experts.pack(plan, *c.w)
        for _ in range(2):
            c.run(experts, plan, packed, y, ws)
        torch.cuda.synchronize()
        assert (full[:32] == 7).all() and (full[32 + rows:] == 7).all()
        assert (buf[:256] == 91).all() and (buf[256 + size:] == 91).all()
        assert not ws[:experts.WORKSPACE_ZEROED].any()
        end = min(max(offsets[-1], 0), rows)
        cut = [min(max(o, 0), end) for o in offsets]
        covered = torch.zeros(rows, dtype=torch.bool)
        for a, b in zip(cut, cut[1:]):
            covered[a:max(a, b)] = True
        assert (y[~covered.cuda()] == 7).all()
        if end > 0 and cut == sorted(cut) and cut[0] == 0:
            c.counts = [b - a for a, b in zip(cut, cut[1:])]
            ref, bound = c.reference()
            bk.check(y[:end], ref, bound, None, BF, what)


@pytest.mark.parametrize("way", CASES)
def test_tokens_that_no_row_has(way):
    """Tokens out of range are the nearest row of x, on every way."""
    counts, k, n, spare = CASES[way]
    log(f"tokens {way}")
    for planes in (1, 2):
        c = kit.ProductCase(planes, k, n, "silu", BF, counts=counts, tokens=10, seed=3, spare=spare)
        want = c.token.clone()
        for at, value, near in ((3, -1, 0), (c.kept - 1, 2 ** 31 - 1, 9), (c.kept // 2, -2 ** 31, 0),
                                (c.rows - 1, 10, 9)):
            c.token[at], want[at] = value, near
        plan = c.plan(experts)
        packed, ws = experts.pack(plan, *c.w), plan.new_workspace()
        outs = []
        for token in (c.token, want):
            c.token = token
            outs.append(torch.full((c.rows, n), 7.0, dtype=BF, device="cuda"))
            c.run(experts, plan, packed, outs[-1], ws)
        torch.cuda.synchronize()
        assert torch.equal(*outs)
        ref, bound = c.reference()
        bk.check(outs[1][:c.kept], ref, bound, None, BF, "tokens")
