"""Precision of the norm's summed gradients in FP32, beyond the worst case."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

block = pytest.importorskip("latent_projection_top_amd.block")


def test_dbias_rounds_as_a_shallow_tree():
    """517 rows of FP32. An addition rounds its result s to within 2^-24 of its
    binade's start: in the RMS 2^-24 / sqrt(3) of |s| times sqrt(E[1/m^2]) =
    0.735 for a mantissa m spread evenly by its logarithm. Adding n independent
    terms in order makes partial sums of 1..n terms, together n / 2 of the
    result's square, and a level of a tree 1. Blocks of two rows (1), slices of
    14 blocks (7) and 32 slices pairwise (5) are 13, sqrt(13) x 2.53e-8 =
    0.91e-7 of dbias in the RMS; a tenth more is allowed for the sample."""
    rows, width = 517, 4096
    gen = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(rows, width, generator=gen, device="cuda")
    dy = torch.randn(rows, width, generator=gen, device="cuda")
    plan = block.NormPlan(rows, 1019, dtype=torch.float32)
    got, want = [], []
    for c in range(0, width - 1019, 1019):  # the columns of four calls
        xs, ds = x[:, c:c + 1019].contiguous(), dy[:, c:c + 1019].contiguous()
        y, dx = torch.empty_like(xs), torch.empty_like(xs)
        m, r = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        dw, db = torch.empty(1019, device="cuda"), torch.empty(1019, device="cuda")
        block.layer_norm(plan, xs, None, None, y, m, r)
        block.layer_norm_backward(plan, ds, xs, None, m, r, dx, dw, db, plan.new_workspace())
        torch.cuda.synchronize()
        got.append(db.double())
        want.append(ds.double().sum(0))
    got, want = torch.cat(got), torch.cat(want)
    rms = float((got - want).norm() / want.norm())
    assert rms <= 1.1 * math.sqrt(13) * 2.0 ** -24 / math.sqrt(3) * 0.735, rms
