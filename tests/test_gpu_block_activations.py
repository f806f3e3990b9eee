"""The activations themselves, value and slope, against their FP64 definitions
through both matrix kernels: an identity weight brings each argument to the
activation unchanged (its products with zero add nothing), so the bounds are
the activation's own.

Bounds: the output's rounding (2^-8 of the value in BF16) and, for the FP32
arithmetic, 4e-5 of the terms that make it up. That covers the exponential in
the negative tail: its argument reaches 127 in base 2, where four roundings of
2^-24 move the result by 127 x 4 x 2^-24 x ln 2 = 2.1e-5. What FP32 holds only
as a subnormal number may be zero: 1e-36 absolute."""
import pytest
import torch

from tests import blockkit as kit

pytestmark = pytest.mark.gpu

block = pytest.importorskip("latent_projection_top_amd.block")

BF = torch.bfloat16
SIZE = 64
ACTS = ("relu", "silu", "gelu", "gelu_tanh")


def run(act, rows, x, bias):
    plan = block.LinearPlan(rows, SIZE, SIZE, act, BF, training=True)
    w = torch.eye(SIZE, dtype=BF, device="cuda")
    y, slope = (torch.full((rows, SIZE), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    block.linear(plan, x, w, y, plan.new_workspace(), bias, None, slope)
    torch.cuda.synchronize()
    return y.double().cpu(), slope.double().cpu()


@pytest.mark.parametrize("rows", (16, 64))  # streamed, tiled
@pytest.mark.parametrize("act", ACTS)
def test_value_and_slope_keep_relative_precision(act, rows):
    z = torch.linspace(-12.5, 12.5, rows * SIZE, dtype=torch.float64).reshape(rows, SIZE).to(BF)
    y, slope = run(act, rows, z.cuda(), None)
    z = z.double()
    # 1 + erf and 1 + tanh cancel in the negative tail, also in 64 bits
    if act == "gelu":
        gate = 0.5 * torch.special.erfc(-z / 2.0 ** 0.5)
        rest = z * torch.exp(-0.5 * z * z) * 0.3989422804014327
    elif act == "gelu_tanh":
        c = 2.0 * (2.0 / torch.pi) ** 0.5
        gate = torch.sigmoid(c * (z + 0.044715 * z ** 3))
        rest = z * gate * torch.sigmoid(-c * (z + 0.044715 * z ** 3)) * c * (1 + 3 * 0.044715 * z * z)
    elif act == "silu":
        gate = torch.sigmoid(z)
        rest = z * gate * torch.sigmoid(-z)
    else:
        gate, rest = (z > 0).double(), torch.zeros_like(z)
    value, d = z * gate, gate + rest
    assert torch.allclose(d, kit.slope(act, z), rtol=0, atol=1e-12)
    bound = (2.0 ** -8 + 4e-5) * value.abs() + 1e-36
    assert bool(((y - value).abs() <= bound).all()), ((y - value).abs() / bound).max()
    bound = 2.0 ** -8 * d.abs() + 4e-5 * (gate + rest.abs()) + 1e-36
    assert bool(((slope - d).abs() <= bound).all()), ((slope - d).abs() / bound).max()


@pytest.mark.parametrize("rows", (16, 64))
@pytest.mark.parametrize("act", ACTS)
def test_infinite_and_huge_arguments(act, rows):
    special = torch.tensor([float("inf"), float("nan"), 1e30, -1e30, 0.0, -0.0])
    bias = torch.zeros(SIZE)
    bias[:6] = special
    y, slope = run(act, rows, torch.zeros(rows, SIZE, dtype=BF, device="cuda"), bias.to(BF).cuda())
    at = 0.0 if act == "relu" else 0.5  # slope at zero
    assert bool((y[:, 0] == float("inf")).all()) and bool((slope[:, 0] == 1).all())
    assert bool(y[:, 1].isnan().all()) and bool(slope[:, 1].isnan().all())
    big = bias[2].to(BF).double()
    assert bool((y[:, 2] == big).all()) and bool((slope[:, 2] == 1).all())
    assert bool((y[:, 3] == 0).all()) and bool((slope[:, 3] == 0).all())
    assert bool((y[:, 4:] == 0).all()) and bool((slope[:, 4:] == at).all())
