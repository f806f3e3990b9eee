"""The activations through every ending of a product: the gated and the linear
one, BF16 and F16, streamed, tiled and joined from split sums, with whole and
partial groups of columns.

As for the activations alone, an identity matrix brings each argument to its
column unchanged: one term of a sum is the argument, the rest are zeros, in
whatever order they are added and over however many splits. In the gated
product the second matrix multiplies an input column of ones, so u = 1 and its
outputs are the value (h, d_up) and the slope (d_gate) themselves.

Bounds: the output's rounding (the type's unit of the value, and half the
spacing of its subnormals) and for the FP32 arithmetic 4e-5 of the terms: in
the negative tail the exponential's argument reaches 127 in base 2, where four
roundings of 2^-24 move the result by 127 x 4 x 2^-24 x ln 2 = 2.1e-5."""
import pytest
import torch

from tests import blockkit as kit
from tests.routekit import log

pytestmark = pytest.mark.gpu

block = pytest.importorskip("latent_projection_top_amd.block")

BF, HF = torch.bfloat16, torch.float16
ACTS = ("relu", "silu", "gelu", "gelu_tanh")
# rows, K, columns: streamed, tiled, and with K long enough to be split
SHAPES = [(4, 72, 61), (16, 72, 64), (8, 4096, 61), (32, 4096, 64), (64, 72, 64), (64, 4096, 61), (64, 4096, 64),
          (130, 2048, 40)]


def run(op, act, dtype, z, k, diagonal=None, bias=None):
    """(value, slope, d_up or None) of the arguments z [rows][n]."""
    rows, n = z.shape
    x = torch.zeros(rows, k, dtype=dtype, device="cuda")
    x[:, :n] = z.to(dtype)
    eye = torch.zeros(k, n, dtype=dtype, device="cuda")
    eye[:n] = torch.diag(torch.ones(n) if diagonal is None else diagonal).to(dtype)
    out = [torch.full((rows, n), 7.0, dtype=dtype, device="cuda") for _ in range(3)]
    if op == "gated":
        x[:, n] = 1
        up = torch.zeros(k, n, dtype=dtype, device="cuda")
        up[n] = 1
        plan = block.GatedPlan(rows, k, n, act, dtype, training=True)
        block.gated(plan, x, eye, up, out[0], plan.new_workspace(), out[1], out[2])
    else:
        plan = block.LinearPlan(rows, k, n, act, dtype, training=True)
        block.linear(plan, x, eye, out[0], plan.new_workspace(), None if bias is None else bias.to(dtype).cuda(),
                     None, out[1])
    torch.cuda.synchronize()
    out = [t.double().cpu() for t in out]
    return out if op == "gated" else out[:2]


def exact(act, z):
    """The gate, the rest of the slope beside it; value = z gate, slope =
    gate + rest. Written without the cancellation of 1 + erf and 1 + tanh."""
    if act == "gelu":
        return 0.5 * torch.special.erfc(-z / 2.0 ** 0.5), z * torch.exp(-0.5 * z * z) * 0.3989422804014327
    if act == "gelu_tanh":
        c = 2.0 * (2.0 / torch.pi) ** 0.5
        t = c * (z + 0.044715 * z ** 3)
        return torch.sigmoid(t), z * torch.sigmoid(t) * torch.sigmoid(-t) * c * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        return torch.sigmoid(z), z * torch.sigmoid(z) * torch.sigmoid(-z)
    return (z > 0).double(), torch.zeros_like(z)


@pytest.mark.parametrize("dtype", (BF, HF))
@pytest.mark.parametrize("op", ("gated", "linear"))
@pytest.mark.parametrize("act", ACTS)
def test_value_and_slope(act, op, dtype):
    u, tiny = kit.UNIT[dtype], max(kit.TINY[dtype], 1e-36)
    for rows, k, n in SHAPES:
        log(f"ending {op} {act} {dtype} {rows}x{k}x{n}")
        z = torch.linspace(-12.5, 12.5, rows * n, dtype=torch.float64).reshape(rows, n).to(dtype)
        got = run(op, act, dtype, z, k)
        gate, rest = exact(act, z.double())
        value, slope = z.double() * gate, gate + rest
        assert torch.allclose(slope, kit.slope(act, z.double()), rtol=0, atol=1e-12)
        bound = (u + 4e-5) * value.abs() + tiny
        for v in got[::2]:
            assert bool(((v - value).abs() <= bound).all()), ((v - value).abs() / bound).max()
        bound = u * slope.abs() + 4e-5 * (gate + rest.abs()) + tiny
        assert bool(((got[1] - slope).abs() <= bound).all()), ((got[1] - slope).abs() / bound).max()


@pytest.mark.parametrize("dtype", (BF, HF))
@pytest.mark.parametrize("op", ("gated", "linear"))
@pytest.mark.parametrize("act", ACTS)
def test_infinite_nan_and_huge_arguments(act, op, dtype):
    """Through a matrix whose diagonal holds infinity, NaN and huge values at
    an input of one; every other column keeps its ordinary value."""
    big = 1e30 if dtype == BF else 6e4
    special = [float("inf"), float("nan"), big, -big, 0.0, -0.0]
    at = 0.0 if act == "relu" else 0.5  # slope at zero
    for rows, k, n in SHAPES:
        log(f"special {op} {act} {dtype} {rows}x{k}x{n}")
        z = torch.ones(rows, n)
        clean = run(op, act, dtype, z, k)
        d = torch.ones(n)
        d[:6] = torch.tensor(special)
        got = run(op, act, dtype, z, k, diagonal=d)
        if op == "linear":  # the same arguments as a bias
            z[:, :6] = 0
            b = torch.zeros(n)
            b[:6] = torch.tensor(special)
            with_bias = run(op, act, dtype, z, k, bias=b)
            assert all(torch.equal(torch.nan_to_num(p, nan=5.0), torch.nan_to_num(q, nan=5.0))
                       for p, q in zip(with_bias, got))
        huge = torch.tensor(big).to(dtype).double()
        for v in got[::2]:
            assert bool((v[:, 0] == float("inf")).all()) and bool(v[:, 1].isnan().all())
            assert bool((v[:, 2] == huge).all()) and bool((v[:, 3:6] == 0).all())
        s = got[1]
        assert bool((s[:, 0] == 1).all()) and bool(s[:, 1].isnan().all()) and bool((s[:, 2] == 1).all())
        assert bool((s[:, 3] == 0).all()) and bool((s[:, 4:6] == at).all())
        assert all(torch.equal(p[:, 6:], q[:, 6:]) for p, q in zip(got, clean))
