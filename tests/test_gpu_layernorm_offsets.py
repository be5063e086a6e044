"""Layer norm's forward on rows whose mean is far above their deviation, constant rows among them.

Bounds as in test_gpu_layernorm.py: U = 2^-24 for each fp32 rounding, DEPTH for
the depth of a row's sum.
"""
import pytest
import torch

from normalisation_row_bf16_b200 import build as nbuild
from normalisation_row_bf16_b200 import ops
from test_gpu_layernorm import DEPTH, TYPES, U, half_step, make

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _built():
    nbuild.build()


LENGTHS = [7, 33, 200, 256, 257, 800, 1544, 4095, 4096, 5003, 8192, 20481, 32767, 32768]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D", LENGTHS)
def test_constant_rows(D, dtype):
    """A constant row has its value for a mean and no deviation: y is beta, bit for bit."""
    c = torch.tensor([1e4, -12345.678, 65000.0, 1e-3, 0.1, 0.0, 700.7, -3.14159, 1.0], device="cuda").to(dtype)
    x = c[:, None].expand(-1, D).contiguous()
    beta = torch.linspace(-1, 1, D, device="cuda").to(dtype)
    y, mean, rstd = ops.layernorm_fwd(x, None, beta)
    assert torch.equal(mean, c.float())
    assert torch.equal(y, beta[None].expand_as(y))
    assert ((rstd.double() - 1e-5 ** -0.5).abs() <= 4 * U * 1e-5 ** -0.5 + 317 * 1e-7).all()


@pytest.mark.parametrize("offset", [1e4, 1e6])
@pytest.mark.parametrize("T,D", [(3, 33), (40, 512), (40, 800), (40, 4096), (1300, 4096), (40, 4095), (3, 20483), (3, 32768)])
def test_forward_far_mean(T, D, offset):
    """The mean is right to its own rounding, and y to what that rounding leaves."""
    x, gamma, beta, _ = make(T, D, torch.float32, seed=D, offset=offset)
    y, mean, rstd = ops.layernorm_fwd(x, gamma, beta)
    v = x.double()
    rm = v.mean(1, keepdim=True)
    d = v - rm
    rr = (d.square().mean(1, keepdim=True) + 1e-5).rsqrt()
    # the first mean is off by up to dm1; the second adds the mean of what is left, summed in fp32, and rounds once
    dm1 = U * (DEPTH + 2) * v.abs().mean(1, keepdim=True)
    dm = 1.01 * U * rm.abs() + U * (DEPTH + 4) * (d.abs().mean(1, keepdim=True) + dm1)
    dvar = U * (DEPTH + 6) * d.square().mean(1, keepdim=True) + dm * dm + 2 * dm * d.abs().mean(1, keepdim=True)
    dr = 0.5 * dvar * rr ** 3 + 4 * U * rr
    assert ((mean.double()[:, None] - rm).abs() <= dm).all()
    assert ((rstd.double()[:, None] - rr).abs() <= dr).all()
    xh = d * rr
    ry = xh * gamma.double() + beta.double()
    err = gamma.double().abs() * (rr * (dm + U * d.abs()) + d.abs() * dr + 3 * U * xh.abs()) + 2 * U * ry.abs()
    assert ((y.double() - ry).abs() <= half_step(torch.float32, ry.abs() + err) + err).all()
