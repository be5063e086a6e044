"""Layer norm's backward on rows whose mean is far above their deviation.

Bounds as in test_gpu_layernorm.py: U = 2^-24 for each fp32 rounding, DEPTH for
the depth of a row's sum.
"""
import pytest
import torch

from normalisation_row_bf16_b200 import build as nbuild
from normalisation_row_bf16_b200 import ops
from test_gpu_layernorm import DEPTH, U, half_step, make

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _built():
    nbuild.build()


def check_bwd(x, dy, gamma, mean, rstd, dx, dgamma, dbeta):
    """Against the formula on the given statistics; xh = (x - mean) * rstd takes two roundings, whatever the mean is."""
    t = x.dtype
    x, dy, m, r = x.double(), dy.double(), mean.double()[:, None], rstd.double()[:, None]
    T = x.shape[0]
    g = dy if gamma is None else dy * gamma.double()
    xh = (x - m) * r
    e = 2.01 * U * xh.abs()
    c1, c2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    rdx = r * (g - c1 - xh * c2)
    d1 = U * (DEPTH + 4) * g.abs().mean(1, keepdim=True)
    d2 = U * (DEPTH + 6) * (g * xh).abs().mean(1, keepdim=True) + (g.abs() * e).mean(1, keepdim=True)
    err = r * (d1 + xh.abs() * d2 + e * (c2.abs() + d2) + U * (4 * g.abs() + 3 * (xh * c2).abs() + 3 * c1.abs()))
    assert ((dx.double() - rdx).abs() <= half_step(t, rdx.abs() + err) + err).all()
    depth = -(-T // 100) + 16 + 32        # rows a group, groups a CTA, CTAs (a device of 148 SMs)
    rg, s = (dy * xh).sum(0), (dy * xh).abs().sum(0)
    eg = U * (depth + 2) * s + (dy.abs() * e).sum(0)
    assert ((dgamma.double() - rg).abs() <= half_step(t, rg.abs() + eg) + eg).all()
    rb, eb = dy.sum(0), U * depth * dy.abs().sum(0)
    assert ((dbeta.double() - rb).abs() <= half_step(t, rb.abs() + eb) + eb).all()


@pytest.mark.parametrize("offset", [1e3, 1e5])
@pytest.mark.parametrize("T,D", [(20, 512), (20, 4096), (20, 4095), (400, 1031), (400, 1032), (9, 16384), (9, 200)])
def test_backward_far_mean(T, D, offset):
    x, gamma, _, g = make(T, D, torch.float32, seed=D, offset=offset)
    dy = torch.randn(T, D, generator=g, device="cuda").abs()
    _, mean, rstd = ops.layernorm_fwd(x, gamma)
    check_bwd(x, dy, gamma, mean, rstd, *ops.layernorm_bwd(x, dy, gamma, mean, rstd))


@pytest.mark.parametrize("dtype,offset", [(torch.bfloat16, 300.0), (torch.float16, 3000.0)])
@pytest.mark.parametrize("D", [4096, 1000, 1001, 14336])
def test_backward_far_mean_16_bit(D, dtype, offset):
    x, gamma, _, g = make(50, D, dtype, seed=D, offset=offset)
    dy = torch.randn(50, D, generator=g, device="cuda").abs().to(dtype)
    _, mean, rstd = ops.layernorm_fwd(x, gamma)
    check_bwd(x, dy, gamma, mean, rstd, *ops.layernorm_bwd(x, dy, gamma, mean, rstd))
