"""The gated feed-forward backward where a gate is so far out that its powers overflow fp32."""
import pytest
import torch

from normalisation_row_bf16_b200 import build as nbuild
from normalisation_row_bf16_b200 import ops

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _built():
    nbuild.build()


@pytest.mark.parametrize("name", ["silu", "gelu", "gelu_tanh"])
def test_gates_whose_powers_overflow(name):
    """Far above zero act(g) is g and act'(g) is 1, far below both are 0; dg = dh * up * act'(g), du = dh * act(g).

    At a distance a the activations are within a e^-a of that and their derivatives within (1 + a) e^-a: with s the
    sigmoid, s(-a) < e^-a and silu'(-a) = s(-a) (1 - a s(a)), silu'(a) = 1 - silu'(-a); the normal distribution and its
    tanh form fall off faster.  bf16 adds half a step.
    """
    F, D = 16, 8
    far = torch.tensor([30.0, 1e4, 1e10, 1e13, 5e18, 1e19, 6e19, 1e20, 1e30, 3e38], device="cuda")
    for gates, grad in ((far, 1.0), (-far, 0.0)):
        T = gates.numel()
        for t in range(T):
            gate = gates[t].bfloat16().expand(1, F).contiguous()
            one = torch.ones(1, F, device="cuda", dtype=torch.bfloat16)
            x = torch.ones(1, D, device="cuda", dtype=torch.bfloat16)
            w = torch.eye(F, D, device="cuda").bfloat16()
            _, dwg, dwu = ops.gated_ffn_bwd(one, x, w, torch.zeros_like(w), gate, one, act=name)
            a = gate[0, 0].double().abs()
            off = 1.01 * (1 + a) * torch.exp(-a)
            for got, want in ((dwg, grad), (dwu, a if grad else 0.0)):
                assert ((got.double() - want).abs() <= off + 2.0 ** -8 * off).all(), (name, float(gates[t]), got[0, 0].item())
