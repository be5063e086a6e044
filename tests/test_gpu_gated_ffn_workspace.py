"""The workspace of the gated feed-forward backward: any size from dg and du on serves."""
import pytest
import torch

from normalisation_row_bf16_b200 import build as nbuild
from normalisation_row_bf16_b200 import ops
from test_gpu_gated_ffn import check_bwd, inputs, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _built():
    nbuild.build()


@pytest.mark.parametrize("t_max,T", [(160, 128), (256, 128), (256, 8), (256, 100), (160, 160), (640, 333)])
@pytest.mark.parametrize("D,F", [(2048, 768), (1032, 2744)])
def test_a_workspace_of_a_larger_batch_serves_a_smaller_one(D, F, t_max, T):
    x, wg, wu = inputs(T, D, F, seed=T)
    dh = rand((T, F), 5, 0.1)
    _, gate, up = ops.gated_ffn_fwd(x, wg, wu, save=True)
    n = ops.gated_ffn_bwd_workspace_bytes(t_max, D, F)
    ws = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    check_bwd(dh, x, wg, wu, gate, up, "silu", *ops.gated_ffn_bwd(dh, x, wg, wu, gate, up, workspace=ws[:n]))
    assert (ws[n:] == 0xA5).all()
    assert ops.device_status() == ops.MXN_OK


@pytest.mark.parametrize("T,D,F", [(128, 2048, 768), (333, 1032, 2744), (4096, 512, 1408), (37, 136, 72)])
def test_any_workspace_from_dg_and_du_on(T, D, F):
    """The contractions are split into what the workspace has room for; nothing behind it is written, and one of the
    size asked for gives the same as the call's own."""
    x, wg, wu = inputs(T, D, F, seed=T)
    dh = rand((T, F), 5, 0.1)
    _, gate, up = ops.gated_ffn_fwd(x, wg, wu, save=True)
    full = max(ops.gated_ffn_bwd_workspace_bytes(T, D, F), 4 * T * F)
    own = ops.gated_ffn_bwd(dh, x, wg, wu, gate, up)
    for n in (4 * T * F, 4 * T * F + 4 * T * D, (4 * T * F + full) // 2, full - 1, full, full + 1000):
        n = max(n, 4 * T * F)
        ws = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        got = ops.gated_ffn_bwd(dh, x, wg, wu, gate, up, workspace=ws[:n])
        check_bwd(dh, x, wg, wu, gate, up, "silu", *got)
        assert (ws[n:] == 0xA5).all()
        if n >= full:
            assert all(torch.equal(a, b) for a, b in zip(got, own))
    with pytest.raises(ValueError):
        ops.gated_ffn_bwd(dh, x, wg, wu, gate, up, workspace=torch.empty(4 * T * F - 2, dtype=torch.uint8, device="cuda"))
    assert ops.device_status() == ops.MXN_OK
