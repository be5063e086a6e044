"""Calls on a stream that is not the current one, whose inputs the caller gives up right away."""
import pytest
import torch

from normalisation_row_bf16_b200 import build as nbuild
from normalisation_row_bf16_b200 import ops

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(autouse=True, scope="module")
def _built():
    nbuild.build()


def rand(*shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF)


def _ln_args():
    return rand(512, 1024, seed=3), rand(512, 1024, seed=4)


def _mx_args():
    return [t for n in (256, 512, 520) for t in ops.mxfp8_cast(rand(n, 256, seed=n, scale=0.1), scale_layout=ops.SCALES_MMA)]


def _bwd_inputs():
    x, dy = _ln_args()
    return (x, dy, *ops.layernorm_fwd(x)[1:])


def _ffn_inputs():
    return [rand(256, 512, seed=1), rand(1024, 512, seed=2, scale=0.05), rand(1024, 512, seed=3, scale=0.05)]


def _ffn_bwd_inputs():
    x, wg, wu = _ffn_inputs()
    _, gate, up = ops.gated_ffn_fwd(x, wg, wu, save=True)
    return [rand(256, 1024, seed=9), x, wg, wu, gate, up]


NEW = {
    "layernorm_fwd": (_ln_args, lambda a, **k: ops.layernorm_fwd(a[0], **k)),
    "layernorm_bwd": (_bwd_inputs, lambda a, **k: ops.layernorm_bwd(a[0], a[1], None, a[2], a[3], **k)),
    "gated_ffn_fwd": (_ffn_inputs, lambda a, **k: ops.gated_ffn_fwd(*a, **k)),
    "gated_ffn_bwd": (_ffn_bwd_inputs, lambda a, **k: ops.gated_ffn_bwd(*a, **k)),
    "mxfp8_gated_ffn": (_mx_args, lambda a, **k: ops.mxfp8_gated_ffn(*a, 256, 512, 256, **k)),
}


def flat(r):
    return [t for t in (r if isinstance(r, tuple) else (r,)) if t is not None]


def dropped_inputs(make, call):
    want = [t.clone() for t in flat(call(make()))]
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    args = make()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)           # about 0.1 s: the call below has yet to run
    got = call(args, stream=side)
    sizes = [t.untyped_storage().nbytes() for t in args]
    del args
    # memory of the inputs' sizes, and of what the call may have taken for itself, on the current stream
    sizes += [512, 1 << 14, 1 << 16, 1 << 18, 600_000]
    taken = [torch.full((n,), 0x7B, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(3)]
    torch.cuda.current_stream().synchronize()
    side.synchronize()
    torch.cuda.synchronize()
    return want, flat(got), taken


@pytest.mark.parametrize("name", list(NEW))
def test_inputs_dropped_behind_a_call_on_another_stream(name):
    want, got, taken = dropped_inputs(*NEW[name])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all((t == 0x7B).all() for t in taken)


@pytest.mark.parametrize("name", list(NEW))
def test_forked_stream_in_a_graph(name):
    """The call on a stream that a captured one forked and joins again, its inputs given up after the capture."""
    make, call = NEW[name]
    args = make()
    want = [t.clone() for t in flat(call(args))]
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        side.wait_stream(torch.cuda.current_stream())
        got = flat(call(args, stream=side))
        torch.cuda.current_stream().wait_stream(side)
    for t in got:
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    del args, got, g
    torch.cuda.empty_cache()


def _mxnorm_bwd_inputs():
    x, dy = _ln_args()
    gamma = torch.ones(1024, device="cuda", dtype=BF)
    return [x, dy, gamma, ops.mxnorm_fwd(x, gamma)[2]]


OLD = {
    "mxnorm_fwd": (_ln_args, lambda a, **k: ops.mxnorm_fwd(a[0], **k)),
    "mxnorm_fwd_ex": (_ln_args, lambda a, **k: ops.mxnorm_fwd_ex(a[0], elem="nvfp4", **k)),
    "mxfp8_cast": (_ln_args, lambda a, **k: ops.mxfp8_cast(a[0], **k)),
    "mx_cast": (_ln_args, lambda a, **k: ops.mx_cast(a[0], elem="e2m1", **k)),
    "fold_weight": (_ln_args, lambda a, **k: ops.fold_weight(a[0], a[1][0].contiguous(), **k)),
    "rmsnorm_bf16": (_ln_args, lambda a, **k: ops.rmsnorm_bf16(a[0], **k)),
    "rmsnorm_then_mxcast": (_ln_args, lambda a, **k: ops.rmsnorm_then_mxcast(a[0], **k)),
    "mxnorm_bwd": (_mxnorm_bwd_inputs, lambda a, **k: ops.mxnorm_bwd(*a, **k)),
    "mxnorm_bwd_noalloc": (_mxnorm_bwd_inputs, lambda a, **k: ops.mxnorm_bwd_noalloc(*a, **k)),
    "mxfp8_gemm": (_mx_args, lambda a, **k: ops.mxfp8_gemm(a[0], a[1], a[2], a[3], 256, 512, 256, **k)),
}


@pytest.mark.parametrize("name", list(OLD))
def test_inputs_dropped_behind_an_older_call_on_another_stream(name):
    want, got, taken = dropped_inputs(*OLD[name])
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert all((t == 0x7B).all() for t in taken)
