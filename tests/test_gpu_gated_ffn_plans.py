"""The feed-forward products in every form of their plan (see test_ffn_plans.py), the CTA pairs among them: results,
repeats, two calls at once, and a captured graph."""
import ctypes

import pytest
import torch

from normalisation_row_bf16_b200 import build as nbuild
from normalisation_row_bf16_b200 import ops
from test_ffn_plans import DW, DX, FWD, MXFP8, PAIR_SHAPES, PLENTY, SINGLE_SHAPES, form, plan
from test_gpu_gated_ffn import BF, check_bwd, check_fwd, check_mxfp8, h_bounds, half_step, inputs, mma_rows, mx_case, product_bounds, rand

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, scope="module")
def _built():
    nbuild.build()


def on_device(product, T, D, F):
    out = (ctypes.c_int * 8)()
    assert ops.lib().mxnorm_debug_ffn_plan(product, T, D, F, 0, 0, PLENTY, out) == ops.MXN_OK
    return tuple(out)


def test_shapes_take_pairs_on_this_device():
    """The forms that test_ffn_plans.py counts on 148 SMs and 74 pairs are this device's."""
    L = ops.lib()
    for shapes in (PAIR_SHAPES, SINGLE_SHAPES):
        for product in shapes:
            for s in shapes[product]:
                assert on_device(product, *s) == plan(L, product, *s), (product, s)


@pytest.mark.parametrize("T,D,F", PAIR_SHAPES[FWD] + SINGLE_SHAPES[FWD])
def test_forward(T, D, F):
    x, wg, wu = inputs(T, D, F, seed=T)
    h, gate, up = ops.gated_ffn_fwd(x, wg, wu, act="gelu_tanh", save=True)
    check_fwd(x, wg, wu, "gelu_tanh", h, gate, up)
    assert torch.equal(h, ops.gated_ffn_fwd(x, wg, wu, act="gelu_tanh")[0])
    assert ops.device_status() == ops.MXN_OK


def backward_case(T, D, F):
    """dh, x, weights and projections: the backward takes any gate and up."""
    x, wg, wu = inputs(T, D, F, seed=T)
    return rand((T, F), 5, 0.1), x, wg, wu, rand((T, F), 6), rand((T, F), 7)


@pytest.mark.parametrize("T,D,F", PAIR_SHAPES[DX] + SINGLE_SHAPES[DX])
def test_dx(T, D, F):
    case = backward_case(T, D, F)
    dx, none, _ = ops.gated_ffn_bwd(*case, want_dw=False)
    assert none is None
    check_bwd(*case, "silu", dx, None, None)
    assert ops.device_status() == ops.MXN_OK


@pytest.mark.parametrize("T,D,F", PAIR_SHAPES[DW] + SINGLE_SHAPES[DW])
def test_dw(T, D, F):
    case = backward_case(T, D, F)
    _, dwg, dwu = ops.gated_ffn_bwd(*case, want_dx=False)
    check_bwd(*case, "silu", None, dwg, dwu)
    assert ops.device_status() == ops.MXN_OK


def test_strided_operands_on_pairs():
    T, D, F = PAIR_SHAPES[FWD][1]
    x, wg, wu = inputs(T, D, F, seed=3, pad=24)
    check_fwd(x, wg, wu, "silu", *ops.gated_ffn_fwd(x, wg, wu, save=True))
    T, D, F = PAIR_SHAPES[DX][4]
    x, wg, wu = inputs(T, D, F, seed=3, pad=24)
    case = (rand((T, F), 5, 0.1), x, wg, wu, rand((T, F), 6), rand((T, F), 7))
    check_bwd(*case, "silu", *ops.gated_ffn_bwd(*case))


def mx_inputs(T, F, K, seed=0):
    (aq, as_, _), (gq, gs, _), (uq, us, _) = mx_case(T, F, K, seed)
    return aq, as_, gq, gs, uq, us, T, F, K


MX_SINGLE, MX_PAIR = (300, 6272, 256), (600, 9440, 256)


def calls():
    """Name -> (inputs of a seed, call of the inputs and a stream), the pairs' kernels and the split ones."""
    def fwd(shape):
        return (lambda seed: inputs(*shape, seed=seed),
                lambda a, s: ops.gated_ffn_fwd(*a, save=True, stream=s))

    def bwd(shape, **kw):
        def make(seed):
            T, D, F = shape
            return (rand((T, F), seed, 0.1), *inputs(T, D, F, seed=seed + 1), rand((T, F), seed + 5), rand((T, F), seed + 6))
        return make, lambda a, s: [t for t in ops.gated_ffn_bwd(*a, stream=s, **kw) if t is not None]

    def mx(shape, out):
        return (lambda seed: mx_inputs(*shape, seed=seed),
                lambda a, s: [t for t in ops.mxfp8_gated_ffn(*a, out=out, stream=s) if t is not None])
    return {
        "forward, pairs": fwd(PAIR_SHAPES[FWD][1]),
        "forward, pairs, dealt": fwd(PAIR_SHAPES[FWD][3]),
        "dx, pairs, dealt and odd": bwd(PAIR_SHAPES[DX][4], want_dw=False),
        "dx, pairs, split": bwd(PAIR_SHAPES[DX][6], want_dw=False),
        "dx, split": bwd((333, 1032, 2744), want_dw=False),
        "dw, pairs, dealt and odd": bwd(PAIR_SHAPES[DW][6], want_dx=False),
        "dw, split": bwd((4096, 512, 1408), want_dx=False),
        "mxfp8": mx(MX_SINGLE, "bf16"),
        "mxfp8, pairs": mx(MX_PAIR, "bf16"),
        "mxfp8, pairs, codes": mx(MX_PAIR, "e4m3"),
    }


CALLS = calls()


def test_mxfp8_shapes_take_both_forms():
    assert on_device(MXFP8, MX_SINGLE[0], MX_SINGLE[2], MX_SINGLE[1])[0] == 0
    assert on_device(MXFP8, MX_PAIR[0], MX_PAIR[2], MX_PAIR[1])[0] == 1


@pytest.mark.parametrize("name", list(CALLS))
def test_repeats_bit_for_bit(name):
    make, call = CALLS[name]
    args = make(1)
    want = call(args, None)
    for _ in range(12):
        assert all(torch.equal(a, b) for a, b in zip(call(args, None), want))
    assert ops.device_status() == ops.MXN_OK


@pytest.mark.parametrize("name", list(CALLS))
def test_two_calls_at_once(name):
    make, call = CALLS[name]
    sets = [make(1), make(31)]
    want = [call(s, None) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        got = [call(s, st) for s, st in zip(sets, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert ops.device_status() == ops.MXN_OK


@pytest.mark.parametrize("name", list(CALLS))
def test_captured_and_replayed(name):
    """Two graphs that share a pool, replayed in turn on inputs that change in place, agree with plain calls."""
    make, call = CALLS[name]
    args, other = make(1), make(31)
    call(args, None)
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    with torch.cuda.graph(graphs[0]):
        outs.append(call(args, None))
    with torch.cuda.graph(graphs[1], pool=graphs[0].pool()):
        outs.append(call(args, None))
    for source in (other, make(1)):
        for a, b in zip(args, source):
            if isinstance(a, torch.Tensor):
                a.copy_(b)
        want = call(args, None)
        for g, o in zip(graphs, outs):
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(o, want))


def test_mxfp8_offsets_past_32_bits():
    """Rows behind the 2^31st element of h, as bf16 and as codes."""
    T, F, K = 150100, 14336, 128
    (aq, as_, av), (gq, gs, gv), (uq, us, uv) = mx_case(T, F, K)
    at = 2 ** 31 // F - 2
    rows = [slice(at, at + 5), slice(T - 3, T)]
    bounds = [h_bounds(*product_bounds(av[r], gv, uv, K), "silu") for r in rows]
    h, _ = ops.mxfp8_gated_ffn(aq, as_, gq, gs, uq, us, T, F, K)
    for r, (rh, eh) in zip(rows, bounds):
        assert ((h[r].double() - rh).abs() <= half_step(BF, rh.abs() + eh) + eh).all()
    del h
    for layout in (ops.SCALES_ROWMAJOR, ops.SCALES_MMA):
        q, s = ops.mxfp8_gated_ffn(aq, as_, gq, gs, uq, us, T, F, K, out="e4m3", scale_layout=layout)
        if layout == ops.SCALES_MMA:
            s = mma_rows(s, T, F // 32)
        for r, (rh, eh) in zip(rows, bounds):
            check_mxfp8(rh, eh, q[r], s[r])
    assert ops.device_status() == ops.MXN_OK
