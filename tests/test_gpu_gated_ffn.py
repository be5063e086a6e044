"""The gated feed-forward operators, bf16 and MXFP8, against the formulas in float64.

Bounds: a product of K terms accumulated in fp32 tensor memory is off by at
most `acc(K)` of the sum of the terms' magnitudes (one rounding of up to 2^-22
for each step of 16 or 32 terms and as many again inside it, whatever the
rounding mode); the activations' exp, division and erfc are good to a few
2^-23 and the argument's 2^-23 |g|; each output adds half a step of its type.
"""
import math

import pytest
import torch

from normalisation_row_bf16_b200 import build as nbuild
from normalisation_row_bf16_b200 import ops

pytestmark = pytest.mark.gpu

ACTS = ["silu", "gelu", "gelu_tanh"]
BF = torch.bfloat16


@pytest.fixture(autouse=True, scope="module")
def _built():
    nbuild.build()


def acc(K):
    return (K / 16 + 16) * 2.0 ** -22


def half_step(t, v):
    f = torch.finfo(t)
    return v.abs() * (f.eps / 2) + f.smallest_normal * f.eps / 2


def act(g, name):
    if name == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * torch.sigmoid(-g))
    if name == "gelu":
        phi = torch.special.ndtr(g)
        return g * phi, phi + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g ** 3))
    return g * (1 + t) / 2, (1 + t) / 2 + g * (1 - t * t) / 2 * k * (1 + 3 * 0.044715 * g * g)


def act_err(g, a):
    """Bound on the kernel's activation: relative to its value, and absolute where the value underflows."""
    return a.abs() * (24 + 4 * g.abs() + 4 * g.abs() ** 3) * 2.0 ** -23 + 1e-36


def rand(shape, seed, scale=1.0, pad=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(shape[0], shape[1] + pad, generator=g, device="cuda") * scale).to(BF)[:, :shape[1]]


def inputs(T, D, F, seed=0, pad=0, wscale=None):
    ws = 1.3 / math.sqrt(D) if wscale is None else wscale
    return rand((T, D), seed, pad=pad), rand((F, D), seed + 1, ws, pad), rand((F, D), seed + 2, ws, pad)


def product_bounds(x, wg, wu, K):
    gate, up = x @ wg.t(), x @ wu.t()
    return gate, up, acc(K) * (x.abs() @ wg.abs().t()), acc(K) * (x.abs() @ wu.abs().t())


def h_bounds(gate, up, eg, eu, name):
    a, _ = act(gate, name)
    ea = act_err(gate, a) + 1.2 * eg          # |act'| <= 1.13
    h = a * up
    return h, ea * (up.abs() + eu) + a.abs() * eu + h.abs() * 2.0 ** -23


def check_fwd(x, wg, wu, name, h, gate=None, up=None):
    K = x.shape[1]
    rg, ru, eg, eu = product_bounds(x.double(), wg.double(), wu.double(), K)
    rh, eh = h_bounds(rg, ru, eg, eu, name)
    for got, ref, err in ((h, rh, eh), (gate, rg, eg), (up, ru, eu)):
        if got is not None:
            assert ((got.double() - ref).abs() <= half_step(BF, ref.abs() + err) + err).all()


FWD_SHAPES = [(1, 8, 8), (1, 64, 16), (3, 72, 40), (16, 256, 264), (127, 128, 128), (128, 512, 392), (129, 520, 1000),
              (333, 1032, 2744), (1, 4096, 4096), (64, 1024, 2816), (300, 264, 4736), (1029, 256, 520), (2050, 136, 264)]


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("T,D,F", FWD_SHAPES)
def test_forward(T, D, F, name):
    x, wg, wu = inputs(T, D, F, seed=T + D + F)
    h, gate, up = ops.gated_ffn_fwd(x, wg, wu, act=name, save=True)
    check_fwd(x, wg, wu, name, h, gate, up)
    h1, g1, u1 = ops.gated_ffn_fwd(x, wg, wu, act=name)
    assert g1 is None and u1 is None and torch.equal(h, h1)
    assert ops.device_status() == ops.MXN_OK


@pytest.mark.parametrize("T,D,F,pad", [(50, 256, 264, 8), (130, 264, 128, 24), (1, 512, 64, 8)])
def test_strided_operands(T, D, F, pad):
    x, wg, wu = inputs(T, D, F, pad=pad)
    h, gate, up = ops.gated_ffn_fwd(x, wg, wu, save=True)
    check_fwd(x, wg, wu, "silu", h, gate, up)
    dh = rand((T, F), 9, 0.1)
    check_bwd(dh, x, wg, wu, gate, up, "silu", *ops.gated_ffn_bwd(dh, x, wg, wu, gate, up))


@pytest.mark.parametrize("name", ACTS)
def test_far_gates(name):
    """Gates from -200 to 200: the activation's limits, without NaN."""
    T, D, F = 8, 8, 48
    x = torch.zeros(T, D, device="cuda", dtype=BF)
    x[:, 0] = torch.tensor([-200.0, -90.0, -30.0, -6.0, 0.0, 6.0, 90.0, 200.0], device="cuda").to(BF)
    x[:, 1] = 1.0
    wg, wu = torch.zeros(F, D, device="cuda", dtype=BF), torch.zeros(F, D, device="cuda", dtype=BF)
    wg[:, 0] = 1.0
    wu[:, 1] = torch.linspace(-2, 2, F, device="cuda").to(BF)
    h, gate, up = ops.gated_ffn_fwd(x, wg, wu, act=name, save=True)
    check_fwd(x, wg, wu, name, h, gate, up)
    dh = torch.ones(T, F, device="cuda", dtype=BF)
    check_bwd(dh, x, wg, wu, gate, up, name, *ops.gated_ffn_bwd(dh, x, wg, wu, gate, up, act=name))


def test_nonfinite_tokens_stay_apart():
    x, wg, wu = inputs(140, 128, 264)
    h = ops.gated_ffn_fwd(x, wg, wu)[0]
    x = x.clone()
    x[5] = float("nan")
    x[131, 3] = float("inf")
    h1 = ops.gated_ffn_fwd(x, wg, wu)[0]
    keep = [i for i in range(140) if i not in (5, 131)]
    assert torch.equal(h[keep], h1[keep]) and h1[5].isnan().all()


# ------------------------------------------------------------------- backward

def interval(v, err):
    """Width of what v +- err may round to in bf16, and the rounded value."""
    lo, hi = (v - err).to(BF).double(), (v + err).to(BF).double()
    return v.to(BF).double(), hi - lo


def check_bwd(dh, x, wg, wu, gate, up, name, dx, dwg, dwu):
    T, D = x.shape
    F = wg.shape[0]
    dh, x, wg, wu, g, u = (t.double() for t in (dh, x, wg, wu, gate, up))
    a, da = act(g, name)
    # derivative: s and its complement to a few 2^-23 and the argument's error
    e_da = (40 + 8 * g.abs() + 8 * g.abs() ** 3) * 2.0 ** -23 * (da.abs() + (g.abs() + 1) * torch.exp(-g.abs())) + 1e-36
    du, wu_du = interval(dh * a, dh.abs() * act_err(g, a) + (dh * a).abs() * 2.0 ** -23)
    dg, wu_dg = interval(dh * u * da, (dh * u).abs() * e_da + (dh * u * da).abs() * 2.0 ** -22)
    if dx is not None:
        ref = dg @ wg + du @ wu
        err = wu_dg @ wg.abs() + wu_du @ wu.abs() + acc(2 * F) * (dg.abs() @ wg.abs() + du.abs() @ wu.abs())
        assert ((dx.double() - ref).abs() <= half_step(BF, ref.abs() + err) + err).all()
    for got, d, w in ((dwg, dg, wu_dg), (dwu, du, wu_du)):
        if got is not None:
            ref = d.t() @ x
            err = w.t() @ x.abs() + acc(T) * (d.abs().t() @ x.abs())
            assert ((got.double() - ref).abs() <= half_step(BF, ref.abs() + err) + err).all()


BWD_SHAPES = [(1, 8, 8), (1, 64, 64), (3, 72, 40), (16, 256, 264), (63, 128, 128), (64, 512, 392), (129, 520, 1000),
              (333, 1032, 2744), (300, 264, 4736), (1029, 256, 520), (2050, 136, 264), (70, 2056, 72)]


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("T,D,F", BWD_SHAPES)
def test_backward(T, D, F, name):
    x, wg, wu = inputs(T, D, F, seed=T + D + F)
    dh = rand((T, F), 77, 0.1)
    _, gate, up = ops.gated_ffn_fwd(x, wg, wu, act=name, save=True)
    check_bwd(dh, x, wg, wu, gate, up, name, *ops.gated_ffn_bwd(dh, x, wg, wu, gate, up, act=name))
    assert ops.device_status() == ops.MXN_OK


def test_backward_selected_gradients():
    x, wg, wu = inputs(100, 256, 264)
    dh = rand((100, 264), 3)
    _, gate, up = ops.gated_ffn_fwd(x, wg, wu, save=True)
    full = ops.gated_ffn_bwd(dh, x, wg, wu, gate, up)
    dx, a, b = ops.gated_ffn_bwd(dh, x, wg, wu, gate, up, want_dw=False)
    assert a is None and b is None and torch.equal(dx, full[0])
    dx, a, b = ops.gated_ffn_bwd(dh, x, wg, wu, gate, up, want_dx=False)
    assert dx is None and torch.equal(a, full[1]) and torch.equal(b, full[2])
    assert ops.gated_ffn_bwd(dh, x, wg, wu, gate, up, want_dx=False, want_dw=False) == (None, None, None)


def test_empty_batch():
    x, wg, wu = inputs(4, 64, 128)
    x = x[:0]
    h, gate, up = ops.gated_ffn_fwd(x, wg, wu, save=True)
    assert h.shape == (0, 128)
    dx, dwg, dwu = ops.gated_ffn_bwd(h, x, wg, wu, gate, up)
    assert dx.shape == (0, 64) and (dwg == 0).all() and (dwu == 0).all()


@pytest.mark.parametrize("T,D,F", [(37, 136, 72), (129, 264, 328)])
def test_memory_around_the_outputs_is_left_alone(T, D, F):
    x, wg, wu = inputs(T, D, F)
    dh = rand((T, F), 3)

    def guarded(rows, cols):
        b = torch.full((rows * cols + 4096,), 7.0, device="cuda", dtype=BF)
        return b, b[:rows * cols]
    (hb, h), (gb, g), (ub, u) = guarded(T, F), guarded(T, F), guarded(T, F)
    ops.gated_ffn_fwd(x, wg, wu, h=h, gate=g, up=u)
    (xb, dx), (ab, dwg), (bb, dwu) = guarded(T, D), guarded(F, D), guarded(F, D)
    ops.gated_ffn_bwd(dh, x, wg, wu, g.view(T, F), u.view(T, F), dx=dx, dw_gate=dwg, dw_up=dwu)
    for b in (hb, gb, ub, xb, ab, bb):
        assert (b[-4096:] == 7).all()


def test_repeats_bit_for_bit():
    x, wg, wu = inputs(700, 512, 1032)
    dh = rand((700, 1032), 3)
    first = None
    for _ in range(24):
        h, gate, up = ops.gated_ffn_fwd(x, wg, wu, save=True)
        out = (h, gate, up, *ops.gated_ffn_bwd(dh, x, wg, wu, gate, up))
        if first is None:
            first = out
        assert all(torch.equal(a, b) for a, b in zip(out, first))


def test_other_stream_and_graph():
    x, wg, wu = inputs(200, 256, 520)
    dh = rand((200, 520), 3)

    def step(stream=None):
        h, gate, up = ops.gated_ffn_fwd(x, wg, wu, save=True, stream=stream)
        return (h, *ops.gated_ffn_bwd(dh, x, wg, wu, gate, up, stream=stream))
    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    with torch.cuda.graph(graphs[0]):
        outs.append(step())
    with torch.cuda.graph(graphs[1], pool=graphs[0].pool()):
        outs.append(step())
    for scale in (1.0, 0.5):
        x.mul_(scale)
        want = step()
        for gr, o in zip(graphs, outs):
            gr.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(o, want))


def test_binding_refusals():
    x, wg, wu = inputs(8, 64, 32)
    h, gate, up = ops.gated_ffn_fwd(x, wg, wu, save=True)
    for bad in (lambda: ops.gated_ffn_fwd(x, wg, wu, act="tanh"), lambda: ops.gated_ffn_fwd(x[0], wg, wu),
                lambda: ops.gated_ffn_fwd(x, wg, wu[:16]), lambda: ops.gated_ffn_fwd(x, wg[:, :32], wu),
                lambda: ops.gated_ffn_fwd(x.float(), wg, wu), lambda: ops.gated_ffn_fwd(x, wg.cpu(), wu),
                lambda: ops.gated_ffn_fwd(x, wg.t().contiguous().t(), wu),
                lambda: ops.gated_ffn_fwd(x, wg, wu, h=h[:2].clone()),
                lambda: ops.gated_ffn_fwd(x, rand((32, 64), 1, pad=8), wu),       # weights of unlike strides
                lambda: ops.gated_ffn_bwd(h[:4], x, wg, wu, gate, up),
                lambda: ops.gated_ffn_bwd(h, x, wg, wu, gate.float(), up),
                lambda: ops.gated_ffn_bwd(h, x, wg, wu, gate, up, workspace=torch.empty(64, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    x4, wg4, wu4 = inputs(8, 60, 32)
    with pytest.raises(ops.MXNormError):
        ops.gated_ffn_fwd(x4, wg4, wu4)              # D not a multiple of 8
    with pytest.raises(ops.MXNormError):
        ops.gated_ffn_fwd(*inputs(8, 64, 36))        # F not a multiple of 8
    with pytest.raises(ops.MXNormError):
        ops.gated_ffn_fwd(rand((8, 64), 1, pad=4), wg, wu)   # rows off 16 bytes


def test_training_chain_against_differences():
    """layernorm -> gated projection -> back: the gradients that reach x and the weights, against central
    differences of the same chain in float64 along random directions."""
    T, D, F = 40, 128, 264
    x, wg, wu = inputs(T, D, F, seed=4)
    g = torch.Generator(device="cuda").manual_seed(8)
    gamma = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(BF)
    beta = (0.1 * torch.randn(D, generator=g, device="cuda")).to(BF)
    dh = rand((T, F), 5)
    y, mean, rstd = ops.layernorm_fwd(x, gamma, beta)
    h, gate, up = ops.gated_ffn_fwd(y, wg, wu, save=True)
    dy, dwg, dwu = ops.gated_ffn_bwd(dh, y, wg, wu, gate, up)
    dx, dgamma, dbeta = ops.layernorm_bwd(x, dy, gamma, mean, rstd)

    def loss(x, gamma, beta, wg, wu):
        n = (x - x.mean(1, keepdim=True)) * (x.var(1, unbiased=False, keepdim=True) + 1e-5).rsqrt() * gamma + beta
        return (act(n @ wg.t(), "silu")[0] * (n @ wu.t()) * dh.double()).sum()
    at = [t.double() for t in (x, gamma, beta, wg, wu)]
    for i, got in enumerate((dx, dgamma, dbeta, dwg, dwu)):
        # along the gradient's own signs every term adds up: the sum is its 1-norm, and bf16's roundings (a few
        # 2^-8 of each term: y, gate, up, dg, du, dy and the result) stay a small share of it
        v = got.double().sign()
        step = 1e-6
        hi, lo = list(at), list(at)
        hi[i], lo[i] = at[i] + step * v, at[i] - step * v
        want = (loss(*hi) - loss(*lo)) / (2 * step)
        assert (got.double().abs().sum() - want).abs() <= 7 * 2.0 ** -8 * want.abs()


# ---------------------------------------------------------------------- MXFP8

def quantised(rows, K, seed, scale=1.0, pattern=None):
    w = rand((rows, K), seed, scale) if pattern is None else pattern
    q, s = ops.mxfp8_cast(w, scale_layout=ops.SCALES_MMA)
    row = ops.mxfp8_cast(w)[1]
    v = q.view(torch.float8_e4m3fn).double().view(rows, K // 32, 32) * torch.exp2(row.double() - 127)[..., None]
    return q, s, v.view(rows, K)


def mx_case(T, F, K, seed=0):
    ws = 1.3 / math.sqrt(K)
    return quantised(T, K, seed), quantised(F, K, seed + 1, ws), quantised(F, K, seed + 2, ws)


def mma_rows(s, rows, blocks):
    """Row-major [rows, blocks] view of scales in the MMA layout."""
    kp = -(-blocks // 4) * 4
    t = s[:(-(-rows // 128) * 128) * kp].view(-1, kp // 4, 32, 4, 4)
    return t.permute(0, 3, 2, 1, 4).reshape(-1, kp)[:rows, :blocks]


def check_mxfp8(h, eh, codes, scales):
    T, F = h.shape
    b, e = h.view(T, F // 32, 32), eh.view(T, F // 32, 32)
    amax = b.abs().amax(-1)
    slack = e.amax(-1)

    def exponent(a):
        m, x = torch.frexp(a)
        return torch.where(a > 0, x - 9 + (m > 0.875).to(x.dtype), -127).clamp(-127, 127)
    got = scales.to(torch.int32) - 127
    assert (got >= exponent((amax - slack).clamp(min=0))).all() and (got <= exponent(amax + slack)).all()
    inv = torch.exp2(-got.double())[..., None]
    lim = lambda v: (v * inv).clamp(-448, 448).float().to(torch.float8_e4m3fn).double()  # noqa: E731
    val = codes.view(torch.float8_e4m3fn).double().view_as(b)
    # fp32 rounds the end points once more on their way to E4M3: widen by it
    d = e + b.abs() * 2.0 ** -23
    assert ((val >= lim(b - d)) & (val <= lim(b + d))).all()


MX_SHAPES = [(1, 8, 128), (1, 256, 512), (3, 40, 128), (16, 512, 1024), (127, 128, 256), (129, 264, 384), (300, 1000, 512),
             (1, 4096, 4096), (700, 1544, 256)]


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("T,F,K", MX_SHAPES)
def test_mxfp8_bf16_output(T, F, K, name):
    (aq, as_, av), (gq, gs, gv), (uq, us, uv) = mx_case(T, F, K, seed=T + F)
    h, none = ops.mxfp8_gated_ffn(aq, as_, gq, gs, uq, us, T, F, K, act=name)
    assert none is None
    rh, eh = h_bounds(*product_bounds(av, gv, uv, K), name)
    assert ((h.double() - rh).abs() <= half_step(BF, rh.abs() + eh) + eh).all()
    assert ops.device_status() == ops.MXN_OK


@pytest.mark.parametrize("name", ACTS)
@pytest.mark.parametrize("T,F,K", [(1, 32, 128), (5, 64, 256), (128, 256, 512), (130, 288, 384), (300, 992, 512)])
def test_mxfp8_quantised_output(T, F, K, name):
    (aq, as_, av), (gq, gs, gv), (uq, us, uv) = mx_case(T, F, K, seed=T + F)
    rh, eh = h_bounds(*product_bounds(av, gv, uv, K), name)
    q, s = ops.mxfp8_gated_ffn(aq, as_, gq, gs, uq, us, T, F, K, act=name, out="e4m3", scale_layout=ops.SCALES_ROWMAJOR)
    check_mxfp8(rh, eh, q, s)
    q1, s1 = ops.mxfp8_gated_ffn(aq, as_, gq, gs, uq, us, T, F, K, act=name, out="e4m3")
    assert torch.equal(q, q1) and torch.equal(s, mma_rows(s1, T, F // 32))


def test_mxfp8_padding_scales_do_not_matter():
    """Scale bytes of rows that do not exist (0xFF, NaN) leave the result as it is."""
    T, F, K = 5, 40, 256
    (aq, as_, _), (gq, gs, _), (uq, us, _) = mx_case(T, F, K)
    h = ops.mxfp8_gated_ffn(aq, as_, gq, gs, uq, us, T, F, K)[0]

    def spoiled(s, rows):
        t = torch.full_like(s, 0xFF)
        at = torch.arange(s.numel(), device="cuda")
        row = (at // 512 // (K // 128)) * 128 + (at % 512 % 16) // 4 * 32 + at % 512 // 16
        return torch.where(row < rows, s, t)
    h1 = ops.mxfp8_gated_ffn(aq, spoiled(as_, T), gq, spoiled(gs, F), uq, spoiled(us, F), T, F, K)[0]
    assert torch.equal(h, h1)


def test_mxfp8_nonfinite_and_zero_blocks():
    T, F, K = 40, 96, 128
    w = rand((T, K), 1)
    w[3, 40] = float("nan")
    w[7] = 0.0
    (aq, as_, _), (gq, gs, _), (uq, us, _) = quantised(T, K, 0, pattern=w), *mx_case(T, F, K)[1:]
    h = ops.mxfp8_gated_ffn(aq, as_, gq, gs, uq, us, T, F, K)[0]
    q, s = ops.mxfp8_gated_ffn(aq, as_, gq, gs, uq, us, T, F, K, out="e4m3", scale_layout=ops.SCALES_ROWMAJOR)
    assert h[3].isnan().all() and (q[3] == 0x7F).all() and (s[3] == 0xFF).all()
    assert (h[7] == 0).all() and ((q[7] & 0x7F) == 0).all() and (s[7] == 0).all()
    keep = [i for i in range(T) if i != 3]
    assert torch.isfinite(h[keep].float()).all() and (s[keep] != 0xFF).all()


def test_mxfp8_memory_around_the_outputs_is_left_alone():
    T, F, K = 37, 96, 128
    (aq, as_, _), (gq, gs, _), (uq, us, _) = mx_case(T, F, K)
    hb = torch.full((T * F + 4096,), 7.0, device="cuda", dtype=BF)
    ops.mxfp8_gated_ffn(aq, as_, gq, gs, uq, us, T, F, K, h=hb[:T * F])
    assert (hb[T * F:] == 7).all()
    qb = torch.full((T * F + 4096,), 7, device="cuda", dtype=torch.uint8)
    n = ops.scales_bytes(T, F, ops.SCALES_MMA)
    sb = torch.full((n + 4096,), 9, device="cuda", dtype=torch.uint8)
    ops.mxfp8_gated_ffn(aq, as_, gq, gs, uq, us, T, F, K, out="e4m3", h=qb[:T * F], h_s=sb[:n])
    assert (qb[T * F:] == 7).all() and (sb[n:] == 9).all()


def test_mxfp8_refusals():
    T, F, K = 8, 64, 128
    (aq, as_, _), (gq, gs, _), (uq, us, _) = mx_case(T, F, K)
    for bad in (lambda: ops.mxfp8_gated_ffn(aq[:4], as_, gq, gs, uq, us, T, F, K),
                lambda: ops.mxfp8_gated_ffn(aq, as_[:64], gq, gs, uq, us, T, F, K),
                lambda: ops.mxfp8_gated_ffn(aq, as_, gq, None, uq, us, T, F, K),
                lambda: ops.mxfp8_gated_ffn(aq, as_, gq, gs, uq, us, T, F, K, act="x"),
                lambda: ops.mxfp8_gated_ffn(aq, as_, gq, gs, uq, us, T, F, K, out="fp8"),
                lambda: ops.mxfp8_gated_ffn(aq, as_, gq, gs, uq.cpu(), us, T, F, K),
                lambda: ops.mxfp8_gated_ffn(aq, as_, gq, gs, uq, us, T, F, K, h_s=gs)):
        with pytest.raises(ValueError):
            bad()
    for f, k, out in ((64, 96, "bf16"), (60, 128, "bf16"), (40, 128, "e4m3")):
        with pytest.raises(ops.MXNormError):
            ops.mxfp8_gated_ffn(aq, as_, gq, gs, uq, us, T, f, k, out=out)


def test_serving_chain():
    """mxnorm_fwd -> mxfp8_gated_ffn -> mxfp8_gemm: each step on the codes of the one before, the last against the
    product of what the second wrote."""
    T, D, F = 256, 256, 512
    x = rand((T, D), 3)
    gamma = torch.ones(D, device="cuda", dtype=BF)
    aq, as_, _ = ops.mxnorm_fwd(x, gamma, scale_layout=ops.SCALES_MMA)
    a_row = ops.mxnorm_fwd(x, gamma)[1]
    av = (aq.view(torch.float8_e4m3fn).double().view(T, D // 32, 32) * torch.exp2(a_row.double() - 127)[..., None]).view(T, D)
    gq, gs, gv = quantised(F, D, 5, 0.08)
    uq, us, uv = quantised(F, D, 6, 0.08)
    dq, ds, dv = quantised(256, F, 7, 0.05)
    q, s = ops.mxfp8_gated_ffn(aq, as_, gq, gs, uq, us, T, F, D, out="e4m3")
    s_row = mma_rows(s, T, F // 32)
    rh, eh = h_bounds(*product_bounds(av, gv, uv, D), "silu")
    check_mxfp8(rh, eh, q, s_row)
    y = ops.mxfp8_gemm(q, s, dq, ds, T, 256, F)
    hv = (q.view(torch.float8_e4m3fn).double().view(T, F // 32, 32) * torch.exp2(s_row.double() - 127)[..., None]).view(T, F)
    ref = hv @ dv.t()
    err = acc(F) * (hv.abs() @ dv.abs().t())
    assert ((y.double() - ref).abs() <= half_step(BF, ref.abs() + err) + err).all()


def test_offsets_past_32_bits():
    """Rows behind the 2^31st element of h, forward and backward."""
    T, D, F = 150100, 64, 14336
    x, wg, wu = inputs(T, D, F)
    h, _, _ = ops.gated_ffn_fwd(x, wg, wu)
    at = 2 ** 31 // F - 2
    for r in (slice(at, at + 5), slice(T - 3, T)):
        check_fwd(x[r], wg, wu, "silu", h[r])
    gate = h
    dx, dwg, dwu = ops.gated_ffn_bwd(h, x, wg, wu, gate, gate, want_dw=False)
    for r in (slice(at, at + 5), slice(T - 3, T)):
        check_bwd(h[r], x[r], wg, wu, gate[r], gate[r], "silu", dx[r], None, None)


@pytest.mark.parametrize("T,D,F", [(700, 512, 1032), (4096, 256, 2048)])
def test_two_calls_at_once(T, D, F):
    """Calls on two streams do not disturb one another: small tiles and pairs of CTAs."""
    sets = [(*inputs(T, D, F, seed=s), rand((T, F), s + 50, 0.1)) for s in (1, 7)]

    def step(x, wg, wu, dh, stream=None):
        h, gate, up = ops.gated_ffn_fwd(x, wg, wu, save=True, stream=stream)
        return (h, *ops.gated_ffn_bwd(dh, x, wg, wu, gate, up, stream=stream))
    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(6):
        got = [step(*s, stream=st) for s, st in zip(sets, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert ops.device_status() == ops.MXN_OK


# Shapes that reach every plan of the products: one and several rounds of single CTAs and of pairs, whole 512-row tiles,
# halves and the odd half, split contractions.
PLAN_SHAPES = [(257, 512, 4096), (513, 256, 1024), (768, 4096, 2048), (1281, 1536, 4096), (2300, 1024, 4104), (5000, 512, 3000)]


@pytest.mark.parametrize("T,D,F", PLAN_SHAPES)
def test_plans(T, D, F):
    x, wg, wu = inputs(T, D, F, seed=T)
    h, gate, up = ops.gated_ffn_fwd(x, wg, wu, act="gelu", save=True)
    check_fwd(x, wg, wu, "gelu", h, gate, up)
    dh = rand((T, F), 5, 0.1)
    check_bwd(dh, x, wg, wu, gate, up, "gelu", *ops.gated_ffn_bwd(dh, x, wg, wu, gate, up, act="gelu"))
    assert ops.device_status() == ops.MXN_OK


@pytest.mark.parametrize("T,F,K", [(257, 1024, 512), (1000, 4096, 256), (2300, 3104, 384)])
def test_mxfp8_plans(T, F, K):
    (aq, as_, av), (gq, gs, gv), (uq, us, uv) = mx_case(T, F, K, seed=T)
    rh, eh = h_bounds(*product_bounds(av, gv, uv, K), "gelu")
    h, _ = ops.mxfp8_gated_ffn(aq, as_, gq, gs, uq, us, T, F, K, act="gelu")
    assert ((h.double() - rh).abs() <= half_step(BF, rh.abs() + eh) + eh).all()
    q, s = ops.mxfp8_gated_ffn(aq, as_, gq, gs, uq, us, T, F, K, act="gelu", out="e4m3")
    check_mxfp8(rh, eh, q, mma_rows(s, T, F // 32))
    assert ops.device_status() == ops.MXN_OK


def test_mxfp8_repeats_bit_for_bit():
    T, F, K = 600, 1056, 512
    (aq, as_, _), (gq, gs, _), (uq, us, _) = mx_case(T, F, K)
    first = None
    for _ in range(24):
        out = ops.mxfp8_gated_ffn(aq, as_, gq, gs, uq, us, T, F, K, out="e4m3", scale_layout=ops.SCALES_ROWMAJOR)
        first = first or out
        assert all(torch.equal(a, b) for a, b in zip(out, first))


# Few tiles over a long batch: the weight gradients' contraction is dealt to partial products.
@pytest.mark.parametrize("T,D,F", [(2834, 600, 600), (4099, 136, 520), (8192, 64, 64), (3000, 1024, 1032), (4096, 512, 1408)])
def test_backward_long_batches(T, D, F):
    x, wg, wu = inputs(T, D, F, seed=T)
    _, gate, up = ops.gated_ffn_fwd(x, wg, wu, save=True)
    dh = rand((T, F), 5, 0.1)
    first = ops.gated_ffn_bwd(dh, x, wg, wu, gate, up)
    check_bwd(dh, x, wg, wu, gate, up, "silu", *first)
    n = ops.gated_ffn_bwd_workspace_bytes(T, D, F)
    ws = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    again = ops.gated_ffn_bwd(dh, x, wg, wu, gate, up, workspace=ws[:n])
    assert all(torch.equal(a, b) for a, b in zip(first, again)) and (ws[n:] == 0xA5).all()
    only = ops.gated_ffn_bwd(dh, x, wg, wu, gate, up, want_dx=False)
    assert all(torch.equal(a, b) for a, b in zip(first[1:], only[1:]))
    assert ops.device_status() == ops.MXN_OK
