"""Layer norm, forward and backward, against the formulas in float64.

Bounds: fp32 sums of n terms, at most `depth` additions deep, are off by at
most depth * 2^-24 of the sum of magnitudes; each output adds one rounding of
half a step of its type (finfo.eps / 2 relative, half the smallest subnormal
below the normal range).
"""
import pytest
import torch

from normalisation_row_bf16_b200 import build as nbuild
from normalisation_row_bf16_b200 import ops

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DEPTH = 72                       # a thread's 32 elements, 5 shuffle steps, up to 32 warps
TYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(autouse=True, scope="module")
def _built():
    nbuild.build()


def half_step(t, v):
    f = torch.finfo(t)
    return v.abs() * (f.eps / 2) + f.smallest_normal * f.eps / 2


def make(T, D, dtype, seed=0, pad=0, offset=0.0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(T, D + pad, generator=g, device="cuda") * scale
    x[:, :: 97] *= 50.0
    x += offset
    x = x.to(dtype)[:, :D]
    gamma = (1 + 0.1 * torch.randn(D, generator=g, device="cuda")).to(dtype)
    beta = (0.1 * torch.randn(D, generator=g, device="cuda")).to(dtype)
    return x, gamma, beta, g


def reference_fwd(x, gamma, beta, eps):
    """y, mean, rstd in float64 and the bound on the kernel's y."""
    x = x.double()
    mean = x.mean(1, keepdim=True)
    rstd = (x.var(1, unbiased=False, keepdim=True) + eps).rsqrt()
    xh = (x - mean) * rstd
    ga = torch.ones_like(xh[0]) if gamma is None else gamma.double()
    y = xh * ga + (0 if beta is None else beta.double())
    dmean = U * (DEPTH + 2) * x.abs().mean(1, keepdim=True)
    # rstd: half the relative error of var + eps, whose terms are off by dmean and 2^-24 of themselves
    dvar = U * (DEPTH + 6) * (x - mean).square().mean(1, keepdim=True) + dmean * dmean + 2 * dmean * (x - mean).abs().mean(1, keepdim=True)
    drstd = 0.5 * dvar * rstd ** 3 + 4 * U * rstd
    err = ga.abs() * (rstd * (dmean + U * (x - mean).abs()) + (x - mean).abs() * drstd + 3 * U * xh.abs()) + 2 * U * y.abs()
    return y, mean[:, 0], rstd[:, 0], err, dmean[:, 0], drstd[:, 0]


def check_fwd(x, gamma, beta, eps, y, mean, rstd):
    ry, rm, rr, err, dm, dr = reference_fwd(x, gamma, beta, eps)
    assert ((y.double() - ry).abs() <= half_step(x.dtype, ry.abs() + err) + err).all()
    if mean is not None:
        assert ((mean.double() - rm).abs() <= dm + U * rm.abs() + 1e-45).all()
        assert ((rstd.double() - rr).abs() <= dr).all()


SHAPES = [(1, 1), (1, 4096), (2, 7), (3, 32), (5, 33), (64, 1024), (7, 257), (130, 1544), (9, 2047), (33, 4096),
          (149, 5003), (4, 8192), (3, 16384), (2, 16383), (2, 32768), (2, 32767), (1200, 256)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,D", SHAPES)
def test_forward(T, D, dtype):
    x, gamma, beta, _ = make(T, D, dtype, seed=T + D)
    y, mean, rstd = ops.layernorm_fwd(x, gamma, beta)
    check_fwd(x, gamma, beta, 1e-5, y, mean, rstd)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("use_gamma,use_beta", [(False, False), (True, False), (False, True)])
def test_forward_without_parameters(dtype, use_gamma, use_beta):
    x, gamma, beta, _ = make(40, 800, dtype)
    gamma, beta = gamma if use_gamma else None, beta if use_beta else None
    y, mean, rstd = ops.layernorm_fwd(x, gamma, beta, eps=1e-3, want_stats=False)
    assert mean is None and rstd is None
    check_fwd(x, gamma, beta, 1e-3, y, None, None)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("D,pad", [(1024, 8), (1024, 1), (1021, 3), (1000, 24), (4096, 4)])
def test_strided_rows(D, pad, dtype):
    x, gamma, beta, g = make(50, D, dtype, pad=pad)
    y, mean, rstd = ops.layernorm_fwd(x, gamma, beta)
    check_fwd(x, gamma, beta, 1e-5, y, mean, rstd)
    dy = torch.randn(50, D + pad, generator=g, device="cuda").to(dtype)[:, :D]
    check_bwd(x, dy, gamma, mean, rstd, *ops.layernorm_bwd(x, dy, gamma, mean, rstd))
    check_bwd(x, dy.contiguous(), gamma, mean, rstd, *ops.layernorm_bwd(x, dy.contiguous(), gamma, mean, rstd))


@pytest.mark.parametrize("D", [512, 4096, 4095])
def test_offset_far_above_the_deviation(D):
    """The squares are summed about the mean: an offset of 1000 deviations costs what its own rounding costs."""
    x, gamma, beta, _ = make(20, D, torch.float32, offset=1000.0)
    y, mean, rstd = ops.layernorm_fwd(x, gamma, beta)
    check_fwd(x, gamma, beta, 1e-5, y, mean, rstd)


def test_constant_and_zero_rows():
    x = torch.zeros(3, 96, device="cuda")
    x[1] = 4.0
    x[2] = torch.arange(96.0)
    y, mean, rstd = ops.layernorm_fwd(x, eps=1e-5)
    assert (y[:2] == 0).all() and mean.tolist()[:2] == [0.0, 4.0]
    assert ((rstd[:2].double() - 1e-5 ** -0.5).abs() <= 4 * U * 1e-5 ** -0.5 + 317 * 1e-7).all()
    dx, dg, db = ops.layernorm_bwd(x, torch.ones_like(x), None, mean, rstd)
    assert dg is None and (db == 3).all() and (dx[:2] == 0).all()


@pytest.mark.parametrize("dtype", TYPES)
def test_nonfinite_rows_stay_apart(dtype):
    x, gamma, beta, _ = make(9, 640, dtype)
    clean = ops.layernorm_fwd(x, gamma, beta)
    x = x.clone()
    x[2, 5] = float("nan")
    x[6, 639] = float("inf")
    y, mean, rstd = ops.layernorm_fwd(x, gamma, beta)
    assert y[2].isnan().all() and y[6].isnan().all()
    keep = [0, 1, 3, 4, 5, 7, 8]
    assert torch.equal(y[keep], clean[0][keep]) and torch.equal(mean[keep], clean[1][keep])
    dy = torch.ones_like(x)
    dx, dg, db = ops.layernorm_bwd(x, dy, gamma, mean, rstd)
    dxc, _, _ = ops.layernorm_bwd(x[3:6].clone(), dy[3:6].clone(), gamma, mean[3:7].clone()[:3], rstd[3:7].clone()[:3])
    assert dx[2].isnan().all() and torch.equal(dx[3:6], dxc) and torch.isfinite(db.float()).all()


# ------------------------------------------------------------------- backward

def check_bwd(x, dy, gamma, mean, rstd, dx, dgamma, dbeta):
    t = x.dtype
    x, dy, m, r = x.double(), dy.double(), mean.double()[:, None], rstd.double()[:, None]
    T, D = x.shape
    g = dy if gamma is None else dy * gamma.double()
    xh = (x - m) * r
    e = U * (2 * (m * r).abs() + 2 * xh.abs() + (x * r).abs())           # of xh = a x + b
    c1, c2 = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    rdx = r * (g - c1 - xh * c2)
    d1 = U * (DEPTH + 4) * g.abs().mean(1, keepdim=True)
    d2 = U * (DEPTH + 6) * (g * xh).abs().mean(1, keepdim=True) + (g.abs() * e).mean(1, keepdim=True)
    err = r * (d1 + xh.abs() * d2 + e * (c2.abs() + d2) + U * (4 * g.abs() + 3 * (xh * c2).abs() + 3 * c1.abs()))
    assert ((dx.double() - rdx).abs() <= half_step(t, rdx.abs() + err) + err).all()
    depth = -(-T // 100) + 16 + 32        # rows a group, groups a CTA, CTAs (a device of 148 SMs)
    if dgamma is not None:
        rg, s = (dy * xh).sum(0), (dy * xh).abs().sum(0)
        eg = U * (depth + 2) * s + (dy.abs() * e).sum(0)
        assert ((dgamma.double() - rg).abs() <= half_step(t, rg.abs() + eg) + eg).all()
    if dbeta is not None:
        rb, eb = dy.sum(0), U * depth * dy.abs().sum(0)
        assert ((dbeta.double() - rb).abs() <= half_step(t, rb.abs() + eb) + eb).all()


BWD_SHAPES = [(1, 1), (1, 4096), (2, 7), (3, 32), (5, 33), (64, 1024), (7, 257), (1037, 1544), (9, 2047), (333, 4096),
              (149, 5003), (4, 8192), (301, 8192), (5, 16384), (160, 16384), (3, 16383), (2100, 256), (700, 264)]


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("T,D", BWD_SHAPES)
def test_backward(T, D, dtype):
    x, gamma, _, g = make(T, D, dtype, seed=T * 3 + D)
    dy = torch.randn(T, D, generator=g, device="cuda").to(dtype)
    _, mean, rstd = ops.layernorm_fwd(x, gamma)
    check_bwd(x, dy, gamma, mean, rstd, *ops.layernorm_bwd(x, dy, gamma, mean, rstd))
    assert ops.device_status() == ops.MXN_OK


@pytest.mark.parametrize("D", [1024, 1023])
def test_backward_selected_gradients(D):
    x, gamma, _, g = make(70, D, torch.bfloat16)
    dy = torch.randn(70, D, generator=g, device="cuda").bfloat16()
    _, mean, rstd = ops.layernorm_fwd(x, gamma)
    dx, dg, db = ops.layernorm_bwd(x, dy, gamma, mean, rstd)
    for kw in (dict(want_dgamma=False), dict(want_dbeta=False), dict(want_dgamma=False, want_dbeta=False)):
        dx1, dg1, db1 = ops.layernorm_bwd(x, dy, gamma, mean, rstd, **kw)
        assert torch.equal(dx, dx1)
        assert (dg1 is None) if not kw.get("want_dgamma", True) else torch.equal(dg, dg1)
        assert (db1 is None) if not kw.get("want_dbeta", True) else torch.equal(db, db1)
    dx2, dg2, db2 = ops.layernorm_bwd(x, dy, None, mean, rstd)
    check_bwd(x, dy, None, mean, rstd, dx2, dg2, db2)
    assert dg2 is None


@pytest.mark.parametrize("D", [48, 1031])
def test_backward_against_differences(D):
    """<dx, v> and <dgamma, w> against central differences of the float64 forward."""
    T, dtype = 11, torch.float32
    x, gamma, beta, g = make(T, D, dtype, seed=5)
    dy = torch.randn(T, D, generator=g, device="cuda")
    v, w = torch.randn(T, D, generator=g, device="cuda").double(), torch.randn(D, generator=g, device="cuda").double()
    _, mean, rstd = ops.layernorm_fwd(x, gamma, beta)
    dx, dg, db = ops.layernorm_bwd(x, dy, gamma, mean, rstd)

    def loss(x, gamma, beta):
        xh = (x - x.mean(1, keepdim=True)) * (x.var(1, unbiased=False, keepdim=True) + 1e-5).rsqrt()
        return ((xh * gamma + beta) * dy.double()).sum()
    a, b, c, h = x.double(), gamma.double(), beta.double(), 1e-5
    for got, hi, lo in ((dx.double() * v, loss(a + h * v, b, c), loss(a - h * v, b, c)),
                        (dg.double() * w, loss(a, b + h * w, c), loss(a, b - h * w, c)),
                        (db.double() * w, loss(a, b, c + h * w), loss(a, b, c - h * w))):
        want = (hi - lo) / (2 * h)
        # fp32 gradients: a few hundred roundings of the terms; the differences' own error is ~h^2 of the terms
        assert (got.sum() - want).abs() <= 2e-5 * got.abs().sum() + 1e-6


# ------------------------------------------------------------- use of the calls

def test_empty_batch():
    x = torch.empty(0, 256, device="cuda", dtype=torch.bfloat16)
    gamma = torch.ones(256, device="cuda", dtype=torch.bfloat16)
    y, mean, rstd = ops.layernorm_fwd(x, gamma)
    assert y.shape == (0, 256) and mean.shape == (0,)
    dx, dg, db = ops.layernorm_bwd(x, x, gamma, mean, rstd)
    assert dx.shape == (0, 256) and (dg == 0).all() and (db == 0).all()


@pytest.mark.parametrize("dtype,D", [(torch.bfloat16, 768), (torch.float32, 515)])
def test_memory_around_the_outputs_is_left_alone(dtype, D):
    T = 37
    x, gamma, beta, g = make(T, D, dtype)
    buf = torch.full(((T + 2) * D + 64,), 7.0, device="cuda", dtype=dtype)
    y = buf[:T * D]
    ops.layernorm_fwd(x, gamma, beta, y=y)
    assert (buf[T * D:] == 7).all()
    buf.fill_(7.0)
    _, mean, rstd = ops.layernorm_fwd(x, gamma, beta)
    dg, db = torch.full((D + 9,), 7.0, device="cuda", dtype=dtype), torch.full((D + 9,), 7.0, device="cuda", dtype=dtype)
    ops.layernorm_bwd(x, x.contiguous(), gamma, mean, rstd, dx=buf[:T * D], dgamma=dg[:D], dbeta=db[:D])
    assert (buf[T * D:] == 7).all() and (dg[D:] == 7).all() and (db[D:] == 7).all()


@pytest.mark.parametrize("D", [4096, 1027])
def test_repeats_bit_for_bit(D):
    x, gamma, beta, g = make(900, D, torch.bfloat16)
    dy = torch.randn(900, D, generator=g, device="cuda").bfloat16()
    first = None
    for _ in range(32):
        y, mean, rstd = ops.layernorm_fwd(x, gamma, beta)
        out = (y, mean, rstd, *ops.layernorm_bwd(x, dy, gamma, mean, rstd))
        if first is None:
            first = out
        assert all(torch.equal(a, b) for a, b in zip(out, first))


def test_other_stream_and_graph():
    """Two captured graphs that share a pool and an eager call on a stream of its own agree with plain calls."""
    x, gamma, beta, g = make(300, 1024, torch.bfloat16)
    dy = torch.randn(300, 1024, generator=g, device="cuda").bfloat16()

    def step(stream=None):
        y, mean, rstd = ops.layernorm_fwd(x, gamma, beta, stream=stream)
        return (y, *ops.layernorm_bwd(x, dy, gamma, mean, rstd, stream=stream))
    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = step(s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    outs = []
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
    x, gamma, beta, _ = make(8, 64, torch.bfloat16)
    _, mean, rstd = ops.layernorm_fwd(x)
    for bad in (lambda: ops.layernorm_fwd(x[0]), lambda: ops.layernorm_fwd(x.double()),
                lambda: ops.layernorm_fwd(x.t()), lambda: ops.layernorm_fwd(x, gamma.float()),
                lambda: ops.layernorm_fwd(x, gamma[:32]), lambda: ops.layernorm_fwd(x, gamma.cpu()),
                lambda: ops.layernorm_fwd(x, beta=beta[::2]), lambda: ops.layernorm_fwd(x, y=x[:4].clone()),
                lambda: ops.layernorm_bwd(x, x[:4], gamma, mean, rstd),
                lambda: ops.layernorm_bwd(x, x, gamma, mean[:3], rstd),
                lambda: ops.layernorm_bwd(x, x.half(), gamma, mean, rstd),
                lambda: ops.layernorm_bwd(x, x, gamma, mean, rstd.double()),
                lambda: ops.layernorm_bwd(x, x, gamma, mean, rstd, workspace=torch.empty(8, device="cuda"))):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(ops.MXNormError):
        ops.layernorm_fwd(x, eps=-1.0)
    with pytest.raises(ops.MXNormError):
        ops.layernorm_fwd(x, eps=float("nan"))
    with pytest.raises(ops.MXNormError):
        ops.layernorm_fwd(torch.empty(513, device="cuda", dtype=torch.bfloat16)[1:].view(8, 64))   # base off 16 bytes
    wide = torch.zeros(1, 16385, device="cuda")
    one = torch.zeros(1, device="cuda")
    with pytest.raises(ops.MXNormError):
        ops.layernorm_bwd(wide, wide, None, one, one)
    with pytest.raises(ops.MXNormError):
        ops.layernorm_fwd(torch.zeros(1, 32769, device="cuda"))


def test_offsets_past_32_bits():
    """Rows behind the 2^31st element, forward and backward, odd and aligned row lengths."""
    for T, D in ((66000, 32767), (140001, 16384)):
        x = torch.empty(T, D, device="cuda", dtype=torch.bfloat16).normal_()
        y, mean, rstd = ops.layernorm_fwd(x)
        at = 2 ** 31 // D - 1
        for r in (slice(0, 2), slice(at, at + 4), slice(T - 2, T)):
            check_fwd(x[r], None, None, 1e-5, y[r], mean[r], rstd[r])
        if D <= 16384:
            dx, _, _ = ops.layernorm_bwd(x, y, None, mean, rstd, want_dbeta=False)
            for r in (slice(at, at + 4), slice(T - 2, T)):
                check_bwd(x[r], y[r], None, mean[r], rstd[r], dx[r], None, None)
        del x, y


def test_two_calls_at_once():
    """Calls on two streams, each with its own outputs and workspace, do not disturb one another."""
    sets = []
    for seed in (1, 2):
        x, gamma, beta, g = make(2000, 1024, torch.bfloat16, seed=seed)
        dy = torch.randn(2000, 1024, generator=g, device="cuda").bfloat16()
        sets.append((x, gamma, beta, dy))

    def step(x, gamma, beta, dy, stream=None):
        y, mean, rstd = ops.layernorm_fwd(x, gamma, beta, stream=stream)
        return (y, *ops.layernorm_bwd(x, dy, gamma, mean, rstd, stream=stream))
    want = [step(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(8):
        got = [step(*s, stream=st) for s, st in zip(sets, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


# Row lengths that take every number of chunks a lane and of warps a row, whole and ragged, few rows and many.
@pytest.mark.parametrize("T", [3, 700])
@pytest.mark.parametrize("D", [264, 520, 1288, 2304, 2560, 2824, 3584, 3592, 4104, 5120, 6144, 6752, 7168, 10240, 12000, 12288,
                               14336, 20480, 24584, 32760])
@pytest.mark.parametrize("dtype", TYPES)
def test_forward_plans(T, D, dtype):
    x, gamma, beta, _ = make(T, D, dtype, seed=T + D)
    y, mean, rstd = ops.layernorm_fwd(x, gamma, beta)
    check_fwd(x, gamma, beta, 1e-5, y, mean, rstd)


@pytest.mark.parametrize("T,D,pad", [(1, 20481, 0), (200, 30001, 0), (3, 19999, 1), (5, 32764, 1), (300, 32767, 3)])
@pytest.mark.parametrize("dtype", TYPES)
def test_forward_long_rows_off_boundaries(T, D, pad, dtype):
    x, gamma, beta, _ = make(T, D, dtype, seed=T + D, pad=pad)
    check_fwd(x, gamma, beta, 1e-5, *ops.layernorm_fwd(x, gamma, beta))
    y, mean, rstd = ops.layernorm_fwd(x, None, None)
    check_fwd(x, None, None, 1e-5, y, mean, rstd)
