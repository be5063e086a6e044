"""The C entry points called from host threads of a program's own (ctypes releases the interpreter's lock), and two sizes of
a kernel in one graph."""
import ctypes
import threading

import pytest
import torch

from normalisation_row_bf16_b200 import build as nbuild
from normalisation_row_bf16_b200 import ops

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(autouse=True, scope="module")
def _built():
    nbuild.build()


def P(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def rand(*shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(BF)


def ln_fwd(T, D):
    x, y = rand(T, D, seed=D), torch.empty(T, D, device="cuda", dtype=BF)
    return (lambda L, s: L.layernorm_fwd(P(x), None, None, P(y), None, None, T, D, D, 1e-5, 0, s)), y, (x,)


def ln_bwd(T, D):
    x, dy = rand(T, D, seed=D), rand(T, D, seed=D + 1)
    _, mean, rstd = ops.layernorm_fwd(x)
    dx = torch.empty(T, D, device="cuda", dtype=BF)
    return (lambda L, s: L.layernorm_bwd(P(x), P(dy), None, P(mean), P(rstd), P(dx), None, None, T, D, D, D, 0, None, 0, s),
            dx, (x, dy, mean, rstd))


def ffn_fwd(T, D, F):
    x, wg, wu = rand(T, D, seed=T), rand(F, D, seed=1, scale=0.02), rand(F, D, seed=2, scale=0.02)
    h = torch.empty(T, F, device="cuda", dtype=BF)
    return (lambda L, s: L.gated_ffn_fwd(P(x), P(wg), P(wu), P(h), None, None, T, D, F, D, D, 0, s)), h, (x, wg, wu)


def mx_ffn(T, F, K):
    ops_ = [ops.mxfp8_cast(rand(n, K, seed=n, scale=0.1), scale_layout=ops.SCALES_MMA) for n in (T, F, F + 8)]
    (aq, as_), (gq, gs), (uq, us) = ops_
    h = torch.empty(T, F, device="cuda", dtype=BF)
    return (lambda L, s: L.mxfp8_gated_ffn(P(aq), P(as_), P(gq), P(gs), P(uq), P(us), P(h), None, T, F, K, 0, 0, 0, s),
            h, (ops_,))


def gemm(M, N, K):
    (aq, as_), (bq, bs) = ops_ = [ops.mxfp8_cast(rand(n, K, seed=n, scale=0.1), scale_layout=ops.SCALES_MMA) for n in (M, N)]
    c = torch.empty(M, N, device="cuda", dtype=BF)
    return (lambda L, s: L.mxfp8_gemm(P(aq), P(as_), P(bq), P(bs), P(c), M, N, K, s)), c, (ops_,)


FIRST = {
    "layernorm_fwd": lambda: ln_fwd(40, 1001),
    "layernorm_bwd": lambda: ln_bwd(40, 1001),
    "gated_ffn_fwd": lambda: ffn_fwd(1, 64, 64),
    "mxfp8_gated_ffn": lambda: mx_ffn(1, 256, 256),
    "mxfp8_gemm": lambda: gemm(256, 512, 256),
}


@pytest.mark.parametrize("name", list(FIRST))
def test_first_cuda_call_of_a_thread(name):
    """A thread that has not touched the device calls the library first."""
    L = ops.lib()
    call, out, _ = FIRST[name]()
    assert call(L, None) == ops.MXN_OK
    torch.cuda.synchronize()
    want = out.clone()
    out.zero_()
    torch.cuda.synchronize()
    got = []

    def work():
        got.append((call(L, None), L.mxnorm_last_error().decode()))
    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert got[0][0] == ops.MXN_OK, got
    assert torch.equal(out, want)


# Two sizes of one kernel that ask for different amounts of shared memory.
PAIRS = {
    "layernorm_fwd": lambda: (ln_fwd(40, 1001), ln_fwd(40, 5003)),
    "layernorm_bwd": lambda: (ln_bwd(40, 1001), ln_bwd(40, 5003)),
    "gated_ffn_fwd": lambda: (ffn_fwd(1, 64, 64), ffn_fwd(100, 1024, 2048)),
    "mxfp8_gated_ffn": lambda: (mx_ffn(1, 256, 256), mx_ffn(120, 256, 256)),
}


@pytest.mark.parametrize("name", list(PAIRS))
def test_two_host_threads(name):
    """Two threads call two sizes of one kernel: each call succeeds and leaves its own result."""
    L = ops.lib()
    calls = PAIRS[name]()
    want = []
    for call, out, _ in calls:
        assert call(L, None) == ops.MXN_OK
        torch.cuda.synchronize()
        want.append(out.clone())
        out.zero_()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    codes = [set(), set()]
    start = threading.Barrier(2)

    def work(i):
        s = ctypes.c_void_p(streams[i].cuda_stream)
        start.wait()
        for _ in range(20000):
            codes[i].add(calls[i][0](L, s))
    threads = [threading.Thread(target=work, args=(i,)) for i in (0, 1)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [{ops.MXN_OK}, {ops.MXN_OK}], codes
    for (_, out, _), w in zip(calls, want):
        assert torch.equal(out, w)


def test_one_graph_of_two_sizes():
    """A graph holds both sizes of each kernel, the larger first."""
    L = ops.lib()
    pairs = [PAIRS[n]() for n in PAIRS]
    want = []
    for pair in pairs:
        for call, out, _ in pair:
            assert call(L, None) == ops.MXN_OK
            torch.cuda.synchronize()
            want.append(out.clone())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
        for small, large in pairs:
            assert large[0](L, s) == ops.MXN_OK and small[0](L, s) == ops.MXN_OK
    outs = [out for pair in pairs for _, out, _ in pair]
    for _ in range(2):
        for o in outs:
            o.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, want))


