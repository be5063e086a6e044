"""Argument checks of the layer-norm and feed-forward entry points.

No test here launches a kernel: invalid calls return during validation, and
the fault-injection hook fails a call on the host before any CUDA call.
"""
import ctypes

import pytest

from normalisation_row_bf16_b200 import build as nbuild
from normalisation_row_bf16_b200 import ops

P = ctypes.c_void_p(0x10000)             # aligned, never dereferenced on these paths
BAD = ctypes.c_void_p(0x10008)
ARG, UNSUP, CUDA, OK = ops.MXN_ERR_ARG, ops.MXN_ERR_UNSUPPORTED, ops.MXN_ERR_CUDA, ops.MXN_OK


@pytest.fixture(scope="module")
def L():
    nbuild.build()
    return ops.lib()


def ln_fwd(L, x=P, gamma=P, beta=P, y=P, mean=P, rstd=P, T=4, D=64, ld=64, eps=1e-5, dtype=0):
    return L.layernorm_fwd(x, gamma, beta, y, mean, rstd, T, D, ld, eps, dtype, None)


def ln_bwd(L, x=P, dy=P, gamma=P, mean=P, rstd=P, dx=P, dgamma=None, dbeta=None, T=4, D=64, ld_x=64, ld_dy=64, dtype=0,
           ws=P, n=1 << 30):
    return L.layernorm_bwd(x, dy, gamma, mean, rstd, dx, dgamma, dbeta, T, D, ld_x, ld_dy, dtype, ws, n, None)


def ffn_fwd(L, x=P, wg=P, wu=P, h=P, gate=None, up=None, T=4, D=64, F=64, ld_x=64, ld_w=64, act=0):
    return L.gated_ffn_fwd(x, wg, wu, h, gate, up, T, D, F, ld_x, ld_w, act, None)


def ffn_bwd(L, dh=P, x=P, wg=P, wu=P, gate=P, up=P, dx=P, dwg=P, dwu=P, T=4, D=64, F=64, ld_x=64, ld_w=64, act=0, ws=P,
            n=1 << 30):
    return L.gated_ffn_bwd(dh, x, wg, wu, gate, up, dx, dwg, dwu, T, D, F, ld_x, ld_w, act, ws, n, None)


def mx_ffn(L, aq=P, as_=P, gq=P, gs=P, uq=P, us=P, h=P, hs=None, T=4, F=64, K=128, act=0, out=0, layout=0):
    return L.mxfp8_gated_ffn(aq, as_, gq, gs, uq, us, h, hs, T, F, K, act, out, layout, None)


@pytest.mark.parametrize("call,kw,code", [
    (ln_fwd, dict(x=None), ARG), (ln_fwd, dict(y=None), ARG), (ln_fwd, dict(x=BAD), ARG), (ln_fwd, dict(gamma=BAD), ARG),
    (ln_fwd, dict(rstd=BAD), ARG), (ln_fwd, dict(T=-1), ARG), (ln_fwd, dict(D=0), ARG), (ln_fwd, dict(ld=63), ARG),
    (ln_fwd, dict(eps=-1e-5), ARG), (ln_fwd, dict(eps=float("nan")), ARG), (ln_fwd, dict(eps=float("inf")), ARG),
    (ln_fwd, dict(dtype=3), ARG), (ln_fwd, dict(dtype=-1), ARG), (ln_fwd, dict(D=32769, ld=32769), UNSUP),
    (ln_bwd, dict(x=None), ARG), (ln_bwd, dict(dy=None), ARG), (ln_bwd, dict(mean=None), ARG), (ln_bwd, dict(dx=None), ARG),
    (ln_bwd, dict(ld_x=60), ARG), (ln_bwd, dict(ld_dy=60), ARG), (ln_bwd, dict(dtype=7), ARG),
    (ln_bwd, dict(gamma=None, dgamma=P), ARG), (ln_bwd, dict(dbeta=BAD), ARG),
    (ln_bwd, dict(D=16385, ld_x=16385, ld_dy=16385), UNSUP),
    (ffn_fwd, dict(x=None), ARG), (ffn_fwd, dict(h=None), ARG), (ffn_fwd, dict(wu=BAD), ARG), (ffn_fwd, dict(gate=P), ARG),
    (ffn_fwd, dict(up=P), ARG), (ffn_fwd, dict(T=-1), ARG), (ffn_fwd, dict(D=60), ARG), (ffn_fwd, dict(D=0), ARG),
    (ffn_fwd, dict(F=36), ARG), (ffn_fwd, dict(F=-8), ARG), (ffn_fwd, dict(ld_x=68), ARG), (ffn_fwd, dict(ld_w=56), ARG),
    (ffn_fwd, dict(act=3), ARG), (ffn_fwd, dict(T=1 << 31), UNSUP), (ffn_fwd, dict(F=1 << 33), UNSUP),
    (ffn_bwd, dict(dh=None), ARG), (ffn_bwd, dict(gate=None), ARG), (ffn_bwd, dict(dwg=None), ARG),
    (ffn_bwd, dict(dwu=None), ARG), (ffn_bwd, dict(dx=BAD), ARG), (ffn_bwd, dict(act=-1), ARG),
    (ffn_bwd, dict(ws=None), ARG), (ffn_bwd, dict(ws=BAD), ARG), (ffn_bwd, dict(n=4 * 4 * 64 - 1), ARG),
    (mx_ffn, dict(aq=None), ARG), (mx_ffn, dict(us=None), ARG), (mx_ffn, dict(gs=BAD), ARG), (mx_ffn, dict(h=None), ARG),
    (mx_ffn, dict(K=96), UNSUP), (mx_ffn, dict(K=0), ARG), (mx_ffn, dict(F=60), ARG), (mx_ffn, dict(F=40, out=1, hs=P), ARG),
    (mx_ffn, dict(out=1), ARG), (mx_ffn, dict(hs=P), ARG), (mx_ffn, dict(out=2), ARG), (mx_ffn, dict(layout=2), ARG),
    (mx_ffn, dict(act=9), ARG), (mx_ffn, dict(T=-4), ARG), (mx_ffn, dict(T=1 << 32), UNSUP),
])
def test_argument_errors(L, call, kw, code):
    assert call(L, **kw) == code
    assert L.mxnorm_last_error().decode() != ""


def test_empty_input_is_a_noop(L):
    assert ln_fwd(L, T=0) == OK and ln_fwd(L, T=0, x=None, y=None) == OK
    assert ln_bwd(L, T=0) == OK                       # no gradients to zero
    assert ffn_fwd(L, T=0, x=None, h=None) == OK
    assert ffn_bwd(L, T=0, dwg=None, dwu=None) == OK
    assert mx_ffn(L, T=0) == OK


def test_nothing_wanted_is_a_noop(L):
    assert ffn_bwd(L, dx=None, dwg=None, dwu=None) == OK


def test_host_fault_injection(L):
    for call in (ln_fwd, ln_bwd, ffn_fwd, ffn_bwd, mx_ffn):
        L.mxnorm_debug_fail_next(1)
        assert call(L) == CUDA and "injected" in L.mxnorm_last_error().decode()
    L.mxnorm_debug_fail_next(0)


def test_workspace_sizes(L):
    assert L.gated_ffn_bwd_workspace_size(0, 64, 64) == 0 and L.gated_ffn_bwd_workspace_size(4, 64, 60) == 0
    assert L.gated_ffn_bwd_workspace_size(4, 60, 64) == 0
    assert L.layernorm_bwd_workspace_size(4, 16385, 0) == 0 and L.layernorm_bwd_workspace_size(4, 64, 3) == 0
    assert L.layernorm_bwd_workspace_size(0, 64, 0) == 0


def test_python_bindings_refuse_cpu_tensors(L):
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    s = torch.zeros(4)
    for bad in (lambda: ops.layernorm_fwd(x), lambda: ops.layernorm_bwd(x, x, None, s, s),
                lambda: ops.gated_ffn_fwd(x, x, x), lambda: ops.gated_ffn_bwd(x, x, x, x, x, x),
                lambda: ops.mxfp8_gated_ffn(x, x, x, x, x, x, 4, 64, 128)):
        with pytest.raises(ValueError):
            bad()
