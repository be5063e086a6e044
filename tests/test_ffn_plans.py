"""How the feed-forward products are dealt to a device: the shapes that the GPU tests take reach every form of the plan
(on 148 SMs that run 74 CTA pairs at once, a B200), and partial products stay inside the workspace.  Host arithmetic."""
import ctypes
import random

import pytest

from normalisation_row_bf16_b200 import build as nbuild
from normalisation_row_bf16_b200 import ops

FWD, DX, DW, MXFP8 = range(4)
PLENTY = 1 << 62

# T, D, F that take pairs of CTAs, by what their work units are: whole 512-row tiles of one or several rounds, the halves
# that whole tiles past the last full round are dealt as, the odd 256-row half
PAIR_SHAPES = {
    FWD: [(1411, 880, 5952), (673, 1672, 8992), (7129, 1672, 872), (5658, 1712, 1104), (1205, 1536, 9368), (8004, 1488, 1384),
          (6761, 1488, 1616)],
    DX: [(7557, 792, 128), (7952, 2832, 200), (6905, 2728, 328), (1808, 5624, 400), (7201, 1352, 400), (7848, 2440, 328),
         (3337, 408, 4760), (1030, 4184, 7216), (6446, 416, 8600), (6367, 400, 8248), (6850, 656, 7624)],
    DW: [(134, 4856, 144), (134, 3152, 264), (134, 136, 6400), (128, 576, 6280), (129, 1064, 9544), (132, 832, 9632),
         (133, 808, 9736)],
}
# and that take single CTAs, whole and split
SINGLE_SHAPES = {
    FWD: [(1, 4096, 4096), (64, 1024, 2816), (700, 512, 1032), (2300, 1024, 4104)],
    DX: [(1, 64, 64), (129, 520, 1000), (333, 1032, 2744), (128, 2048, 768), (64, 64, 64)],
    DW: [(63, 128, 128), (333, 1032, 2744), (4096, 512, 1408), (8192, 64, 64), (2834, 600, 600)],
}


@pytest.fixture(scope="module")
def L():
    nbuild.build()
    return ops.lib()


def plan(L, product, T, D, F, sms=148, pairs=74, ws=PLENTY):
    """(pair, tile columns, parts, units, whole, dealt, odd, CTAs)"""
    out = (ctypes.c_int * 8)()
    assert L.mxnorm_debug_ffn_plan(product, T, D, F, sms, pairs, ws, out) == ops.MXN_OK, L.mxnorm_last_error()
    return tuple(out)


def form(p, pairs=74):
    """What of the kernel a plan reaches."""
    pair, _, parts, units, whole, dealt, odd, _ = p
    if not pair:
        return ("single", parts > 1)
    return ("pair", parts > 1, min(whole // pairs, 2), dealt > 0, odd > 0)


def test_shapes_reach_every_form(L):
    got = {p: {form(plan(L, p, *s)) for s in PAIR_SHAPES[p]} for p in PAIR_SHAPES}
    for product, forms in got.items():
        assert all(f[0] == "pair" for f in forms), forms
        assert {(f[3], f[4]) for f in forms} == {(a, b) for a in (False, True) for b in (False, True)}, forms
        assert {f[2] > 1 for f in forms} == {False, True} and {f[1] for f in forms} == ({False, True} if product == DX else {False})
    parts = {f[1:] for f in got[DX] if f[1]}
    assert {(f[2], f[3]) for f in parts} == {(a, b) for a in (False, True) for b in (False, True)}, parts
    assert {(f[3], f[4]) for f in got[DW] if f[2] == 0} >= {(True, False), (False, True), (True, True)}    # no full round at all
    for p, shapes in SINGLE_SHAPES.items():
        forms = {form(plan(L, p, *s)) for s in shapes}
        assert forms == ({("single", False)} if p == FWD else {("single", False), ("single", True)}), (p, forms)


def random_shape(rng):
    return (int(2 ** rng.uniform(0, 13.5)), 8 * int(2 ** rng.uniform(0, 9.5)), 8 * int(2 ** rng.uniform(0, 10.9)))


def test_weight_gradients_on_pairs_are_never_split(L):
    """Nor is the forward: only dx's kernel on pairs writes partial products."""
    rng = random.Random(5)
    for _ in range(20000):
        s, pairs = random_shape(rng), rng.choice([0, 1, 60, 74])
        for product in (FWD, DW):
            p = plan(L, product, *s, pairs=pairs)
            assert p[2] == 1 or (product == DW and not p[0])


def test_parts_fit_the_workspace(L):
    rng = random.Random(6)
    split = 0
    for _ in range(20000):
        T, D, F = random_shape(rng)
        grads = (4 * T * F + 255) // 256 * 256
        ws = rng.choice([4 * T * F, grads, grads + rng.randrange(1, 64 * T * D + 1), grads + rng.randrange(1, 64 * F * D + 1)])
        for product, rows, problems in ((DX, T, 1), (DW, F, 2)):
            parts = plan(L, product, T, D, F, ws=ws)[2]
            assert parts == 1 or grads + parts * problems * rows * D * 4 <= ws
            split += parts > 1
            # with room for them, the parts are those of the size the call asks for
            most = plan(L, product, T, D, F)[2]
            assert plan(L, product, T, D, F, ws=grads + most * problems * rows * D * 4)[2] == most
    assert split > 500


def test_units_cover_the_product(L):
    """Pairs: whole tiles, dealt-out halves and odd halves are all of the 256-row halves, none twice."""
    rng = random.Random(7)
    for _ in range(20000):
        T, D, F = random_shape(rng)
        pairs = rng.choice([1, 3, 60, 74])
        for product, rows, cols, problems, width in ((FWD, T, F, 1, 128), (DX, T, D, 1, 256), (DW, F, D, 2, 256)):
            pair, tile_n, parts, units, whole, dealt, odd, grid = plan(L, product, T, D, F, pairs=pairs)
            n = -(-cols // tile_n) * problems * parts
            if pair:
                assert tile_n == width and units == whole + dealt + odd and dealt % 2 == 0
                assert 2 * whole + dealt + odd == -(-rows // 256) * n
                assert grid == 2 * min(units, pairs)
            else:
                assert units == -(-rows // 128) * n and grid == min(units, 148)


@pytest.mark.parametrize("kw", [dict(product=4), dict(product=-1), dict(T=0), dict(T=-1), dict(D=0), dict(F=-8), dict(sms=-1),
                                dict(pairs=-1), dict(T=1 << 31), dict(F=12)])
def test_refusals(L, kw):
    a = dict(dict(product=DX, T=8, D=64, F=64, sms=148, pairs=74), **kw)
    out = (ctypes.c_int * 8)()
    rc = L.mxnorm_debug_ffn_plan(a["product"], a["T"], a["D"], a["F"], a["sms"], a["pairs"], PLENTY, out)
    assert rc in (ops.MXN_ERR_ARG, ops.MXN_ERR_UNSUPPORTED)
    assert L.mxnorm_debug_ffn_plan(DX, 8, 64, 64, 148, 74, PLENTY, None) == ops.MXN_ERR_ARG
