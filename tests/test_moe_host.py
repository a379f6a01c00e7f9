"""Host-side checks of the expert layer: refusals, and the plain statement the
GPU tests compare with against direct arithmetic."""
import ctypes

import numpy as np
import pytest

import w4a4_mxfp4_outlier_b200 as w4
from w4a4_mxfp4_outlier_b200 import fp8, moe
from tests import fp8_ref as ref

F = 0x1000
INV, SHAPE = w4.ERR_INVALID_ARG, w4.ERR_UNSUPPORTED_SHAPE


def _m(top_k=2, act=moe.SILU_GATED, router=F, E=4, d=128, ff=256, **over):
    ws = {"gate": fp8.Fp8WeightC(d, ff, E, F, F), "up": fp8.Fp8WeightC(d, ff, E, F, F),
          "down": fp8.Fp8WeightC(ff, d, E, F, F)}
    ws.update(over)
    return ctypes.byref(moe.ExpertsC(top_k, act, 1, router, ws["gate"], ws["up"], ws["down"]))


def _call(m, X=F, T=8, ldx=128, ws=F, nb=1 << 40, Y=F, ldy=128, ids=None, wts=None):
    return moe._moe(X, T, ldx, m, ws, nb, Y, ldy, 0, ids, wts, None)


W = fp8.Fp8WeightC


@pytest.mark.parametrize("m,status", [
    (None, INV), (_m(top_k=0), INV), (_m(top_k=5), INV), (_m(act=2), INV), (_m(router=None), INV),
    (_m(router=F + 8), SHAPE), (_m(E=513), SHAPE), (_m(top_k=17, E=32), SHAPE),
    (_m(d=136), SHAPE), (_m(ff=264), SHAPE), (_m(d=65536), SHAPE), (_m(ff=65552), SHAPE),
    (_m(gate=W(0, 0, 0, None, None)), INV), (_m(gate=W(128, 128, 4, F, F)), INV),
    (_m(gate=W(128, 256, 3, F, F)), INV), (_m(down=W(256, 256, 4, F, F)), INV),
    (_m(down=W(256, 128, 5, F, F)), INV), (_m(up=W(128, 256, 4, None, F)), INV),
    (_m(up=W(128, 256, 4, F + 8, F)), SHAPE),
])
def test_layer_refusals(m, status):
    assert _call(m) == status
    n = ctypes.c_size_t()
    assert moe._moe_workspace_size(m, 8, ctypes.byref(n)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), INV), (dict(T=65), SHAPE), (dict(ldx=127), INV), (dict(ldy=120), INV),
    (dict(ldx=132), SHAPE), (dict(ldy=132), SHAPE), (dict(X=None), INV), (dict(Y=None), INV),
    (dict(ws=None), INV), (dict(nb=100), INV), (dict(X=F + 8), SHAPE), (dict(Y=F + 8), SHAPE),
    (dict(ws=F + 4), SHAPE), (dict(ids=F + 2), SHAPE), (dict(wts=F + 1), SHAPE),
    (dict(T=0, X=None, Y=None, ws=None, nb=0), w4.OK),
])
def test_call_refusals(kw, status):
    assert _call(_m(), **kw) == status


def test_workspace_size():
    n, k = ctypes.c_size_t(), ctypes.c_size_t()
    assert moe._moe_workspace_size(_m(), 8, ctypes.byref(n)) == w4.OK and n.value > 0
    assert moe._moe_workspace_size(_m(), 8, None) == INV
    assert moe._moe_workspace_size(_m(), -1, ctypes.byref(k)) == INV
    # one byte short is refused
    assert _call(_m(), nb=n.value - 1) == INV
    # without a gate the gate's record is not looked at
    assert moe._moe_workspace_size(_m(act=moe.GELU, gate=W(0, 0, 0, None, None)), 8, ctypes.byref(k)) == w4.OK
    assert k.value < n.value


def test_reference_is_the_formula():
    # the interval reference's value is the plain formula evaluated element by element
    rng = np.random.default_rng(1)
    T, E, k, d, ff = 3, 5, 2, 144, 272
    x, r = rng.standard_normal((T, d)), rng.standard_normal((E, d)) / 12
    packs = [[ref.pack_weight(rng.standard_normal(s) / 12) for _ in range(E)] for s in ((ff, d), (ff, d), (d, ff))]
    gate, up, down = ((np.stack([p[0] for p in ps]), np.stack([p[1] for p in ps])) for ps in packs)
    _, _, ids, w = ref.route(x, r, k, True)
    y, tol, w2, _ = ref.moe(x, r, gate, up, down, ids, k, True, True, False)
    np.testing.assert_allclose(w2, w, rtol=1e-14)
    xv = ref.act_values(*ref.quant_act(x))
    for t in range(T):
        want = 0
        for j in range(k):
            e = ids[t, j]
            g = ref.weight_values(gate[0][e], gate[1][e]) @ xv[t]
            u = ref.weight_values(up[0][e], up[1][e]) @ xv[t]
            h = (g / (1 + np.exp(-g)) * u)[None]
            want = want + w[t, j] * (ref.weight_values(down[0][e], down[1][e]) @ ref.act_values(*ref.quant_act(h))[0])
        assert (np.abs(y[t] - want) <= 1e-12 * np.abs(want).max() + tol[t]).all()
        assert np.abs(y[t] - want).max() < 1e-3 * np.abs(want).max()
