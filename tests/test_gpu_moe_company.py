"""The expert layer: what the tokens beside it may change of a token.  Only the
order in which float32 sums are made: every token's y stays within the bound
of the plain statement in 64 bits, element by element, whatever the others hold."""
import numpy as np
import pytest
import torch

import w4a4_mxfp4_outlier_b200 as w4
from w4a4_mxfp4_outlier_b200 import moe
from tests import fp8_ref as ref
from tests.test_gpu_moe import _acts, _f64, _layer, _np, _ws

pytestmark = pytest.mark.gpu


def _run(X, m):
    T, k = X.shape[0], m.top_k
    Y = torch.empty_like(X, memory_format=torch.contiguous_format)
    ids, wts = torch.empty(T, k, dtype=torch.int32, device="cuda"), torch.empty(T, k, device="cuda")
    moe.forward(X, m, _ws(T, m), Y, ids, wts)
    assert w4.last_error()[0] == w4.OK
    return Y, ids.cpu().numpy(), wts


def _within(X, m, Y, ids, rows):
    y, tol, _, _ = ref.moe(_f64(X)[rows], _f64(m.router), _np(m.gate) if m.gate else None, _np(m.up), _np(m.down),
                           ids[rows], m.top_k, m.renorm, m.gate is not None, True)
    err = np.abs(_f64(Y)[rows] - y)
    assert (err <= tol).all(), f"{(err > tol).sum()} of {err.size}, worst {(err / tol).max():.3f}"


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("T,at,gated", [(2, 0, True), (3, 1, True), (17, 16, False), (40, 1, True), (64, 33, False)])
def test_tokens_beside_one_that_is_not_finite(bad, T, at, gated):
    rng = np.random.default_rng([1, T])
    m = _layer(rng, 12, 3, 272, 400, gated, True)
    X = _acts(rng, T, 272)
    _, ids, _ = _run(X, m)
    X[at, 100] = bad
    Z, ids_z, _ = _run(X, m)
    keep = [t for t in range(T) if t != at]
    assert torch.isnan(Z[at]).all()
    np.testing.assert_array_equal(ids_z[keep], ids[keep])
    _within(X, m, Z, ids_z, keep)


@pytest.mark.parametrize("T", [1, 5, 30, 64])
def test_a_token_in_batches_of_every_size(T):
    # few experts chosen: K of the up units is split; many: it is not
    rng = np.random.default_rng([2, T])
    m = _layer(rng, 48, 4, 1296, 656, True, False)
    X = _acts(rng, 64, 1296)
    Y, ids, wts = _run(X[:T], m)
    _, ids_all, wts_all = _run(X, m)
    np.testing.assert_array_equal(ids, ids_all[:T])
    assert torch.equal(wts, wts_all[:T])
    _within(X[:T], m, Y, ids, list(range(T)))
