"""The expert layer's selection on the GPU where float32 sums would decide it
wrongly: the chosen experts, and their order, are those of the logits in 64
bits.  All inputs are bf16, so products are exact in float64, and in these
cases their sums are too."""
import numpy as np
import pytest
import torch

import w4a4_mxfp4_outlier_b200 as w4
from w4a4_mxfp4_outlier_b200 import fp8, moe

pytestmark = pytest.mark.gpu


def _select(x, r, k, renorm=True):
    """ids and weights the layer gives for activations x and router r (values exact in bf16)."""
    T, d, E = x.shape[0], x.shape[1], r.shape[0]
    cu = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(torch.bfloat16)
    X, R = cu(x), cu(r)
    assert np.array_equal(X.double().cpu().numpy(), x, equal_nan=True)
    assert np.array_equal(R.double().cpu().numpy(), r, equal_nan=True)
    w = fp8.Fp8Weight(torch.zeros(E, 16, d, dtype=torch.uint8, device="cuda"),
                      torch.ones(E, 1, fp8.blocks(d), device="cuda"))
    dn = fp8.Fp8Weight(torch.zeros(E, d, 16, dtype=torch.uint8, device="cuda"),
                       torch.ones(E, fp8.blocks(d), 1, device="cuda"))
    m = moe.MoE(R, None, w, dn, top_k=k, act=moe.GELU, renorm=renorm)
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    wts = torch.empty(T, k, device="cuda")
    moe.forward(X, m, torch.empty(moe.workspace_size(T, m), dtype=torch.uint8, device="cuda"),
                torch.empty(T, d, dtype=torch.bfloat16, device="cuda"), ids, wts)
    assert w4.last_error()[0] == w4.OK
    return ids.cpu().numpy(), wts.double().cpu().numpy()


def _want(x, r, k):
    return np.argsort(-(x @ r.T), axis=1, kind="stable")[:, :k]


def _bf16(a):
    return torch.from_numpy(np.asarray(a, np.float32)).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("E,d", [(2, 16), (9, 272), (40, 1040), (64, 2048), (130, 512), (512, 256)])
@pytest.mark.parametrize("eps", [2.0 ** -25, 2.0 ** -30])
def test_logits_one_small_term_apart(E, d, eps):
    # every logit is 1 + e * eps: equal in float32 (up to E * eps), in 64 bits in
    # descending order of the index.  e = 0 .. E-1 as two bf16 numbers, e // 32 and e % 32
    x, r = np.zeros((3, d)), np.zeros((E, d))
    x[:, 0] = 1.0
    r[:, 0] = 1.0
    e = np.arange(E)
    x[:, d - 3], x[:, d - 1] = 32 * eps, eps
    r[:, d - 3], r[:, d - 1] = e // 32, e % 32
    k = min(E, 16)
    ids, wts = _select(x, r, k)
    np.testing.assert_array_equal(ids, np.broadcast_to(E - 1 - np.arange(k), (3, k)))
    assert np.abs(wts - 1 / k).max() <= 2.0 ** -20


@pytest.mark.parametrize("T", [1, 64])
def test_cancelling_terms(T):
    # large terms that cancel leave the small ones to decide; with float32 sums
    # the small ones are lost beside the large
    rng = np.random.default_rng([1, T])
    E, d, k = 48, 1296, 8
    x = _bf16(rng.standard_normal((T, d)))
    r = _bf16(rng.standard_normal((E, d)) * 2.0 ** -12)
    x[:, 10], x[:, d - 7] = 1024.0, 1024.0
    big = _bf16(rng.integers(1, 128, E) * 8.0)
    r[:, 10], r[:, d - 7] = big, -big
    ids, _ = _select(x, r, k)
    np.testing.assert_array_equal(ids, _want(x, r, k))


def test_logits_past_the_float32_range():
    # 2^120 * 2^20 * e, finite in 64 bits: in order, and the first has all the weight
    E, d, k = 20, 272, 4
    x, r = np.zeros((2, d)), np.zeros((E, d))
    x[:, 100], r[:, 100] = 2.0 ** 120, 2.0 ** 20 * (np.arange(E) + 1.0)
    x[1] *= -1
    for renorm in (True, False):
        ids, wts = _select(x, r, k, renorm)
        np.testing.assert_array_equal(ids, _want(x, r, k))
        np.testing.assert_array_equal(wts, np.broadcast_to([1.0, 0, 0, 0], (2, k)))


def test_subnormal_numbers_count():
    # the smallest bf16 numbers on both sides: products of 2^-266
    E, d, k = 6, 144, 3
    x, r = np.zeros((1, d)), np.zeros((E, d))
    x[0, 77] = 2.0 ** -133
    r[:, 77] = 2.0 ** -133 * np.array([3.0, 5, 1, 6, 2, 4])
    ids, _ = _select(x, r, k)
    assert ids.tolist() == [[3, 1, 5]]


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
@pytest.mark.parametrize("E", [5, 100])
def test_router_rows_that_are_not_finite(bad, E):
    # a logit of NaN comes last; -inf last too (no weight), inf first
    rng = np.random.default_rng(2)
    d, k = 528, 4
    x, r = _bf16(rng.standard_normal((3, d))), _bf16(rng.standard_normal((E, d)) / 16)
    r[2, 300] = bad
    x[:, 300] = 1.5
    ids, wts = _select(x, r, k)
    with np.errstate(invalid="ignore"):
        logits = x @ r.T
    logits[np.isnan(logits)] = -np.inf
    if np.isinf(bad) and bad > 0:
        assert (ids[:, 0] == 2).all()
        np.testing.assert_array_equal(ids[:, 1:], np.argsort(-np.delete(logits, 2, 1), 1, kind="stable")[:, :k - 1] +
                                      (np.argsort(-np.delete(logits, 2, 1), 1, kind="stable")[:, :k - 1] >= 2))
        return
    want = np.argsort(-logits, axis=1, kind="stable")[:, :k]
    np.testing.assert_array_equal(ids, want)
    assert (ids != 2).all() and np.isfinite(wts).all() and np.abs(wts.sum(1) - 1).max() < 2.0 ** -20


@pytest.mark.parametrize("T,E,k,d", [(64, 64, 8, 1024), (64, 512, 16, 256), (64, 128, 8, 2048), (37, 20, 3, 1040)])
def test_random_batches_select_as_in_64_bits(T, E, k, d):
    rng = np.random.default_rng([3, T, E, d])
    for _ in range(4):
        x, r = _bf16(rng.standard_normal((T, d))), _bf16(rng.standard_normal((E, d)) * 2 / np.sqrt(d))
        # pairs of experts that differ in the last bit of one small number
        r[1::2] = r[::2]
        at = np.abs(r[1::2]).argmin(1)
        r[np.arange(1, E, 2), at] *= 1 + 2.0 ** -7
        r = _bf16(r)
        ids, _ = _select(x, r, k)
        np.testing.assert_array_equal(ids, _want(x, r, k))
