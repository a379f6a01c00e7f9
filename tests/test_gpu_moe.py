"""The expert layer for a few tokens on the GPU against its plain statement in
64 bits (tests/fp8_ref.py)."""
import numpy as np
import pytest
import torch

import w4a4_mxfp4_outlier_b200 as w4
from w4a4_mxfp4_outlier_b200 import fp8, moe
from tests import fp8_ref as ref

pytestmark = pytest.mark.gpu


def _bf16(a) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(torch.bfloat16)


def _f64(t) -> np.ndarray:
    return t.double().cpu().numpy()


def _stack(rng, E, rows, cols):
    """Quantised weights with scales that are not powers of two."""
    w = fp8.pack_weight(_bf16(rng.standard_normal((E, rows, cols)) / np.sqrt(cols)))
    w.scale.mul_(torch.from_numpy(rng.uniform(0.7, 1.4, tuple(w.scale.shape)).astype(np.float32)).cuda())
    return w


def _layer(rng, E, k, d, ff, gated, renorm):
    router = _bf16(rng.standard_normal((E, d)) * 2 / np.sqrt(d))
    return moe.MoE(router, _stack(rng, E, ff, d) if gated else None, _stack(rng, E, ff, d),
                   _stack(rng, E, d, ff), top_k=k, act=moe.SILU_GATED if gated else moe.GELU,
                   renorm=renorm)


def _acts(rng, T, d, pad=0):
    x = rng.standard_normal((T, d + pad))
    x[:, rng.random(d + pad) < 0.02] *= 6
    return _bf16(x)[:, :d]


def _ws(T, m):
    # garbage, as a caller's buffer may hold: NaN patterns in every type
    return torch.full((moe.workspace_size(T, m),), 0xFF, dtype=torch.uint8, device="cuda")


def _no_error():
    st, bits = w4.last_error()
    assert st == w4.OK, hex(bits)


def _np(w):
    return w.q.view(torch.uint8).cpu().numpy(), w.scale.cpu().numpy().astype(np.float64)


def _check(X, m, Y, ids, wts):
    x, r, k = _f64(X), _f64(m.router), m.top_k
    logits, lerr, want, _ = ref.route(x, r, k, m.renorm)
    got = ids.cpu().numpy()
    for t in range(x.shape[0]):
        assert len(set(got[t])) == k and got[t].min() >= 0 and got[t].max() < r.shape[0]
        if not np.array_equal(got[t], want[t]):
            # only logits that lie within their errors may change places
            assert (np.abs(logits[t, got[t]] - logits[t, want[t]]) <=
                    2 * lerr[t].max()).all(), (t, got[t], want[t])
    bf16 = Y.dtype == torch.bfloat16
    y, tol, w, werr = ref.moe(x, r, _np(m.gate) if m.gate else None, _np(m.up), _np(m.down), got, k,
                              m.renorm, m.gate is not None, bf16)
    err = np.abs(_f64(Y) - y)
    assert (err <= tol).all(), f"{(err > tol).sum()} of {err.size}, worst {(err / tol).max():.3f}"
    assert (np.abs(_f64(wts) - w) <= werr).all()


# T, E, top_k, d, d_ff, gated, renorm: single tokens and both sides of every
# tile width; one expert; more experts than a warp and the most; every expert
# chosen; widths below a block, off the block grid, with a half-empty last
# tile pair, and with K split over several CTAs
CASES = [
    (1, 1, 1, 16, 16, True, True), (1, 2, 2, 144, 272, False, True), (1, 8, 2, 2048, 1024, True, True),
    (1, 512, 16, 256, 128, True, False), (2, 5, 5, 400, 144, True, False), (3, 20, 3, 1040, 528, False, False),
    (4, 33, 4, 512, 384, True, True), (5, 130, 7, 272, 256, True, True), (15, 8, 2, 528, 640, False, True),
    (16, 64, 8, 512, 256, True, False), (17, 8, 8, 272, 144, True, True), (31, 6, 1, 144, 400, False, True),
    (32, 40, 6, 384, 272, True, True), (33, 16, 4, 656, 128, True, True), (63, 3, 2, 256, 272, False, False),
    (64, 128, 8, 256, 144, True, True), (64, 2, 1, 2064, 16, True, True), (64, 16, 16, 128, 128, False, True),
]


@pytest.mark.parametrize("T,E,k,d,ff,gated,renorm", CASES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_layer(T, E, k, d, ff, gated, renorm, dtype):
    rng = np.random.default_rng([1, T, E, k, d, ff])
    m = _layer(rng, E, k, d, ff, gated, renorm)
    X = _acts(rng, T, d, 24)
    buf = torch.full((T + 2, d + 16), 7.0, dtype=dtype, device="cuda")
    Y = buf[1:T + 1, 8:8 + d]
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    wts = torch.full((T, k), -1.0, device="cuda")
    ws = _ws(T, m)
    moe.forward(X, m, ws, Y, ids, wts)
    _no_error()
    _check(X, m, Y, ids, wts)
    rest = buf.clone()
    rest[1:T + 1, 8:8 + d] = 7.0
    assert (rest == 7.0).all(), "wrote outside Y"
    for _ in range(3):                       # the same workspace, and without the optional outputs
        again = torch.empty(T, d, dtype=dtype, device="cuda")
        moe.forward(X, m, ws, again)
        assert torch.equal(again, Y), "two runs differ"


def test_equal_logits_take_the_lower_index():
    rng = np.random.default_rng(2)
    m = _layer(rng, 40, 6, 256, 128, True, True)
    m.router[:] = m.router[:1]
    X, Y = _acts(rng, 9, 256), torch.empty(9, 256, dtype=torch.bfloat16, device="cuda")
    ids, wts = torch.empty(9, 6, dtype=torch.int32, device="cuda"), torch.empty(9, 6, device="cuda")
    moe.forward(X, m, _ws(9, m), Y, ids, wts)
    assert (ids == torch.arange(6, device="cuda", dtype=torch.int32)).all()
    assert (wts - 1 / 6).abs().max() <= 2.0 ** -23
    _no_error()


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("T", [3, 40])
def test_non_finite_token_stays_alone(bad, T):
    rng = np.random.default_rng([3, T])
    m = _layer(rng, 12, 3, 272, 256, True, True)
    X = _acts(rng, T, 272)
    ws = _ws(T, m)
    Y, Z = (torch.empty(T, 272, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ids = torch.empty(T, 3, dtype=torch.int32, device="cuda")
    moe.forward(X, m, ws, Y)
    X[1, 100] = bad
    moe.forward(X, m, ws, Z, ids)
    assert torch.isnan(Z[1]).all()
    assert ids.min() >= 0 and ids.max() < 12 and len(set(ids[1].tolist())) == 3
    keep = [t for t in range(T) if t != 1]
    # the other tokens' experts may now have other company, so K may be split
    # otherwise: compare with the tolerance of their own values
    y, z = _f64(Y)[keep], _f64(Z)[keep]
    assert (np.abs(y - z) <= 2.0 ** -5 * np.abs(y).max()).all() and np.isfinite(z).all()
    _no_error()


def test_all_tokens_to_one_expert_and_spread():
    # the longest and the shortest lists of tokens, and experts without any
    rng = np.random.default_rng(4)
    m = _layer(rng, 64, 1, 256, 256, True, True)
    T = 64
    X = _acts(rng, T, 256)
    X[:, 0] = 8.0
    for target in (lambda t: 37, lambda t: t, lambda t: 63 - t // 2):
        r = torch.zeros(64, 256)
        m.router.copy_(r)
        X[:, 64:128] = 0
        for t in range(T):
            X[t, 64 + target(t)] = 4.0
            m.router[target(t), 64 + target(t)] = 4.0
        Y = torch.empty(T, 256, dtype=torch.float32, device="cuda")
        ids, wts = torch.empty(T, 1, dtype=torch.int32, device="cuda"), torch.empty(T, 1, device="cuda")
        moe.forward(X, m, _ws(T, m), Y, ids, wts)
        _no_error()
        assert ids[:, 0].tolist() == [target(t) for t in range(T)]
        _check(X, m, Y, ids, wts)


def test_stack_past_32_bits():
    # expert weights whose byte offsets pass 2^32: the last experts of a stack of 4.5 GB
    E, d, ff = 70, 8192, 8192
    gen = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randint(0, 256, (E, ff, d), dtype=torch.uint8, device="cuda", generator=gen)
    q[(q & 0x7F) == 0x7F] = 0x30
    s = torch.full((E, 64, 64), 2.0 ** -12, device="cuda")
    up, down = fp8.Fp8Weight(q, s), fp8.Fp8Weight(q, s)
    router = torch.zeros(E, d, dtype=torch.bfloat16, device="cuda")
    router[68, 0], router[3, 0] = 2.0, 1.0
    m = moe.MoE(router, None, up, down, top_k=2, act=moe.GELU)
    X = _acts(np.random.default_rng(6), 2, d)
    X[:, 0] = 1.0
    Y = torch.empty(2, d, device="cuda")
    ids, wts = torch.empty(2, 2, dtype=torch.int32, device="cuda"), torch.empty(2, 2, device="cuda")
    moe.forward(X, m, _ws(2, m), Y, ids, wts)
    _no_error()
    assert ids.tolist() == [[68, 3], [68, 3]]
    small = moe.MoE(router[[3, 68]].contiguous(), None, fp8.Fp8Weight(q[[3, 68]], s[[3, 68]]),
                    fp8.Fp8Weight(q[[3, 68]], s[[3, 68]]), top_k=2, act=moe.GELU)
    Z = torch.empty(2, d, device="cuda")
    moe.forward(X, small, _ws(2, small), Z, ids, wts)
    assert ids.tolist() == [[1, 0], [1, 0]]
    assert torch.equal(Y, Z)


def test_empty_batch_touches_nothing():
    m = _layer(np.random.default_rng(7), 4, 2, 128, 128, True, True)
    ws = torch.full((64,), 5, dtype=torch.uint8, device="cuda")
    moe.forward(torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"), m, ws,
                torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"))
    assert (ws == 5).all()


def test_two_streams():
    rng = np.random.default_rng(8)
    m = _layer(rng, 32, 4, 1024, 512, True, True)
    jobs = []
    for T in (1, 64, 20, 7):
        X, ws = _acts(rng, T, 1024), _ws(T, m)
        Y, Z = (torch.empty(T, 1024, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        moe.forward(X, m, ws, Z)
        jobs.append((X, ws, Y, Z, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(25):
        for X, ws, Y, _, s in jobs:
            moe.forward(X, m, ws, Y, stream=s)
    torch.cuda.synchronize()
    for _, _, Y, Z, _ in jobs:
        assert torch.equal(Y, Z)
    _no_error()


@pytest.mark.parametrize("T", [1, 24])
def test_run_of_layers_captured_and_replayed(T):
    """As a block of a network would use them: an 8-bit projection, the expert
    layer, another projection, then the 4-bit layer, all on shared scratch."""
    rng = np.random.default_rng([9, T])
    d = 512
    w_in, w_out = (fp8.pack_weight(_bf16(rng.standard_normal((d, d)) / np.sqrt(d))) for _ in range(2))
    m = _layer(rng, 16, 4, d, 384, True, True)
    W4 = _bf16(rng.standard_normal((d, d)) / np.sqrt(d))
    pw = w4.calibrate(_acts(rng, 64, d), W4, 0.5, 16)
    ws = _ws(T, m)
    ws_l = torch.empty(fp8.workspace_size(T, w_in), dtype=torch.uint8, device="cuda")
    ws_4 = torch.empty(w4.workspace_size(T, d, d, 16), dtype=torch.uint8, device="cuda")
    X = _acts(rng, T, d)
    A, B, C, D = (torch.empty(T, d, dtype=torch.bfloat16, device="cuda") for _ in range(4))

    def block(pause=lambda: None):
        fp8.linear(X, w_in, ws_l, A)
        pause()
        moe.forward(A, m, ws, B)
        pause()
        fp8.linear(B, w_out, ws_l, C)
        pause()
        w4.linear(C, pw, ws_4, D)

    block()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        block()
    for seed in range(4):
        X.copy_(_acts(np.random.default_rng([10, seed]), T, d))
        block(torch.cuda.synchronize)
        torch.cuda.synchronize()
        want = [t.clone() for t in (A, B, C, D)]
        for run in (block, g.replay):
            for t in (A, B, C, D):
                t.zero_()
            run()
            torch.cuda.synchronize()
            assert all(torch.equal(t, v) for t, v in zip((A, B, C, D), want))
    _no_error()


def test_binding_refuses():
    rng = np.random.default_rng(11)
    m = _layer(rng, 4, 2, 128, 256, True, True)
    X, ws = _acts(rng, 8, 128), _ws(8, m)
    Y = torch.empty(8, 128, dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: moe.forward(X[:, :64], m, ws, Y), lambda: moe.forward(X.half(), m, ws, Y),
                lambda: moe.forward(X, m, ws[:-1], Y), lambda: moe.forward(X, m, ws, Y[:7]),
                lambda: moe.forward(X, m, ws, Y, torch.empty(8, 2, device="cuda")),
                lambda: moe.forward(X, m, ws, Y, None, torch.empty(8, 3, device="cuda")),
                lambda: moe.workspace_size(65, m),
                lambda: moe.MoE(m.router, None, m.up, m.down, 2),
                lambda: moe.MoE(m.router, m.gate, m.up, m.down, 2, act=moe.GELU),
                lambda: moe.MoE(m.router[:3], m.gate, m.up, m.down, 2),
                lambda: moe.MoE(m.router, m.gate, m.up, m.up, 2),
                lambda: moe.workspace_size(8, moe.MoE(m.router, m.gate, m.up, m.down, 5)),
                lambda: moe.workspace_size(8, moe.MoE(m.router, m.gate, m.up, m.down, 0))):
        with pytest.raises(w4.W4A4Error):
            bad()
