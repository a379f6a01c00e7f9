"""The e4m3 quantisers, product and linear layer on the GPU against their plain
statement in 64 bits (tests/fp8_ref.py)."""
import ctypes

import numpy as np
import pytest
import torch

import w4a4_mxfp4_outlier_b200 as w4
from w4a4_mxfp4_outlier_b200 import fp8
from tests import fp8_ref as ref

pytestmark = pytest.mark.gpu


def _rng(*key):
    return np.random.default_rng(list(key))


def _bf16(a: np.ndarray) -> torch.Tensor:
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(torch.bfloat16)


def _acts(rng, T, d):
    """Rows with a few large channels."""
    x = 0.3 * rng.standard_normal((T, d))
    x[:, rng.random(d) < 0.01] *= 20
    return _bf16(x)


def _f64(t: torch.Tensor) -> np.ndarray:
    return t.double().cpu().numpy()


def _no_error():
    st, bits = w4.last_error()
    assert st == w4.OK, hex(bits)


def _check_quant(X, act, T, d):
    codes, s = ref.quant_act(_f64(X))
    np.testing.assert_array_equal(act.q.cpu().numpy(), codes)
    got = act.scale.cpu().numpy().astype(np.float64)
    np.testing.assert_array_equal(got[:, :T], s)
    assert (got[:, T:(T + 3) // 4 * 4] == 0).all()


@pytest.mark.parametrize("T,d,pad", [(1, 16, 0), (1, 5120, 0), (3, 144, 8), (5, 128, 0), (33, 1008, 40),
                                     (130, 2064, 16), (1027, 272, 0)])
def test_quant_act(T, d, pad):
    X = _acts(_rng(1, T, d), T, d + pad)[:, :d]
    act = fp8.quant_act(X, fp8.alloc_act(T, d))
    _check_quant(X, act, T, d)
    _no_error()


def test_quant_act_every_finite_pattern_and_edges():
    # every finite bf16 beside a block maximum of its own size, and the block
    # maxima at which the scale changes, with their neighbours
    bits = np.arange(65536, dtype=np.uint32)
    bits = bits[(bits & 0x7F80) != 0x7F80].astype(np.uint16)
    bits = bits[np.argsort(bits & 0x7FFF, kind="stable")]
    bits = np.concatenate([bits, np.zeros(-len(bits) % 1024, np.uint16)]).reshape(-1, 1024)
    X = torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16)
    _check_quant(X, fp8.quant_act(X, fp8.alloc_act(*X.shape)), *X.shape)
    rng = _rng(2)
    top = np.array([(e << 7 | m) for e in range(0, 255) for m in (0, 95, 96, 97, 127)], np.uint16)
    rows = (rng.integers(0, 65536, (len(top), 128)) & 0x8000).astype(np.uint16)
    rows |= (rng.random((len(top), 128)) * (top[:, None] + 1.0)).astype(np.uint16)
    rows[np.arange(len(top)), rng.integers(0, 128, len(top))] = top
    X = torch.from_numpy(rows.view(np.int16)).cuda().view(torch.bfloat16)
    _check_quant(X, fp8.quant_act(X, fp8.alloc_act(*X.shape)), *X.shape)


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan")])
def test_quant_act_non_finite_block(bad):
    X = _acts(_rng(3), 9, 400)
    X[4, 130] = bad
    act = fp8.quant_act(X, fp8.alloc_act(9, 400))
    codes, s = ref.quant_act(_f64(X))
    assert np.isnan(s[1, 4]) and np.isfinite(np.delete(s.reshape(-1), 1 * 9 + 4)).all()
    np.testing.assert_array_equal(act.q.cpu().numpy(), codes)
    np.testing.assert_array_equal(act.scale.cpu().numpy()[:, :9].astype(np.float64), s)
    assert (act.q[4, 128:256] == 0).all()


@pytest.mark.parametrize("experts,rows,cols,pad", [(0, 16, 16, 0), (0, 128, 128, 0), (0, 272, 400, 24),
                                                   (3, 144, 272, 0)])
def test_pack_weight(experts, rows, cols, pad):
    rng = _rng(4, rows, cols)
    shape = (experts, rows, cols) if experts else (rows, cols + pad)
    W = _bf16(0.02 * rng.standard_normal(shape))
    if not experts:
        W = W[:, :cols]
    w = fp8.pack_weight(W)
    Wn, qn, sn = _f64(W), w.q.cpu().numpy(), w.scale.cpu().numpy().astype(np.float64)
    for e in range(max(1, experts)):
        q, s = ref.pack_weight(Wn[e] if experts else Wn)
        np.testing.assert_array_equal(qn[e] if experts else qn, q)
        np.testing.assert_array_equal(sn[e] if experts else sn, s)
    assert (w.d_out, w.d_in, w.experts) == (rows, cols, max(1, experts))


def _random_operands(rng, T, d_in, d_out):
    """Random codes (no NaN) and scales of both signs and several binades."""
    def codes(*shape):
        c = rng.integers(0, 255, shape).astype(np.uint8)
        c[(c & 0x7F) == 0x7F] = 0x38
        return c
    aq, wq = codes(T, d_in), codes(d_out, d_in)
    sa = (rng.standard_normal((ref.blocks(d_in), T)) * 2.0 ** rng.integers(-8, 8, T)).astype(np.float32)
    sw = (rng.standard_normal((ref.blocks(d_out), ref.blocks(d_in))) / 64).astype(np.float32)
    return aq, sa, wq, sw


def _to_gpu(aq, sa, wq, sw):
    T = aq.shape[0]
    act = fp8.alloc_act(T, aq.shape[1])
    act.q.copy_(torch.from_numpy(aq))
    act.scale.fill_(float("nan"))
    act.scale[:, :T] = torch.from_numpy(sa)
    return act, fp8.Fp8Weight(torch.from_numpy(wq).cuda(), torch.from_numpy(sw).cuda())


# single tokens, both sides of every tile width and of the kernels' limit;
# widths of less than a block, off the block grid, with K ranges of a cluster
SHAPES = [(1, 16, 16), (1, 2048, 144), (2, 128, 128), (15, 400, 272), (16, 1040, 128), (17, 256, 16),
          (32, 5120, 256), (33, 144, 528), (48, 1040, 400), (49, 2064, 144), (64, 1168, 384),
          (65, 2048, 272), (127, 272, 1040), (128, 512, 128), (129, 640, 400), (257, 1040, 272),
          (512, 256, 528), (513, 272, 272), (600, 2064, 1552), (769, 128, 16), (1100, 1296, 784),
          # more tiles than CTA pairs, an odd number of K blocks: buffers and stages change places
          (2600, 400, 2064),
          # K split over clusters, of few-token tiles and of large ones, in even and uneven ranges
          (66, 1808, 16), (65, 3856, 400), (128, 5120, 256), (129, 1808, 2064), (129, 4000, 2576),
          (100, 4112, 7184), (200, 4752, 4624), (260, 6416, 4880)]


@pytest.mark.parametrize("T,d_in,d_out", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_gemm(T, d_in, d_out, dtype):
    ops = _random_operands(_rng(5, T, d_in, d_out), T, d_in, d_out)
    act, w = _to_gpu(*ops)
    buf = torch.full((T + 2, d_out + 24), 7.0, dtype=dtype, device="cuda")
    Y = buf[1:T + 1, 8:8 + d_out]
    fp8.gemm(act, w, Y)
    _no_error()
    y, mag = ref.product(*ops)
    tol = ref.product_tolerance(y, mag, d_in, dtype == torch.bfloat16)
    err = np.abs(_f64(Y) - y)
    assert (err <= tol).all(), f"{(err > tol).sum()} of {err.size}, worst {(err / tol).max():.3f}"
    rest = buf.clone()
    rest[1:T + 1, 8:8 + d_out] = 7.0
    assert (rest == 7.0).all(), "wrote outside Y"
    again = torch.empty_like(Y)
    fp8.gemm(act, w, again)
    assert torch.equal(again, Y), "two runs differ"


@pytest.mark.parametrize("T", [1, 40, 200, 700])
def test_linear_is_quant_then_gemm(T):
    rng = _rng(6, T)
    X = _acts(rng, T, 1296 + 16)[:, :1296]
    w = fp8.pack_weight(_bf16(0.02 * rng.standard_normal((528, 1296))))
    ws = torch.empty(fp8.workspace_size(T, w), dtype=torch.uint8, device="cuda")
    Y = torch.empty(T, 528, dtype=torch.bfloat16, device="cuda")
    Y2 = torch.empty_like(Y)
    for _ in range(3):          # back to back on one workspace
        fp8.linear(X, w, ws, Y)
    fp8.gemm(fp8.quant_act(X, fp8.alloc_act(T, 1296)), w, Y2)
    _no_error()
    assert torch.equal(Y, Y2)
    y, mag = ref.product(*ref.quant_act(_f64(X)), w.q.cpu().numpy(), w.scale.cpu().numpy())
    assert (np.abs(_f64(Y) - y) <= ref.product_tolerance(y, mag, 1296, True)).all()


def test_pack_then_linear_without_a_pause():
    # the weight is written by the kernel just before the layer's own two
    rng = _rng(7)
    X, W = _acts(rng, 4, 4096), _bf16(0.02 * rng.standard_normal((2048, 4096)))
    Y, Y2 = (torch.empty(4, 2048, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    w = fp8.pack_weight(W)
    ws = torch.empty(fp8.workspace_size(4, w), dtype=torch.uint8, device="cuda")
    fp8.linear(X, w, ws, Y)
    torch.cuda.synchronize()
    for _ in range(20):
        w.q.zero_()
        w.scale.zero_()
        assert fp8._pack_weight(W.data_ptr(), W.stride(0), ctypes.byref(w.c),
                                torch.cuda.current_stream().cuda_stream) == w4.OK
        fp8.linear(X, w, ws, Y2)
    assert torch.equal(Y, Y2)


@pytest.mark.parametrize("T", [3, 100, 700])
def test_non_finite_token_stays_alone(T):
    rng = _rng(8, T)
    X = _acts(rng, T, 512)
    w = fp8.pack_weight(_bf16(0.02 * rng.standard_normal((272, 512))))
    ws = torch.empty(fp8.workspace_size(T, w), dtype=torch.uint8, device="cuda")
    Y, Z = (torch.empty(T, 272, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fp8.linear(X, w, ws, Y)
    X[1, 300] = float("nan")
    fp8.linear(X, w, ws, Z)
    assert torch.isnan(Z[1]).all()
    keep = [t for t in range(T) if t != 1]
    assert torch.equal(Y[keep], Z[keep])


def test_empty_batch_touches_nothing():
    w = fp8.pack_weight(_bf16(np.ones((128, 128))))
    X = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    Y = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    ws = torch.full((64,), 5, dtype=torch.uint8, device="cuda")
    fp8.linear(X, w, ws, Y)
    fp8.gemm(fp8.quant_act(X, fp8.alloc_act(0, 128)), w, Y)
    assert (ws == 5).all()
    _no_error()


@pytest.mark.parametrize("T,ld", [(100, 1 << 25), (520, 1 << 23)])
def test_offsets_past_32_bits(T, ld):
    rng = _rng(9, T)
    ops = _random_operands(rng, T, 256, 128)
    act, w = _to_gpu(*ops)
    buf = torch.empty(T * ld, dtype=torch.bfloat16, device="cuda")
    Y = buf.view(T, ld)[:, :128]
    fp8.gemm(act, w, Y)
    _no_error()
    y, mag = ref.product(*ops)
    assert (np.abs(_f64(Y) - y) <= ref.product_tolerance(y, mag, 256, True)).all()


@pytest.mark.parametrize("T", [1, 48, 640, 4000])
def test_captured_and_replayed(T):
    rng = _rng(10, T)
    w = fp8.pack_weight(_bf16(0.02 * rng.standard_normal((400, 2048))))
    X = _acts(rng, T, 2048)
    ws = torch.empty(fp8.workspace_size(T, w), dtype=torch.uint8, device="cuda")
    Y, Z = (torch.empty(T, 400, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    fp8.linear(X, w, ws, Y)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fp8.linear(X, w, ws, Y)
        fp8.linear(X, w, ws, Z)
    for seed in range(3):
        X.copy_(_acts(_rng(11, seed), T, 2048))
        Y.zero_()
        g.replay()
        ref_y = torch.empty_like(Y)
        fp8.linear(X, w, ws, ref_y)
        torch.cuda.synchronize()
        assert torch.equal(Y, ref_y) and torch.equal(Z, ref_y)
    _no_error()


def test_two_streams():
    rng = _rng(12)
    w = fp8.pack_weight(_bf16(0.02 * rng.standard_normal((1040, 2048))))
    jobs = []
    for i, T in enumerate((5, 300, 700, 48, 4000)):
        X = _acts(_rng(13, i), T, 2048)
        ws = torch.empty(fp8.workspace_size(T, w), dtype=torch.uint8, device="cuda")
        Y, Z = (torch.empty(T, 1040, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        fp8.linear(X, w, ws, Z)
        jobs.append((X, ws, Y, Z, torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for X, ws, Y, _, s in jobs:
            fp8.linear(X, w, ws, Y, stream=s)
    torch.cuda.synchronize()
    for _, _, Y, Z, _ in jobs:
        assert torch.equal(Y, Z)
    _no_error()


def test_split_k_captured_beside_another_stream():
    # clusters that join through shared memory, in a graph and eagerly at once;
    # a token that is not finite touches no other
    rng = _rng(15)
    w = fp8.pack_weight(_bf16(0.02 * rng.standard_normal((2064, 4112))))
    T = 150
    X, V = _acts(rng, T, 4112), _acts(rng, T, 4112)
    ws, ws2 = (torch.empty(fp8.workspace_size(T, w), dtype=torch.uint8, device="cuda") for _ in range(2))
    Y, Z, U, R, S = (torch.empty(T, 2064, dtype=torch.bfloat16, device="cuda") for _ in range(5))
    fp8.linear(X, w, ws, R)
    fp8.linear(V, w, ws, S)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fp8.linear(X, w, ws, Y)
        fp8.linear(X, w, ws, Z)
    other = torch.cuda.Stream()
    for _ in range(5):
        g.replay()
        fp8.linear(V, w, ws2, U, stream=other)
    torch.cuda.synchronize()
    assert torch.equal(Y, R) and torch.equal(Z, R) and torch.equal(U, S)
    X[149, 4100] = float("inf")
    g.replay()
    torch.cuda.synchronize()
    assert torch.isnan(Y[149]).all() and torch.equal(Y[:149], R[:149])
    _no_error()


def test_binding_refuses():
    w = fp8.pack_weight(_bf16(np.ones((128, 256))))
    X = _acts(_rng(14), 4, 256)
    ws = torch.empty(fp8.workspace_size(4, w), dtype=torch.uint8, device="cuda")
    Y = torch.empty(4, 128, dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: fp8.linear(X[:, :128], w, ws, Y), lambda: fp8.linear(X.float(), w, ws, Y),
                lambda: fp8.linear(X, w, ws[:-1], Y), lambda: fp8.linear(X, w, ws, Y[:3]),
                lambda: fp8.linear(X, w, ws, Y.half()), lambda: fp8.linear(X, w, ws.cpu(), Y),
                lambda: fp8.linear(X, w, ws, torch.empty(128, 4, dtype=torch.bfloat16, device="cuda").T),
                lambda: fp8.linear(X.T.contiguous().T, w, ws, Y),
                lambda: fp8.Fp8Weight(w.q, w.scale.double()), lambda: fp8.Fp8Weight(w.q.T, w.scale.T),
                lambda: fp8.Fp8Weight(w.q, w.scale[:, :1]),
                lambda: fp8.gemm(fp8.alloc_act(4, 128), w, Y),
                lambda: fp8.quant_act(X, fp8.alloc_act(5, 256))):
        with pytest.raises(w4.W4A4Error):
            bad()
