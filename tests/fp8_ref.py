"""Plain statements, in 64 bits, of the e4m3 operators, for their tests."""
from __future__ import annotations

import numpy as np

BLOCK = 128


def e4m3_table() -> np.ndarray:
    """The value of every e4m3 code: 4 exponent bits (bias 7), 3 mantissa bits,
    no infinity, 0x7F / 0xFF NaN."""
    v = np.empty(256, np.float64)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = (m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        v[c] = np.nan if (c & 0x7F) == 0x7F else (-x if c & 0x80 else x)
    return v


TABLE = e4m3_table()
_POS = TABLE[:0x7F]                     # 0 .. 448, ascending: index = code


def e4m3_encode(x: np.ndarray) -> np.ndarray:
    """Codes of the values nearest x, ties to the even code, saturating, sign kept."""
    a = np.minimum(np.abs(x), 448.0)
    hi = np.searchsorted(_POS, a, side="left")          # first value >= a
    lo = np.maximum(hi - 1, 0)
    dlo, dhi = a - _POS[lo], _POS[hi] - a
    code = np.where(dlo < dhi, lo, np.where(dhi < dlo, hi, np.where(lo % 2 == 0, lo, hi)))
    code = np.where(_POS[hi] == a, hi, code)
    return (code | np.where(np.signbit(x), 0x80, 0)).astype(np.uint8)


def pow2_scale(amax: np.ndarray) -> np.ndarray:
    """The smallest 2^e >= 2^-126 with amax <= 448 2^e; NaN where amax is not finite."""
    out = np.empty(amax.shape, np.float64)
    for i, a in np.ndenumerate(amax):
        if not np.isfinite(a):
            out[i] = np.nan
            continue
        e = -126
        if a > 448.0 * 2.0 ** -126:
            e = int(np.floor(np.log2(a / 448.0))) - 1
            while a > 448.0 * 2.0 ** e:
                e += 1
        out[i] = 2.0 ** max(e, -126)
    return out


def blocks(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK


def quant_act(x: np.ndarray):
    """x float64 [T, d] -> codes [T, d], scales [blocks, T]."""
    T, d = x.shape
    nb = blocks(d)
    p = np.zeros((T, nb * BLOCK))
    p[:, :d] = x
    p = p.reshape(T, nb, BLOCK)
    with np.errstate(invalid="ignore"):
        s = pow2_scale(np.abs(p).max(-1))
    ok = np.isfinite(s)[..., None]
    with np.errstate(invalid="ignore"):
        r = np.where(ok, p / s[..., None], 0.0)
    return e4m3_encode(r).reshape(T, -1)[:, :d], s.T


def pack_weight(w: np.ndarray):
    """w float64 [rows, cols] -> codes, scales [row tiles, column tiles]."""
    rows, cols = w.shape
    nr, nc = blocks(rows), blocks(cols)
    p = np.zeros((nr * BLOCK, nc * BLOCK))
    p[:rows, :cols] = w
    t = p.reshape(nr, BLOCK, nc, BLOCK)
    s = pow2_scale(np.abs(t).max(axis=(1, 3)))
    with np.errstate(invalid="ignore"):
        r = np.where(np.isfinite(s)[:, None, :, None], t / s[:, None, :, None], 0.0)
    return e4m3_encode(r).reshape(nr * BLOCK, nc * BLOCK)[:rows, :cols], s


def act_values(q: np.ndarray, s: np.ndarray) -> np.ndarray:
    """Codes [T, d], scales [blocks, T] -> values."""
    return TABLE[q] * np.repeat(s.T.astype(np.float64), BLOCK, axis=1)[:, : q.shape[1]]


def weight_values(q: np.ndarray, s: np.ndarray) -> np.ndarray:
    r = np.repeat(np.repeat(s.astype(np.float64), BLOCK, axis=0), BLOCK, axis=1)
    return TABLE[q] * r[: q.shape[0], : q.shape[1]]


def product(aq, sa, wq, sw):
    """The product and the sum of its terms' magnitudes."""
    a, w = act_values(aq, sa), weight_values(wq, sw)
    return a @ w.T, np.abs(a) @ np.abs(w).T


def product_tolerance(y: np.ndarray, mag: np.ndarray, d_in: int, bf16: bool) -> np.ndarray:
    """Bound of the product's error, from its arithmetic alone.  The 128
    products of a block are exact in float32 (4-bit times 4-bit significands)
    and are added with at most 128 roundings or truncations, the blocks with
    one each, and the scales with three more (their product, the rounding of
    the scaled sum, one join per range of K: at most 8): each at most 2^-23 of
    the magnitudes' sum.  A bf16 output is rounded once more, by at most 2^-8
    of its value (half of finfo.eps)."""
    f32 = (128 + blocks(d_in) + 3 + 8) * 2.0 ** -23 * mag
    return f32 + (2.0 ** -8 * (np.abs(y) + f32) if bf16 else 0.0)


# ---------------------------------------------------------------------------
# Expert layer.  The hidden values are quantised halfway, so a value whose
# rounding error reaches a border of the e4m3 grid may take either neighbour:
# the reference keeps an interval for each hidden value, every code between the
# roundings of its ends (rounding is monotone), and the output's tolerance
# includes the interval.
# ---------------------------------------------------------------------------
EPS = 2.0 ** -23


def route(x, r, k, renorm):
    """Logits, their error bound, the selection and its weights.  Bound: a
    float32 sum of exact products, eight in a chain, then a chain over at most
    ceil(d / 256) of those and five pairwise steps, half an eps each."""
    d = x.shape[1]
    logits = x @ r.T
    err = (8 + -(-d // 256) + 5) * 2.0 ** -24 * (np.abs(x) @ np.abs(r).T)
    idx = np.argsort(-logits, axis=1, kind="stable")[:, :k]
    z = np.exp(logits - logits.max(1, keepdims=True))
    zk = np.take_along_axis(z, idx, 1)
    return logits, err, idx, zk / (zk if renorm else z).sum(1, keepdims=True)


def sigmoid(x):
    return 0.5 * (1.0 + np.tanh(0.5 * x))


def hidden(xq, xs, gate, up, gated):
    """One expert's hidden values for quantised rows and a bound of the float32
    computation's error.  silu' <= 1.1 and gelu' <= 1.13; the sums' errors are
    those of the product; exp, the quotient and the products add some units in
    the last place, of exp's argument where that is large."""
    d_in = xq.shape[1]
    u, mu = product(xq, xs, *up)
    tu = product_tolerance(u, mu, d_in, False)
    if gated:
        g, mg = product(xq, xs, *gate)
        tg = product_tolerance(g, mg, d_in, False)
        h = g * sigmoid(g) * u
        lip = 1.1 * tg * (np.abs(u) + tu) + (np.abs(g * sigmoid(g)) + 1.1 * tg) * tu
        arg = np.abs(g)
    else:
        z = np.sqrt(2 / np.pi) * (u + 0.044715 * u ** 3)
        h = u * sigmoid(2 * z)
        lip = 1.13 * tu
        arg = 2 * np.abs(z)
    return h, lip + (16 + 4 * np.minimum(arg, 88.0)) * EPS * np.abs(h) + 2.0 ** -126


def quant_interval(h, err):
    """Values of the codes of h, and how far another admissible rounding may be."""
    T, d = h.shape
    nb = blocks(d)

    def pad(a):
        p = np.zeros((T, nb * BLOCK))
        p[:, :d] = a
        return p.reshape(T, nb, BLOCK)

    p, e = pad(h), pad(err)
    a, ae = np.abs(p).max(-1), e.max(-1)
    mid = pow2_scale(a)
    lo_s, hi_s = pow2_scale(np.maximum(a - ae, 0)), pow2_scale(a + ae)
    val = TABLE[e4m3_encode(p / mid[..., None])] * mid[..., None]
    lo = np.minimum(*(TABLE[e4m3_encode((p - e) / s[..., None])] * s[..., None] for s in (lo_s, hi_s)))
    hi = np.maximum(*(TABLE[e4m3_encode((p + e) / s[..., None])] * s[..., None] for s in (lo_s, hi_s)))
    dev = np.maximum(hi - val, val - lo)
    return val.reshape(T, -1)[:, :d], np.maximum(dev, 0).reshape(T, -1)[:, :d]


def moe(x, r, gate, up, down, ids, k, renorm, gated, bf16):
    """y and its tolerance for the given selection ids [T, k] (checked apart);
    gate, up, down: (codes, scales) stacks."""
    T, d = x.shape
    xq, xs = quant_act(x)
    logits, lerr, _, _ = route(x, r, k, renorm)
    z = np.exp(logits - logits.max(1, keepdims=True))
    zk = np.take_along_axis(z, ids, 1)
    w = zk / (zk if renorm else z).sum(1, keepdims=True)
    # numerator and denominator each off by the logits' errors (two of them, to
    # first order, with a factor to cover the second) and some roundings
    werr = w * (4.5 * lerr.max(1, keepdims=True) + (z.shape[1] + 32) * EPS)
    y, tol, mag = np.zeros((T, d)), np.zeros((T, d)), np.zeros((T, d))
    for e in np.unique(ids):
        rows, js = np.nonzero(ids == e)
        h, herr = hidden(xq[rows], xs[:, rows], (gate[0][e], gate[1][e]) if gated else None,
                         (up[0][e], up[1][e]), gated)
        hv, hdev = quant_interval(h, herr)
        D = weight_values(down[0][e], down[1][e])
        o = hv @ D.T
        omag = (np.abs(hv) + hdev) @ np.abs(D).T
        otol = hdev @ np.abs(D).T + product_tolerance(o, omag, hv.shape[1], False)
        wt, we = w[rows, js][:, None], werr[rows, js][:, None]
        y[rows] += wt * o
        tol[rows] += wt * otol + we * (np.abs(o) + otol)
        mag[rows] += wt * (np.abs(o) + otol)
    tol += 2 * k * EPS * mag
    if bf16:
        tol += 2.0 ** -8 * (np.abs(y) + tol)
    return y, tol, w, werr
