"""What is measured of the 8-bit operators: the block quantiser, the linear
layer on e4m3 operands with one scale per block of 128, and the
mixture-of-experts layer for a few tokens.

Formats.  An activation row is cut into blocks of 128 columns, a weight matrix
into tiles of 128 x 128; each block has one float32 scale s, its elements are
e4m3 codes c, and it stands for the values c * s.  Activations are quantised
by the operators: s is the smallest power of two with max|x| <= 448 s (2^-126
at the least), c the e4m3 value nearest x / s.  Weights come quantised, as a
checkpoint holds them, with s = max|w| / 448, any float32 number.
"""
import math

import torch

own = False

DEV = "cuda"
BLOCK = 128


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # activations of a whole batch, the width of the up projection
        {"name": "quant_4096x5120", "kind": "quant", "T": 4096, "d": 5120, "pad": 0},
        # a ragged batch out of a wider buffer; 1008 = 7 * 128 + 112 columns, the last block is partial
        {"name": "quant_333x1008_strided", "kind": "quant", "T": 333, "d": 1008, "pad": 40},
        # one token through the up projection: latency, the weight is read once
        {"name": "linear_1_up", "kind": "linear", "T": 1, "d_in": 5120, "d_out": 13824, "pad": 0},
        # a few dozen tokens through the down projection: a serving batch, or a short tail of a sequence
        {"name": "linear_48_down", "kind": "linear", "T": 48, "d_in": 13824, "d_out": 5120, "pad": 0},
        # a middling, odd batch with dimensions off the block grid, rows out of a wider buffer
        {"name": "linear_300_odd", "kind": "linear", "T": 300, "d_in": 4880, "d_out": 5136, "pad": 24},
        # a full batch through the up projection
        {"name": "linear_4096_up", "kind": "linear", "T": 4096, "d_in": 5120, "d_out": 13824, "pad": 0},
        # the largest: a long sequence through the down projection
        {"name": "linear_16384_down", "kind": "linear", "T": 16384, "d_in": 13824, "d_out": 5120, "pad": 0},
        # one token, many small experts: latency of the whole chain
        {"name": "moe_1_small", "kind": "moe", "T": 1, "E": 64, "k": 6, "d": 2048, "ff": 1024,
         "act": "silu", "renorm": True},
        # one token, few large experts
        {"name": "moe_1_large", "kind": "moe", "T": 1, "E": 8, "k": 2, "d": 5120, "ff": 13824,
         "act": "silu", "renorm": True},
        # a small serving batch over many experts
        {"name": "moe_16_many", "kind": "moe", "T": 16, "E": 128, "k": 8, "d": 2048, "ff": 768,
         "act": "silu", "renorm": True},
        # odd sizes: dimensions off the block grid, experts without a gate, weights of all experts' softmax
        {"name": "moe_7_odd", "kind": "moe", "T": 7, "E": 20, "k": 3, "d": 1040, "ff": 528,
         "act": "gelu", "renorm": False},
        # the most tokens: nearly every expert has some
        {"name": "moe_64_wide", "kind": "moe", "T": 64, "E": 64, "k": 8, "d": 5120, "ff": 1536,
         "act": "silu", "renorm": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["quant", "linear", "linear", "moe", "moe"])
    pad = rng.choice([0, 8 * rng.randrange(1, 9)])
    if kind == "quant":
        return {"kind": kind, "T": _log(rng, 1, 8192), "d": 16 * _log(rng, 1, 864), "pad": pad}
    if kind == "linear":
        return {"kind": kind, "T": _log(rng, 1, 8192), "d_in": 16 * _log(rng, 8, 864),
                "d_out": 16 * _log(rng, 8, 864), "pad": pad}
    E = _log(rng, 4, 128)
    return {"kind": kind, "T": _log(rng, 1, 64), "E": E, "k": rng.randint(1, min(8, E)),
            "d": 16 * _log(rng, 16, 240), "ff": 16 * _log(rng, 8, 96),
            "act": rng.choice(["silu", "silu", "gelu"]), "renorm": rng.random() < 0.7}


def _blocks(n):
    return (n + BLOCK - 1) // BLOCK


def work(case):
    if case["kind"] == "quant":
        T, d = case["T"], case["d"]
        return {"bytes": 3 * T * d + 4 * T * _blocks(d), "flops": 0}
    if case["kind"] == "linear":
        T, d, n = case["T"], case["d_in"], case["d_out"]
        return {"bytes": 2 * T * d + n * d + 4 * _blocks(n) * _blocks(d) + 2 * T * n,
                "flops": 2 * T * n * d}
    T, E, k, d, ff = case["T"], case["E"], case["k"], case["d"], case["ff"]
    mats = 3 if case["act"] == "silu" else 2
    # the experts that T tokens meet on average, each one's weights read once
    met = E * (1.0 - (1.0 - k / E) ** T)
    return {"bytes": met * mats * d * ff + 2 * E * d + 4 * T * d, "flops": 2 * T * k * mats * d * ff + 2 * T * E * d}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _rows(g, T, d, pad):
    """bf16 activations [T, d], a few channels much larger than the rest, out of rows of d + pad."""
    x = torch.randn(T, d + pad, generator=g, device=DEV)
    ch = torch.rand(d + pad, generator=g, device=DEV)
    x *= 0.3 * torch.where(ch > 0.99, 8.0 + 2000.0 * (ch - 0.99), torch.ones_like(ch))
    return x.to(torch.bfloat16)[:, :d]


def _checkpoint(g, rows, cols, sigma):
    """A weight as a checkpoint holds it: e4m3 codes and one float32 scale per 128 x 128 tile."""
    nr, nc = _blocks(rows), _blocks(cols)
    w = sigma * torch.randn(rows, cols, generator=g, device=DEV)
    p = torch.zeros(nr * BLOCK, nc * BLOCK, device=DEV)
    p[:rows, :cols] = w
    t = p.view(nr, BLOCK, nc, BLOCK)
    s = t.abs().amax(dim=(1, 3)) / 448.0
    c = (t / s[:, None, :, None]).clamp(-448.0, 448.0).view(nr * BLOCK, nc * BLOCK)[:rows, :cols]
    return c.to(torch.float8_e4m3fn), s


def _experts(g, E, rows, cols, sigma):
    q = torch.empty(E, rows, cols, dtype=torch.float8_e4m3fn, device=DEV)
    s = torch.empty(E, _blocks(rows), _blocks(cols), device=DEV)
    for e in range(E):
        q[e], s[e] = _checkpoint(g, rows, cols, sigma)
    return q, s


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = {"case": case}
    if case["kind"] == "quant":
        st["X"] = _rows(g, case["T"], case["d"], case["pad"])
    elif case["kind"] == "linear":
        st["X"] = _rows(g, case["T"], case["d_in"], case["pad"])
        st["W"] = _checkpoint(g, case["d_out"], case["d_in"], 0.02)
    else:
        E, d, ff = case["E"], case["d"], case["ff"]
        st["X"] = _rows(g, case["T"], d, 0)
        st["router"] = (torch.randn(E, d, generator=g, device=DEV) * (2.0 / math.sqrt(d))).to(torch.bfloat16)
        st["gate"] = _experts(g, E, ff, d, 0.02) if case["act"] == "silu" else None
        st["up"] = _experts(g, E, ff, d, 0.02)
        st["down"] = _experts(g, E, d, ff, 0.02)
    return st


# ---------------------------------------------------------------------------
# the plain forms: elementary torch operations in 32 bits
# ---------------------------------------------------------------------------
def _split(x):
    """[..., d] as [..., blocks, 128], zeros behind the last column."""
    d = x.shape[-1]
    n = _blocks(d)
    if n * BLOCK != d:
        x = torch.cat([x, x.new_zeros(*x.shape[:-1], n * BLOCK - d)], dim=-1)
    return x.reshape(*x.shape[:-1], n, BLOCK)


def _quantise(x):
    """float32 [..., d] -> e4m3 codes [..., d] and scales [..., blocks]."""
    t = _split(x)
    m, ex = torch.frexp(t.abs().amax(dim=-1))            # amax = m 2^ex, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(m > 0, ex - 9 + (m > 0.875).to(ex.dtype), -126).clamp(min=-126)
    s = ((e + 127) << 23).view(torch.float32)            # 2^e
    c = (t / s[..., None]).to(torch.float8_e4m3fn)       # the quotient by a power of two is exact
    return c.reshape(*x.shape[:-1], -1)[..., : x.shape[-1]], s


def _values(c, s):
    """float32 values of codes [..., d] with scales [..., blocks]."""
    return c.float() * s.repeat_interleave(BLOCK, dim=-1)[..., : c.shape[-1]]


def _tile_values(c, s):
    """float32 values of a weight (or a stack of them): codes [..., rows, cols], scales per tile."""
    r = s.repeat_interleave(BLOCK, dim=-2)[..., : c.shape[-2], :]
    return _values(c, r)


def _activation(case, gate, up):
    if case["act"] == "silu":
        return gate / (1.0 + torch.exp(-gate)) * up
    u = 0.7978845608028654 * (up + 0.044715 * up * up * up)
    return up / (1.0 + torch.exp(-2.0 * u))


def _route(case, logits):
    k = case["k"]
    best, idx = torch.sort(logits, dim=-1, descending=True, stable=True)
    part = best[:, :k] - best[:, :1]
    den = (part if case["renorm"] else best - best[:, :1]).exp().sum(-1, keepdim=True)
    return idx[:, :k], part.exp() / den


def _pick(w, at):
    """The chosen experts' matrices of a stack, in 32 bits."""
    return _tile_values(w[0].view(torch.uint8)[at].view(torch.float8_e4m3fn), w[1][at])


def _plain_moe(st):
    case, X = st["case"], st["X"]
    T, E, k = case["T"], case["E"], case["k"]
    idx, wt = _route(case, X.double() @ st["router"].double().T)
    x = _values(*_quantise(X.float()))
    if T * k < E:        # one matrix for each (token, choice)
        at = idx.reshape(-1)
        xp = x.repeat_interleave(k, dim=0)[:, :, None]
        up = torch.bmm(_pick(st["up"], at), xp)[:, :, 0]
        gate = torch.bmm(_pick(st["gate"], at), xp)[:, :, 0] if st["gate"] else None
        h = _values(*_quantise(_activation(case, gate, up)))
        o = torch.bmm(_pick(st["down"], at), h[:, :, None])[:, :, 0].view(T, k, -1)
    else:                # every expert on every token, the chosen ones taken
        up = torch.matmul(x, _tile_values(*st["up"]).transpose(1, 2))
        gate = torch.matmul(x, _tile_values(*st["gate"]).transpose(1, 2)) if st["gate"] else None
        h = _values(*_quantise(_activation(case, gate, up)))
        o = torch.bmm(h, _tile_values(*st["down"]).transpose(1, 2))
        o = o[idx, torch.arange(T, device=DEV)[:, None]]
    y = (o * wt.float()[:, :, None]).sum(1)
    return y.to(torch.bfloat16), idx.to(torch.int32), wt.float()


def _plain(st):
    kind = st["case"]["kind"]
    if kind == "quant":
        c, s = _quantise(st["X"].float())
        return c, s.T.contiguous()
    if kind == "linear":
        x = _values(*_quantise(st["X"].float()))
        return (x @ _tile_values(*st["W"]).T).to(torch.bfloat16)
    return _plain_moe(st)


# ---------------------------------------------------------------------------
# the framework's operators
# ---------------------------------------------------------------------------
def _own(st):
    from w4a4_mxfp4_outlier_b200 import fp8, moe
    case, X = st["case"], st["X"]
    if case["kind"] == "quant":
        if "out" not in st:
            st["out"] = fp8.alloc_act(case["T"], case["d"], X.device)
        fp8.quant_act(X, st["out"])
        return st["out"].q.view(torch.float8_e4m3fn), st["out"].scale[:, : case["T"]]
    if case["kind"] == "linear":
        if "w" not in st:
            st["w"] = fp8.Fp8Weight(*st["W"])
            st["ws"] = torch.empty(fp8.workspace_size(case["T"], st["w"]), dtype=torch.uint8, device=X.device)
            st["Y"] = torch.empty(case["T"], case["d_out"], dtype=torch.bfloat16, device=X.device)
        fp8.linear(X, st["w"], st["ws"], st["Y"])
        return st["Y"]
    if "m" not in st:
        st["m"] = moe.MoE(st["router"], fp8.Fp8Weight(*st["gate"]) if st["gate"] else None,
                          fp8.Fp8Weight(*st["up"]), fp8.Fp8Weight(*st["down"]), top_k=case["k"],
                          act=moe.SILU_GATED if case["act"] == "silu" else moe.GELU, renorm=case["renorm"])
        st["ws"] = torch.empty(moe.workspace_size(case["T"], st["m"]), dtype=torch.uint8, device=X.device)
        st["Y"] = torch.empty(case["T"], case["d"], dtype=torch.bfloat16, device=X.device)
        st["ids"] = torch.empty(case["T"], case["k"], dtype=torch.int32, device=X.device)
        st["wt"] = torch.empty(case["T"], case["k"], device=X.device)
    moe.forward(X, st["m"], st["ws"], st["Y"], st["ids"], st["wt"])
    return st["Y"], st["ids"], st["wt"]


def run(state):
    if own:
        return _own(state)
    return _plain(state)


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------
def _two_to(e):
    """2^e exactly, for whole float64 e of normal numbers."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _exact_codes(x):
    """float64 [T, d] -> values of the codes [T, d] and scales [T, blocks], from the definition."""
    T, d = x.shape
    c = torch.empty_like(x)
    s = torch.empty(T, _blocks(d), dtype=torch.float64, device=x.device)
    for b in range(_blocks(d)):
        v = x[:, b * BLOCK: (b + 1) * BLOCK]
        a = v.abs().max(dim=1).values
        e = torch.floor(torch.log2((a / 448.0).clamp(min=2.0 ** -140))) - 1.0
        for _ in range(3):                                # the smallest e with a <= 448 2^e
            e = torch.where(a > 448.0 * _two_to(e), e + 1.0, e)
        s[:, b] = _two_to(e.clamp(min=-126.0))
        r = v / s[:, b: b + 1]
        ex = torch.floor(torch.log2(r.abs().clamp(min=2.0 ** -6)))
        ex = torch.where(_two_to(ex) > r.abs().clamp(min=2.0 ** -6), ex - 1.0, ex)
        ex = torch.where(_two_to(ex + 1.0) <= r.abs(), ex + 1.0, ex)
        step = _two_to(ex - 3.0)                   # e4m3: three bits behind the first, 2^-9 at the least
        c[:, b * BLOCK: (b + 1) * BLOCK] = torch.round(r / step) * step
    return c, s


def _exact_weight(c, s):
    w = c.double()
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            w[i * BLOCK: (i + 1) * BLOCK, j * BLOCK: (j + 1) * BLOCK] *= s[i, j].double()
    return w


def _exact_scaled(x):
    c, s = _exact_codes(x)
    for b in range(s.shape[1]):
        c[:, b * BLOCK: (b + 1) * BLOCK] *= s[:, b: b + 1]
    return c


def exact(case, seed):
    st = prepare(case, seed)
    X = st["X"].double()
    if case["kind"] == "quant":
        c, s = _exact_codes(X)
        return c, s.T.contiguous()
    if case["kind"] == "linear":
        return torch.matmul(_exact_scaled(X), _exact_weight(*st["W"]).T)
    T, k = case["T"], case["k"]
    p = torch.matmul(X, st["router"].double().T)
    p = torch.exp(p - p.max(dim=1, keepdim=True).values)
    p = p / p.sum(dim=1, keepdim=True)
    ids = torch.empty(T, k, dtype=torch.int32)
    wt = torch.empty(T, k, dtype=torch.float64)
    left = p.cpu()
    for t in range(T):
        row = left[t].tolist()
        order = sorted(range(len(row)), key=lambda e: (-row[e], e))[:k]
        total = sum(row[e] for e in order) if case["renorm"] else 1.0
        for j, e in enumerate(order):
            ids[t, j], wt[t, j] = e, row[e] / total
    x = _exact_scaled(X)
    y = torch.zeros(T, case["d"], dtype=torch.float64, device=X.device)
    for e in sorted(set(ids.reshape(-1).tolist())):
        at = (ids == e).nonzero()
        rows = at[:, 0].to(X.device)
        up = x[rows] @ _exact_weight(st["up"][0][e], st["up"][1][e]).T
        if case["act"] == "silu":
            gt = x[rows] @ _exact_weight(st["gate"][0][e], st["gate"][1][e]).T
            h = gt * torch.sigmoid(gt) * up
        else:
            h = 0.5 * up * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (up + 0.044715 * up ** 3)))
        o = _exact_scaled(h) @ _exact_weight(st["down"][0][e], st["down"][1][e]).T
        y[rows] += o * wt[at[:, 0], at[:, 1]].to(X.device)[:, None]
    return y, ids, wt
