"""The records of the e4m3 operators (Fp8Weight, Fp8Act, MoE) and what the
library gets of them.  A field cannot be assigned, and a tensor whose memory is
exchanged in place is noticed: a call must never use sizes or addresses that
the record no longer stands for."""
import dataclasses

import numpy as np
import pytest
import torch

import w4a4_mxfp4_outlier_b200 as w4
from w4a4_mxfp4_outlier_b200 import fp8, moe


@pytest.fixture
def host_records(monkeypatch):
    """Lets records be made of host tensors (no call is made with them)."""
    def dense(t, dtypes, shape, device, what):
        if t.dtype not in dtypes or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
            raise w4.W4A4Error(w4.ERR_INVALID_ARG, what)
    monkeypatch.setattr(fp8, "_dense", dense)
    monkeypatch.setattr(moe, "_dense", dense)


def _weight(d_out, d_in, *lead, device="cpu"):
    return fp8.Fp8Weight(torch.zeros(*lead, d_out, d_in, dtype=torch.uint8, device=device),
                         torch.ones(*lead, fp8.blocks(d_out), fp8.blocks(d_in), device=device))


def _layer(E=4, d=128, ff=256, k=2):
    return moe.MoE(torch.zeros(E, d, dtype=torch.bfloat16), _weight(ff, d, E), _weight(ff, d, E),
                   _weight(d, ff, E), top_k=k)


def test_no_field_can_be_assigned(host_records):
    w, m, act = _weight(128, 256), _layer(), fp8.alloc_act(4, 256, device="cpu")
    for record in (w, m, act):
        for f in dataclasses.fields(record):
            before = getattr(record, f.name)
            with pytest.raises(AttributeError):
                setattr(record, f.name, before)
            with pytest.raises(AttributeError):
                delattr(record, f.name)


def test_changed_copies_check_again(host_records):
    m = _layer()
    assert dataclasses.replace(m, top_k=3).c.top_k == 3 and m.c.top_k == 2
    with pytest.raises(w4.W4A4Error):
        dataclasses.replace(m, up=m.down)
    with pytest.raises(w4.W4A4Error):
        dataclasses.replace(m.up, scale=m.down.scale[:2])
    # what c gives out is a copy
    m.c.top_k = 7
    m.up.c.d_in = 7
    assert m._ref._obj.top_k == 2 and m.up._ref._obj.d_in == 128


def test_exchanged_memory_is_noticed(host_records):
    act = fp8.alloc_act(4, 256, device="cpu")
    act.q.data = torch.empty(4, 256, dtype=torch.uint8)
    assert act._args == (act.q.data_ptr(), act.scale.data_ptr(), act.ld)
    w = _weight(128, 256)
    w.scale.data = w.scale * 2
    assert w._ref._obj.scale == w.scale.data_ptr() and w.c.scale == w.scale.data_ptr()
    w.q.set_(torch.zeros(128, 256, dtype=torch.uint8))
    assert w._ref._obj.q == w.q.data_ptr()
    m = _layer()
    for t, where in ((m.router, lambda c: c.router), (m.gate.q, lambda c: c.gate.q),
                     (m.up.scale, lambda c: c.up.scale), (m.down.q, lambda c: c.down.q)):
        t.data = t.clone()
        assert where(m._ref._obj) == t.data_ptr()


def test_exchanged_memory_of_another_shape_is_refused_or_followed(host_records):
    # sizes are taken anew with the addresses, and checked against each other
    w = _weight(128, 256)
    w.q.data = torch.zeros(256, 256, dtype=torch.uint8)
    with pytest.raises(w4.W4A4Error):
        w._ref
    w.scale.data = torch.ones(2, 2)
    assert (w._ref._obj.d_out, w.d_out) == (256, 256)
    m = _layer()
    m.up.q.data = torch.zeros(4, 256, 256, dtype=torch.uint8)
    m.up.scale.data = torch.ones(4, 2, 2)
    with pytest.raises(w4.W4A4Error):
        m._ref
    act = fp8.alloc_act(4, 256, device="cpu")
    act.q.data = torch.empty(8, 256, dtype=torch.uint8)
    with pytest.raises(w4.W4A4Error):
        act._args


def test_calls_take_the_record_before_their_checks(host_records):
    # Y is checked against the sizes the library will get
    w = _weight(128, 256)
    w.q.data, w.scale.data = torch.zeros(256, 256, dtype=torch.uint8), torch.ones(2, 2)
    X = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(w4.W4A4Error):
        fp8.linear(X, w, torch.empty(1 << 16, dtype=torch.uint8), torch.empty(4, 128, dtype=torch.bfloat16))
    assert w.d_out == 256


# ---------------------------------------------------------------------------
def _bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda().to(torch.bfloat16)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [3, 200])
def test_linear_follows_exchanged_memory(T):
    rng = np.random.default_rng([1, T])
    X, w = _bf16(rng.standard_normal((T, 512))), fp8.pack_weight(_bf16(rng.standard_normal((272, 512))))
    ws = torch.empty(fp8.workspace_size(T, w), dtype=torch.uint8, device="cuda")
    Y, Z = (torch.empty(T, 272, device="cuda") for _ in range(2))
    fp8.linear(X, w, ws, Y)
    w.scale.data = w.scale * 2                       # exact: every sum doubles
    torch.empty_like(w.scale).fill_(float("nan"))    # (the old scales' memory, where it is given out again)
    fp8.linear(X, w, ws, Z)
    assert torch.equal(Z, 2 * Y)
    act = fp8.quant_act(X, fp8.alloc_act(T, 512))
    q, s = act.q.clone(), act.scale.clone()
    act.q.data, act.scale.data = torch.zeros_like(act.q), torch.zeros_like(act.scale)
    fp8.quant_act(X, act)
    assert torch.equal(act.q, q) and torch.equal(act.scale[:, :T], s[:, :T])
    fp8.gemm(act, w, Y)
    assert torch.equal(Y, Z)
    assert w4.last_error()[0] == w4.OK


@pytest.mark.gpu
def test_layer_follows_exchanged_memory():
    rng = np.random.default_rng(2)
    E, d, ff, T = 6, 256, 384, 5
    pack = lambda *s: fp8.pack_weight(_bf16(rng.standard_normal(s) / np.sqrt(s[-1])))
    m = moe.MoE(_bf16(rng.standard_normal((E, d)) / 8), pack(E, ff, d), pack(E, ff, d), pack(E, d, ff), top_k=2)
    X, ws = _bf16(rng.standard_normal((T, d))), torch.empty(moe.workspace_size(T, m), dtype=torch.uint8, device="cuda")
    Y, Z = (torch.empty(T, d, device="cuda") for _ in range(2))
    moe.forward(X, m, ws, Y)
    m.down.scale.data = m.down.scale * 2
    moe.forward(X, m, ws, Z)
    assert torch.equal(Z, 2 * Y)
    # one expert fewer per token, in a layer of its own: buffers of its own size
    one = dataclasses.replace(m, top_k=1)
    buf = torch.full((T + 1, 1), -1, dtype=torch.int32, device="cuda")
    moe.forward(X, one, ws, Z, ids=buf[:T])
    assert (buf[:T] >= 0).all() and (buf[T:] == -1).all()
    assert w4.last_error()[0] == w4.OK
