"""Host-side checks of the e4m3 operators: the plain statement the GPU tests
compare with, and the refusals (invalid calls return a status and enqueue
nothing)."""
import ctypes

import numpy as np
import pytest
import torch

import w4a4_mxfp4_outlier_b200 as w4
from w4a4_mxfp4_outlier_b200 import fp8
from tests import fp8_ref as ref


def test_e4m3_table_agrees_with_torch():
    v = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(np.nan_to_num(ref.TABLE, nan=1e9), np.nan_to_num(v, nan=1e9))


def test_e4m3_encode_is_nearest_even():
    # every value, every midpoint and both neighbours of each midpoint
    mids = (ref._POS[1:] + ref._POS[:-1]) / 2
    for c in range(0x7F):
        assert ref.e4m3_encode(np.array([ref._POS[c]]))[0] == c
    for i, m in enumerate(mids):
        even = i if i % 2 == 0 else i + 1
        got = ref.e4m3_encode(np.array([np.nextafter(m, 0), m, np.nextafter(m, 1e9), -m]))
        assert list(got) == [i, even, i + 1, even | 0x80]
    assert list(ref.e4m3_encode(np.array([1e9, -1e9, 0.0, -0.0]))) == [0x7E, 0xFE, 0x00, 0x80]


@pytest.mark.parametrize("amax,e", [(448.0, 0), (449.0, 1), (224.0, -1), (225.0, 0), (0.0, -126),
                                    (2.0 ** -133, -126), (3.3895e38, 120)])
def test_pow2_scale(amax, e):
    assert ref.pow2_scale(np.array([amax]))[0] == 2.0 ** e


F = 0x1000      # a 16-byte aligned address that no refused call reads


def _w(d_in=256, d_out=128, experts=1, q=F, scale=F):
    return ctypes.byref(fp8.Fp8WeightC(d_in, d_out, experts, q, scale))


INV, SHAPE = w4.ERR_INVALID_ARG, w4.ERR_UNSUPPORTED_SHAPE


@pytest.mark.parametrize("args,status", [
    ((F, 8, 256, 255, F, F, 8), INV),            # ldx < d
    ((F, -1, 256, 256, F, F, 8), INV),
    ((F, 8, 0, 256, F, F, 8), INV),
    ((F, 8, 256, 256, F, F, 7), INV),            # ld_scale < T
    ((F, 9, 256, 256, F, F, 9), INV),            # ld_scale below T rounded up to 4
    ((None, 8, 256, 256, F, F, 8), INV),
    ((F, 8, 256, 256, None, F, 8), INV),
    ((F, 8, 256, 256, F, None, 8), INV),
    ((F, 8, 248, 256, F, F, 8), SHAPE),          # d % 16
    ((F, 8, 65552, 65552, F, F, 8), SHAPE),      # d > 65535
    ((F, 8, 256, 260, F, F, 8), SHAPE),          # ldx % 8
    ((F, 8, 256, 256, F, F, 10), SHAPE),         # ld_scale % 4
    ((F + 8, 8, 256, 256, F, F, 8), SHAPE),
    ((F, 8, 256, 256, F + 4, F, 8), SHAPE),
    ((F, 8, 256, 256, F, F + 4, 8), SHAPE),
    ((F, (1 << 31) - 200, 256, 256, F, F, 1 << 31), SHAPE),
    ((None, 0, 256, 256, None, None, 0), w4.OK),
])
def test_quant_act_refusals(args, status):
    assert fp8._quant_act(*args, None) == status


@pytest.mark.parametrize("kw,status", [
    (dict(d_in=0), INV), (dict(d_out=-16), INV), (dict(experts=0), INV), (dict(q=None), INV),
    (dict(scale=None), INV), (dict(d_in=264), SHAPE), (dict(d_out=136), SHAPE),
    (dict(d_in=65536), SHAPE), (dict(q=F + 8), SHAPE), (dict(scale=F + 2), SHAPE),
    (dict(experts=65536), SHAPE),
])
def test_weight_refusals(kw, status):
    assert fp8._pack_weight(F, 70000, _w(**kw), None) == status
    assert fp8._gemm(F, F, 8, 8, _w(**kw), F, 256, 0, None) == status
    assert fp8._linear(F, 8, 70000, _w(**kw), F, 1 << 30, F, 256, 0, None) == status


def test_pack_refusals():
    assert fp8._pack_weight(None, 256, _w(), None) == INV
    assert fp8._pack_weight(F, 255, _w(), None) == INV
    assert fp8._pack_weight(F, 260, _w(), None) == SHAPE
    assert fp8._pack_weight(F + 2, 256, _w(), None) == SHAPE
    assert fp8._pack_weight(F, 256, None, None) == INV
    assert fp8._pack_weight(F, 256, _w(d_out=128 * 65536), None) == SHAPE


def test_gemm_and_linear_refusals():
    g = fp8._gemm
    assert g(F, F, 8, 8, None, F, 128, 0, None) == INV
    assert g(F, F, 8, 8, _w(experts=2), F, 128, 0, None) == INV       # a stack is not one weight
    assert g(F, F, 8, -1, _w(), F, 128, 0, None) == INV
    assert g(F, F, 8, 8, _w(), F, 127, 0, None) == INV                # ldy < d_out
    assert g(F, F, 4, 8, _w(), F, 128, 0, None) == INV                # ld_scale < T
    assert g(F, F, 8, 8, _w(), F, 132, 0, None) == SHAPE              # ldy % 8
    assert g(F, F, 10, 8, _w(), F, 128, 0, None) == SHAPE
    for a, s, y in ((None, F, F), (F, None, F), (F, F, None)):
        assert g(a, s, 8, 8, _w(), y, 128, 0, None) == INV
    for a, s, y in ((F + 1, F, F), (F, F + 4, F), (F, F, F + 8)):
        assert g(a, s, 8, 8, _w(), y, 128, 0, None) == SHAPE
    assert g(None, None, 0, 0, _w(), None, 128, 0, None) == w4.OK
    n = ctypes.c_size_t()
    assert fp8._workspace_size(8, 256, ctypes.byref(n)) == w4.OK and n.value == 2048 + 1024
    assert fp8._workspace_size(-1, 256, ctypes.byref(n)) == INV
    assert fp8._workspace_size(8, 250, ctypes.byref(n)) == SHAPE
    assert fp8._workspace_size(8, 256, None) == INV
    li = fp8._linear
    assert li(F, 8, 256, _w(), F, 3071, F, 128, 0, None) == INV       # workspace too small
    assert li(F, 8, 256, _w(), None, 1 << 20, F, 128, 0, None) == INV
    assert li(F, 8, 256, _w(), F + 4, 1 << 20, F, 128, 0, None) == SHAPE
    assert li(F, 8, 255, _w(), F, 1 << 20, F, 128, 0, None) == INV
    assert li(None, 8, 256, _w(), F, 1 << 20, F, 128, 0, None) == INV
    assert li(F, 8, 256, _w(), F, 1 << 20, F, 120, 0, None) == INV
    assert li(F, 8, 256, _w(), F, 1 << 20, F, 132, 0, None) == SHAPE
    assert li(None, 0, 256, _w(), None, 0, None, 128, 0, None) == w4.OK


def test_binding_refuses_host_tensors():
    with pytest.raises(w4.W4A4Error):
        fp8.Fp8Weight(torch.zeros(128, 128, dtype=torch.uint8), torch.zeros(1, 1))
    with pytest.raises(w4.W4A4Error):
        fp8.pack_weight(torch.zeros(128, 128, dtype=torch.bfloat16))
    with pytest.raises(w4.W4A4Error):
        fp8.quant_act(torch.zeros(4, 128, dtype=torch.bfloat16),
                      fp8.alloc_act(4, 128, device="cpu"))
