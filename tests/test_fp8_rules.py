"""The size rules of the 8-bit product (csrc/fp8_rules.h), compiled for the host."""
import ctypes
import os
import subprocess

import numpy as np
import pytest
import torch

import w4a4_mxfp4_outlier_b200 as w4
from w4a4_mxfp4_outlier_b200 import fp8
from tests import fp8_ref as ref

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "w4a4_mxfp4_outlier_b200", "csrc")


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    d = tmp_path_factory.mktemp("rules")
    src, lib = d / "rules.cpp", d / "rules.so"
    src.write_text('#include "fp8_rules.h"\n'
                   'extern "C" int split(long long t, int n, const int* f) { return w4a4::fp8_few_split(t, n, f); }\n'
                   'extern "C" int fit(int q, int c, int p) { return w4a4::fp8_clusters_that_fit(q, c, p); }\n')
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(src), "-o", str(lib)], check=True)
    return ctypes.CDLL(str(lib))


def _fits(**n):
    a = (ctypes.c_int * 9)()
    for c, v in n.items():
        a[int(c[1:])] = v
    return a


# what a B200 holds, two CTAs per SM (148 / 2 slots would be 148, 98, 74, 49, 37)
B200 = dict(c2=148, c3=90, c4=66, c6=44, c8=30)


@pytest.mark.parametrize("tiles,split", [(1, 8), (30, 8), (31, 6), (36, 6), (37, 6), (40, 6), (44, 6), (45, 4), (48, 4),
                                         (49, 4), (66, 4), (67, 3), (74, 3), (90, 3), (91, 2), (98, 2), (108, 2),
                                         (148, 2), (149, 1), (10 ** 7, 1)])
def test_all_clusters_run_at_once(rules, tiles, split):
    assert rules.split(ctypes.c_longlong(tiles), 40, _fits(**B200)) == split
    assert split == 1 or tiles <= B200[f"c{split}"]


@pytest.mark.parametrize("nkb,split", [(1, 1), (2, 2), (3, 3), (5, 4), (7, 6), (8, 8), (100, 8)])
def test_no_more_ranges_than_k_blocks(rules, nkb, split):
    assert rules.split(ctypes.c_longlong(4), nkb, _fits(**B200)) == split


def test_a_smaller_device_takes_smaller_clusters(rules):
    assert rules.split(ctypes.c_longlong(40), 40, _fits(c2=66, c3=40, c4=30, c6=20, c8=14)) == 3
    assert rules.split(ctypes.c_longlong(40), 40, _fits()) == 1


def test_clusters_by_ctas_per_sm(rules):
    # the query may count one CTA per SM where two run, or both
    assert rules.fit(22, 1, 2) == 44 and rules.fit(44, 2, 2) == 44 and rules.fit(74, 1, 1) == 74
    assert rules.fit(22, 0, 2) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("d_out", [3840, 4608, 5632, 5760, 6144, 8448, 8576, 11520, 11664, 18944, 19072])
@pytest.mark.parametrize("T", [1, 48])
def test_product_at_the_rule_s_borders(T, d_out):
    # both sides of the tile counts at which the split changes (30, 44, 66, 90, 148)
    rng = np.random.default_rng([T, d_out])
    d_in = 1152
    aq, wq = (rng.integers(0, 0x7F, s).astype(np.uint8) for s in ((T, d_in), (d_out, d_in)))
    sa = rng.uniform(0.5, 2, (ref.blocks(d_in), T)).astype(np.float32)
    sw = rng.standard_normal((ref.blocks(d_out), ref.blocks(d_in))).astype(np.float32)
    act = fp8.alloc_act(T, d_in)
    act.q.copy_(torch.from_numpy(aq))
    act.scale[:, :T] = torch.from_numpy(sa)
    w = fp8.Fp8Weight(torch.from_numpy(wq).cuda(), torch.from_numpy(sw).cuda())
    Y, Z = (torch.full((T, d_out), 7.0, device="cuda") for _ in range(2))
    fp8.gemm(act, w, Y)
    fp8.gemm(act, w, Z)
    assert w4.last_error()[0] == w4.OK
    y, mag = ref.product(aq, sa, wq, sw)
    assert (np.abs(Y.double().cpu().numpy() - y) <= ref.product_tolerance(y, mag, d_in, False)).all()
    assert torch.equal(Y, Z)
