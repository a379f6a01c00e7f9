"""Failure detection of the e4m3 products and the expert layer, without a GPU
fault: w4a4_test_fault shortens the wait limit to 1 ms and makes the kernels
copy no activation tiles, so the waits for them run out.  Every role gives up in
bounded time, the device error word says so, the kernel returns, and with the
hook cleared the same calls on the same buffers give the same bits as before."""
import time

import numpy as np
import pytest
import torch

import w4a4_mxfp4_outlier_b200 as w4
from w4a4_mxfp4_outlier_b200 import fp8, moe

pytestmark = pytest.mark.gpu

TIMEOUTS = 0x7                     # producer, MMA, epilogue


def _bf16(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda().to(torch.bfloat16)


def _gives_up_and_recovers(call, outputs, repeats=1):
    call()
    assert w4.last_error(clear=True)[0] == w4.OK
    want = [t.clone() for t in outputs]
    w4.test_fault(w4.FAULT_FP8_SKIP_ACTS, 1_000_000)
    try:
        t0 = time.monotonic()
        for _ in range(repeats):
            call()
        st, bits = w4.last_error(clear=True)
        took = time.monotonic() - t0
    finally:
        w4.test_fault(0, 0)
    assert st == w4.ERR_TIMEOUT and bits & TIMEOUTS and not bits & ~TIMEOUTS, hex(bits)
    assert took < 5.0
    assert w4.last_error()[0] == w4.OK
    for t in outputs:
        t.zero_()
    call()
    assert w4.last_error()[0] == w4.OK
    assert all(torch.equal(t, v) for t, v in zip(outputs, want))


# few tokens without and with a split (more K blocks than stages), middle, pairs
# with one tile and with several for each
@pytest.mark.parametrize("T,d_in,d_out,repeats", [(3, 128, 128, 1), (40, 1296, 272, 2), (64, 5120, 1040, 1),
                                                  (129, 4000, 2576, 1), (200, 2064, 400, 2), (513, 272, 272, 1),
                                                  (2600, 400, 2064, 1)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_gives_up_and_recovers(T, d_in, d_out, repeats, dtype):
    rng = np.random.default_rng([1, T])
    X, w = _bf16(rng, T, d_in), fp8.pack_weight(_bf16(rng, d_out, d_in))
    ws = torch.empty(fp8.workspace_size(T, w), dtype=torch.uint8, device="cuda")
    Y = torch.empty(T, d_out, dtype=dtype, device="cuda")
    _gives_up_and_recovers(lambda: fp8.linear(X, w, ws, Y), [Y], repeats)


@pytest.mark.parametrize("T,E,k,d,ff,gated", [(1, 4, 2, 1040, 528, True), (7, 20, 3, 272, 400, False),
                                              (64, 16, 8, 512, 384, True)])
def test_expert_layer_gives_up_and_recovers(T, E, k, d, ff, gated):
    rng = np.random.default_rng([2, T])
    pack = lambda *s: fp8.pack_weight(_bf16(rng, *s) / 16)
    m = moe.MoE(_bf16(rng, E, d) / 8, pack(E, ff, d) if gated else None, pack(E, ff, d), pack(E, d, ff), top_k=k,
                act=moe.SILU_GATED if gated else moe.GELU)
    X, Y = _bf16(rng, T, d), torch.empty(T, d, device="cuda")
    ws = torch.empty(moe.workspace_size(T, m), dtype=torch.uint8, device="cuda")
    ids = torch.empty(T, k, dtype=torch.int32, device="cuda")
    _gives_up_and_recovers(lambda: moe.forward(X, m, ws, Y, ids), [Y, ids], 2)
