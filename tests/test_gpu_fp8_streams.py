"""fp8.pack_weight on a stream of its own: the result's memory must not be
memory that work still waiting on the current stream will write."""
import pytest
import torch

import w4a4_mxfp4_outlier_b200 as w4
from w4a4_mxfp4_outlier_b200 import fp8

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("handle", [lambda s: s, lambda s: s.cuda_stream], ids=["stream", "handle"])
@pytest.mark.parametrize("shape", [(2048, 2048), (3, 512, 1024)])
def test_pack_on_another_stream_beside_freed_memory(shape, handle):
    W = torch.randn(shape, device="cuda").to(torch.bfloat16)
    want = fp8.pack_weight(W)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    # tensors of the result's sizes, written late on the current stream and freed before that
    junk = [torch.empty_like(want.q), torch.empty_like(want.scale)]
    torch.cuda._sleep(100_000_000)                 # some 50 ms
    for t in junk:
        t.fill_(3)
    del junk, t
    w = fp8.pack_weight(W, stream=handle(s))
    s.synchronize()
    torch.cuda.synchronize()
    assert torch.equal(w.q, want.q) and torch.equal(w.scale, want.scale)
    assert w4.last_error()[0] == w4.OK


def test_pack_on_the_default_stream_by_handle():
    W = torch.randn(256, 400, device="cuda").to(torch.bfloat16)
    want = fp8.pack_weight(W)
    with torch.cuda.stream(torch.cuda.Stream()):
        w = fp8.pack_weight(W, stream=0)
    torch.cuda.synchronize()
    assert torch.equal(w.q, want.q) and torch.equal(w.scale, want.scale)
