"""The bounded waits of the attention kernels: a test-only injection stops what
they wait for, so that they run out; the call ends, reports the timeout and
leaves its scratch fit for the next one."""
import time

import numpy as np
import pytest

from tests.gpu_helpers import cuda_or_skip
from tests.test_gpu_kv4_attention import _check, _problem

pytestmark = pytest.mark.gpu


def _run_out(torch, w4, dev, host, flag, scale, **kw):
    first = w4.kv4_attention(**dev, **kw)
    _check(w4, first, host, scale)
    w4.w4a16_debug_inject(flag)
    try:
        t0 = time.monotonic()
        w4.kv4_attention(**dev, **kw)
        status = w4.w4a16_check_device_error()   # synchronises; reads and clears
        waited = time.monotonic() - t0
    finally:
        w4.w4a16_debug_inject(0)
    assert status == 5
    assert 1.5 < waited < 30.0, waited
    for _ in range(3):   # the same context and scratch, the same bits
        assert torch.equal(first, w4.kv4_attention(**dev, **kw))
    assert w4.w4a16_check_device_error() == 0


@pytest.mark.parametrize("requests,Hq,Hkv,D", [(3, 16, 8, 256), (3, 4, 1, 128), (640, 4, 1, 128), (640, 2, 1, 64)])
def test_copies_that_never_come(requests, Hq, Hkv, D):
    # segments that a CTA's warps share, and a warp for each share
    torch, w4 = cuda_or_skip()
    ends = [int(e) for e in np.random.default_rng(D).integers(1, 40, requests)]
    ends[1] = 600
    dev, host = _problem(torch, ends, [1] * requests, Hq, Hkv, D, 16, D)
    _run_out(torch, w4, dev, host, w4.INJECT_STALL_PIPELINE, D ** -0.5, scratch=w4.kv4_attention_scratch(Hq, Hkv, D),
             max_new=1)


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 16, 256), (32, 16, 128), (48, 24, 64)])
@pytest.mark.parametrize("flag", ["producers", "consumers"])
@pytest.mark.parametrize("ends,new", [([600], [300]), ([300, 90, 420], [250, 40, 400])])
def test_items_that_are_never_announced_or_worked_on(Hq, Hkv, D, flag, ends, new):
    # the prompt kernel: no item reaches its roles, or operands are formed and no product is issued
    torch, w4 = cuda_or_skip()
    dev, host = _problem(torch, ends, new, Hq, Hkv, D, 16, D)
    _run_out(torch, w4, dev, host, w4.INJECT_STALL_PIPELINE if flag == "producers" else w4.INJECT_STALL_CONSUMERS,
             D ** -0.5, scratch=w4.kv4_attention_scratch(Hq, Hkv, D), max_new=max(new))


@pytest.mark.parametrize("new", [1, 130])
def test_after_another_call_timed_out(new):
    # the status of an earlier call is still there: this one ends too
    torch, w4 = cuda_or_skip()
    dev, host = _problem(torch, [200, 140], [new] * 2, 32, 16, 128, 16, 3)
    kw = dict(scratch=w4.kv4_attention_scratch(32, 16, 128), max_new=new)
    first = w4.kv4_attention(**dev, **kw)
    x, qw = torch.zeros(512, dtype=torch.bfloat16, device="cuda"), torch.zeros(64, 256, dtype=torch.uint8, device="cuda")
    s = torch.ones(64, 4, dtype=torch.float16, device="cuda")
    torch.cuda.synchronize()
    w4.w4a16_debug_inject(w4.INJECT_STALL_PIPELINE)
    try:
        w4.w4a16_gemv(x, qw, s, s)
        torch.cuda.synchronize()
    finally:
        w4.w4a16_debug_inject(0)
    w4.kv4_attention(**dev, **kw)
    assert w4.w4a16_check_device_error() == 5
    assert torch.equal(first, w4.kv4_attention(**dev, **kw))
    assert w4.w4a16_check_device_error() == 0
