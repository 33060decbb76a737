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
