"""The quantising write for every scale that binary16 has: the bytes are those of
the formula's divisions, whatever the kernel forms quotients with."""
import numpy as np
import pytest

from tests import kv4_helpers as ref
from tests.gpu_helpers import cuda_or_skip

pytestmark = pytest.mark.gpu


def _groups(rng):
    """Groups of 64 BF16 values, one for each positive finite binary16 scale:
    extremes that give that scale, the rest at and about the middles between
    its steps, where a quotient's last bit decides the code."""
    s = np.arange(1, 0x7c00, dtype=np.uint16).view(np.float16).astype(np.float64)
    hi = (15 * s).astype(np.float32).view(np.uint32) & np.uint32(0xFFFF0000)   # the BF16 number below
    hi = hi.view(np.float32).astype(np.float64)
    x = np.empty((s.size, 64))
    step = rng.integers(-8, 16, (s.size, 64)) + 0.5
    x[:] = ref.bf16(step * s[:, None] * (1 + rng.choice([0, 0, 2.0 ** -8, -2.0 ** -8], (s.size, 64))))
    lo = ref.bf16(hi - 15 * s)
    np.clip(x, lo[:, None], hi[:, None], out=x)
    x[:, 0], x[:, 1] = hi, lo
    return x


def test_every_scale():
    torch, w4 = cuda_or_skip()
    rng = np.random.default_rng(1)
    k, v = _groups(rng)[:, None], -_groups(rng)[:, None]
    T = k.shape[0]
    want = ref.Cache(-(-T // 256), 1, 256, 64)
    want.append(k, v, np.arange(T))
    scales = [ref.quantise(x)[1] for x in (k, v)]
    assert len(np.unique(np.concatenate(scales))) == T
    cache = w4.kv4_cache(want.blocks, 1, 256, 64)
    dev = lambda x: torch.tensor(x, device="cuda").to(torch.bfloat16)
    w4.kv4_append(dev(k), dev(v), cache, torch.arange(T, device="cuda"))
    assert np.array_equal(cache.cpu().numpy(), want.raw)
