"""Attention by the tensor cores' kernel repeats itself bit for bit, call after
call: each wait of its roles for one another is for the tile that it means."""
import numpy as np
import pytest

from tests import kv4_helpers as ref
from tests import kv4_long_helpers as lh
from tests.gpu_helpers import cuda_or_skip

pytestmark = pytest.mark.gpu


def _filled(torch, blocks, Hkv, bs, D, g):
    """A cache of random codes, scales and zeros."""
    cache = torch.randint(0, 256, (blocks, Hkv, bs // 16, 18 * D), dtype=torch.uint8, device="cuda", generator=g)
    shape = (blocks, Hkv, bs // 16, D // 2)
    scale = (0.02 + 0.1 * torch.rand(shape, device="cuda", generator=g)).half()
    zero = torch.randint(0, 16, shape, device="cuda", generator=g).half()
    cache[..., 16 * D:] = torch.stack([scale, zero], -1).flatten(-2).view(torch.uint8)
    return cache


@pytest.mark.parametrize("Hq,Hkv,D", [(3, 1, 64), (32, 8, 64), (20, 10, 64), (64, 4, 64), (8, 2, 128), (4, 2, 256)])
def test_prompt_pieces(Hq, Hkv, D):
    # items of one, two and a few key tiles, several to a CTA
    torch, w4 = cuda_or_skip()
    g, rng = torch.Generator("cuda").manual_seed(D + Hq), np.random.default_rng(Hq)
    new = [int(n) for n in rng.integers(40, 300, 60)]
    ends = [n + int(p) for n, p in zip(new, rng.integers(0, 200, 60))]
    width = -(-max(ends) // 64)
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = _filled(torch, 60 * width, Hkv, 64, D, g)
    table = torch.randperm(60 * width, device="cuda", generator=g).to(torch.int32).view(60, width)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(new)]), **i32)
    q = torch.randn(sum(new), Hq, D, device="cuda", generator=g).to(torch.bfloat16)
    args = (q, cache, table, torch.tensor(ends, **i32), cu, w4.kv4_attention_scratch(Hq, Hkv, D))
    first = w4.kv4_attention(*args, max_new=max(new))
    for _ in range(400):
        assert torch.equal(first, w4.kv4_attention(*args, max_new=max(new)))
    # some of the requests against binary64
    c = ref.Cache(60 * width, Hkv, 64, D)
    c.raw = cache.cpu().numpy()
    at = cu.tolist()
    for b in (0, 17, 59):
        rows = slice(at[b], min(at[b] + 40, at[b + 1]))
        n = rows.stop - rows.start
        want, tol = ref.attention(q[rows].double().cpu().numpy(), c, table[b:b + 1].cpu().numpy(), [ends[b] - new[b] + n], [0, n], D ** -0.5)
        lh.check(w4, first[rows], want, tol)


@pytest.mark.parametrize("Hq,Hkv,D", [(16, 8, 64), (64, 4, 64), (8, 2, 128), (16, 8, 256)])
def test_shared_prefixes(Hq, Hkv, D):
    torch, w4 = cuda_or_skip()
    rng = np.random.default_rng(D)
    groups = [(int(rng.integers(1, 40)) * 16, [(int(rng.integers(0, 30)), int(rng.integers(1, 3))) for _ in range(30)]) for _ in range(6)]
    dev, host = lh.grouped(torch, groups, Hq, Hkv, D, 16, D)
    scratch = lh.scratch(w4, dev)
    first = w4.kv4_prefix_attention(**dev, scratch=scratch, max_new=2, max_group=60)
    want, tol = ref.attention(*host, D ** -0.5)
    lh.check(w4, first, want, tol)
    for _ in range(1000):
        assert torch.equal(first, w4.kv4_prefix_attention(**dev, scratch=scratch, max_new=2, max_group=60))
