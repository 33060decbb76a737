"""Attention over the paged 4-bit cache against binary64, with the error bound
derived in kv4_helpers.attention."""
import numpy as np
import pytest

from tests import kv4_helpers as ref
from tests.gpu_helpers import cuda_or_skip

pytestmark = pytest.mark.gpu

POISON = np.array([0x7E00, 0xFC00, 0x7C00, 0x7BFF], np.uint16)   # NaN, -inf, inf, the largest


def _problem(torch, ends, new, Hq, Hkv, D, bs, seed, gap=0, spread=1.0):
    """A cache with the requests' tokens in scattered pages; every other token
    place of it holds NaN, infinite or huge parameters."""
    rng = np.random.default_rng(seed)
    held = [max(0, -(-e // bs)) for e in ends]
    blocks = sum(held) + 3
    c = ref.Cache(blocks, Hkv, bs, D, 0xFF)
    par = c.raw[..., 16 * D:].view(np.uint16)
    par[...] = POISON[rng.integers(0, 4, par.shape)]
    ids = rng.permutation(blocks)
    table = np.full((len(ends), max(held + [1]) + 2), -1)
    at = 0
    for b, h in enumerate(held):
        table[b, :h] = ids[at:at + h]
        at += h
        for j in range(max(0, ends[b])):
            slot = int(table[b, j // bs]) * bs + j % bs
            for part in (0, 1):
                for hd in range(Hkv):
                    s = rng.uniform(0.02, 0.3, D // 64) * spread ** rng.uniform(-1, 1)
                    z = rng.integers(0, 16, D // 64)
                    c.put(part, slot, hd, rng.integers(0, 16, D).astype(np.uint8), s.astype(np.float16), z)
    cu = np.concatenate([[0], np.cumsum(new)])
    q = ref.bf16(rng.normal(0, 1, (cu[-1] + gap, Hq, D)))
    dev = dict(q=torch.tensor(q, device="cuda").to(torch.bfloat16), cache=torch.tensor(c.raw, device="cuda"),
               block_table=torch.tensor(table, dtype=torch.int32, device="cuda"),
               seq_lens=torch.tensor(ends, dtype=torch.int32, device="cuda"),
               cu_new=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    return dev, (q, c, table, ends, cu)


def _check(w4, out, host, scale, window=0, sinks=0):
    q, c, table, ends, cu = host
    want, tol = ref.attention(q, c, table, ends, cu, scale, window, sinks)
    got = out.double().cpu().numpy()
    bad = np.abs(got - want) > tol
    assert np.isfinite(got).all()
    assert not bad.any(), "%d of %d off, first %s: %r, want %r +- %r" % (
        bad.sum(), bad.size, np.argwhere(bad)[0], got[bad][0], want[bad][0], tol[bad][0])
    assert w4.w4a16_check_device_error() == 0


HEADS = [(16, 8, 256), (8, 1, 128), (4, 4, 64), (14, 2, 128), (16, 1, 64), (20, 1, 256), (3, 3, 256), (10, 2, 128)]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("bs", [16, 64])
def test_decode(Hq, Hkv, D, bs):
    # one token each, lengths around the tiles' and pages' ends
    torch, w4 = cuda_or_skip()
    ends = [1, 2, 15, 16, 17, 31, 33, 64, 65, 200]
    dev, host = _problem(torch, ends, [1] * len(ends), Hq, Hkv, D, bs, Hq * D + bs)
    out = w4.kv4_attention(**dev, scratch=w4.kv4_attention_scratch(Hq, Hkv, D), max_new=1)
    _check(w4, out, host, D ** -0.5)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 4), (16, 17), (100, 3), (33, 200), (1000, 4), (7, 16)])
@pytest.mark.parametrize("Hq,Hkv,D", [(16, 8, 256), (7, 1, 128)])
def test_decode_window_and_sinks(window, sinks, Hq, Hkv, D):
    torch, w4 = cuda_or_skip()
    ends = [1, 4, 16, 37, 101, 240, 333]
    dev, host = _problem(torch, ends, [1] * len(ends), Hq, Hkv, D, 32, window + sinks)
    out = w4.kv4_attention(**dev, scratch=w4.kv4_attention_scratch(Hq, Hkv, D), window=window, sinks=sinks, max_new=1,
                           scale=0.11)
    _check(w4, out, host, 0.11, window, sinks)


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (9, 2)])
def test_few_new_tokens(Hq, Hkv, D, window, sinks):
    # several new tokens each, idle requests, one whose history is all new
    torch, w4 = cuda_or_skip()
    ends, new = [40, 5, 19, 7, 130, 3], [3, 5, 0, 2, 1, 0]
    dev, host = _problem(torch, ends, new, Hq, Hkv, D, 16, D + window)
    out = w4.kv4_attention(**dev, scratch=w4.kv4_attention_scratch(Hq, Hkv, D), window=window, sinks=sinks, max_new=5)
    _check(w4, out, host, D ** -0.5, window, sinks)


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 256), (4, 1, 128), (3, 3, 64), (6, 2, 128), (5, 1, 256)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 5), (20, 0)])
@pytest.mark.parametrize("bs", [16, 128])
def test_prompt_pieces(Hq, Hkv, D, window, sinks, bs):
    # pieces longer and shorter than a tile of queries, with and without a past
    torch, w4 = cuda_or_skip()
    ends, new = [150, 70, 257, 1, 0, 90], [150, 33, 130, 1, 0, 65]
    dev, host = _problem(torch, ends, new, Hq, Hkv, D, bs, bs + D + window)
    out = w4.kv4_attention(**dev, scratch=w4.kv4_attention_scratch(Hq, Hkv, D), window=window, sinks=sinks, max_new=150)
    _check(w4, out, host, D ** -0.5, window, sinks)


def test_max_new_is_a_hint():
    # the same answer, within the bound, from either kernel
    torch, w4 = cuda_or_skip()
    dev, host = _problem(torch, [150, 30], [100, 1], 4, 2, 128, 32, 3)
    for hint in (1, 100, 100000):
        out = w4.kv4_attention(**dev, scratch=w4.kv4_attention_scratch(4, 2, 128), max_new=hint)
        _check(w4, out, host, 128 ** -0.5)


@pytest.mark.parametrize("max_new", [1, 200])
def test_rows_that_see_nothing_are_zeros(max_new):
    # a request shorter than its new tokens, an empty one, rows past the last request
    torch, w4 = cuda_or_skip()
    dev, host = _problem(torch, [2, 0, 5], [4, 2, 1], 4, 2, 64, 16, 8, gap=3)
    out = torch.full((10, 4, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    w4.kv4_attention(**dev, scratch=w4.kv4_attention_scratch(4, 2, 64), out=out, max_new=max_new)
    _check(w4, out, host, 0.125)
    assert not out[:2].any() and not out[4:6].any() and not out[7:].any() and out[2:4].any()


@pytest.mark.parametrize("max_new", [1, 300])
def test_large_and_small_scores_scales_and_queries(max_new):
    # scores far apart, scales over four decades, queries of very different size
    torch, w4 = cuda_or_skip()
    ends, new = [90, 300], [1, 1] if max_new == 1 else [20, 130]
    dev, host = _problem(torch, ends, new, 8, 2, 128, 16, 21, spread=100.0)
    host[0][:, ::2] *= 2.0 ** 9
    host[0][:, 1::4] *= 2.0 ** -40
    dev["q"] = torch.tensor(host[0], device="cuda").to(torch.bfloat16)
    out = w4.kv4_attention(**dev, scratch=w4.kv4_attention_scratch(8, 2, 128), scale=0.002, max_new=max_new)
    _check(w4, out, host, 0.002)


@pytest.mark.parametrize("max_new", [1, 200])
def test_unknown_blocks_are_hidden(max_new):
    torch, w4 = cuda_or_skip()
    n = 1 if max_new == 1 else 20
    dev, host = _problem(torch, [100, 40], [n, n], 4, 2, 64, 16, 5)
    host[2][0, 2], host[2][1, 0] = -1, 10 ** 6
    dev["block_table"] = torch.tensor(host[2], dtype=torch.int32, device="cuda")
    out = w4.kv4_attention(**dev, scratch=w4.kv4_attention_scratch(4, 2, 64), max_new=max_new)
    torch.cuda.synchronize()
    assert w4.w4a16_check_device_error() == 6
    _check(w4, out, host, 0.125)


def test_long_split_rows_and_scratch_reuse():
    # lengths that many blocks share; repeated calls on one scratch agree bit for bit
    torch, w4 = cuda_or_skip()
    ends = [3000, 17, 900]
    dev, host = _problem(torch, ends, [1, 1, 1], 4, 2, 64, 64, 6)
    scratch = w4.kv4_attention_scratch(4, 2, 64)
    first = w4.kv4_attention(**dev, scratch=scratch, max_new=1)
    _check(w4, first, host, 0.125)
    for _ in range(20):
        again = w4.kv4_attention(**dev, scratch=scratch, max_new=1)
        assert torch.equal(first, again)


@pytest.mark.parametrize("max_new", [1, 100])
def test_strided_queries_other_stream_and_graph_replay(max_new):
    torch, w4 = cuda_or_skip()
    new = [1, 1] if max_new == 1 else [70, 9]
    dev, host = _problem(torch, [130, 75], new, 6, 2, 128, 32, 12)
    T = dev["q"].shape[0]
    wide = torch.zeros(T, 10 * 128 + 8, dtype=torch.bfloat16, device="cuda")
    wide[:, :768] = dev["q"].flatten(1)
    dev["q"] = wide[:, :768].unflatten(1, (6, 128))
    scratch = w4.kv4_attention_scratch(6, 2, 128)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        out = w4.kv4_attention(**dev, scratch=scratch, max_new=max_new)
    st.synchronize()
    _check(w4, out, host, 128 ** -0.5)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w4.kv4_attention(**dev, scratch=scratch, out=out, max_new=max_new)
    # the lengths are read by each replay
    shorter = [e - 40 for e in host[3]]
    dev["seq_lens"].copy_(torch.tensor(shorter, dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    _check(w4, out, (*host[:3], shorter, host[4]), 128 ** -0.5)


@pytest.mark.parametrize("Hq,Hkv,D,new", [(2, 1, 256, 1), (1, 1, 256, 1), (4, 1, 128, 1), (3, 1, 128, 1), (8, 1, 256, 1),
                                          (7, 1, 128, 1), (8, 1, 64, 1), (16, 1, 64, 1), (6, 1, 256, 2), (5, 1, 128, 3)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3)])
def test_many_requests(Hq, Hkv, D, new, window, sinks):
    # so many segments that each warp works alone; lengths that end and begin
    # inside a share, and a few that several warps share
    torch, w4 = cuda_or_skip()
    rng = np.random.default_rng(D + Hq)
    ends = rng.integers(1, 30, 320)
    ends[[5, 100, 319]] = 700, 333, 512
    ends[[6, 7, 200]] = 16, 17, 0
    n = np.minimum(rng.integers(1, new + 1, 320), np.maximum(ends, 1))
    n[[9, 10, 318]] = 0
    dev, host = _problem(torch, [int(e) for e in ends], [int(v) for v in n], Hq, Hkv, D, 16, D)
    scratch = w4.kv4_attention_scratch(Hq, Hkv, D)
    out = w4.kv4_attention(**dev, scratch=scratch, window=window, sinks=sinks, max_new=new)
    _check(w4, out, host, D ** -0.5, window, sinks)
    assert torch.equal(out, w4.kv4_attention(**dev, scratch=scratch, window=window, sinks=sinks, max_new=new))


@pytest.mark.parametrize("Hq,Hkv,D", [(2, 1, 256), (4, 1, 128), (16, 1, 64)])
def test_mixed_step_of_decodes_and_prompts(Hq, Hkv, D):
    # one call: requests for the prompt kernel beside many for the streaming one
    torch, w4 = cuda_or_skip()
    rng = np.random.default_rng(D)
    new = np.ones(90, int)
    new[[3, 50]] = 140, 61
    ends = new + rng.integers(0, 60, 90)
    ends[80] = 900
    dev, host = _problem(torch, [int(e) for e in ends], [int(v) for v in new], Hq, Hkv, D, 32, D + 1, gap=2)
    out = torch.full((int(new.sum()) + 2, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    w4.kv4_attention(**dev, scratch=w4.kv4_attention_scratch(Hq, Hkv, D), max_new=140, out=out)
    _check(w4, out, host, D ** -0.5)
