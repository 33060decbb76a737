"""The forms of the KV4 kernels that sizes choose: warps alone or together,
blocks of columns, pairs of CTAs for long pieces, several heads in flight."""
import numpy as np
import pytest

from tests import kv4_helpers as ref
from tests.gpu_helpers import cuda_or_skip
from tests.test_gpu_kv4_attention import _check, _problem
from tests.test_gpu_kv4_cache import _i32, _qkv, _rope_table

pytestmark = pytest.mark.gpu


def _check_far(w4, out, host, scale):
    """_check with what its bound leaves out, the smallest numbers of binary16:
    a weight times its scale is kept to 2^-25 where the row's largest such
    product lies above 2^6, so to 2^-31 of that.  A value is its scale times a
    whole number below 16, in units of which the largest scale of a cache tile
    of 16 tokens is at most twice what the tile is scaled by: 2^-26 of the
    largest product for each key, twice that because a weight is rounded again
    when the reference moves."""
    q, c, table, ends, cu = host
    want, tol = ref.attention(q, c, table, ends, cu, scale)
    G = q.shape[1] // c.H
    for b, end in enumerate(ends):
        n = int(cu[b + 1] - cu[b])
        slots = [int(table[b, j // c.bs]) * c.bs + j % c.bs for j in range(max(0, end))]
        for h in range(c.H):
            scales = np.array([c.raw[s // c.bs, h, s % c.bs // 16, 17 * c.D:].reshape(-1, 16, 4)[:, s % 16, :2].copy()
                               .view(np.float16).astype(np.float64).max() for s in slots])
            tiles = np.array([scales[j - j % 16:j - j % 16 + 16].max() for j in range(len(slots))])
            K = np.array([c.values(0, s, h) for s in slots])
            for i in range(n):
                p = end - n + i
                for r in range(G if p >= 0 else 0):
                    sc = scale * (K[:p + 1] @ q[int(cu[b]) + i, h * G + r])
                    w = np.exp(sc - sc.max())
                    tol[int(cu[b]) + i, h * G + r] += 2.0 ** -25 * (p + 1) * np.max(w / w.sum() * tiles[:p + 1])
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all() and (np.abs(got - want) <= tol).all()
    assert w4.w4a16_check_device_error() == 0


@pytest.mark.parametrize("T,Hq,Hkv,D,inter", [(1100, 32, 8, 128, True), (2700, 24, 8, 64, False), (1301, 13, 4, 256, False)])
def test_many_tokens_equal_few_at_a_time(T, Hq, Hkv, D, inter):
    # the same bits, whatever is in flight together
    torch, w4 = cuda_or_skip()
    (q, k, v), _ = _qkv(torch, T, Hq, Hkv, D, D)
    g = torch.Generator().manual_seed(D)
    cs = torch.tensor(_rope_table(90, D), device="cuda")
    pos = torch.randint(-1, 90, (T,), generator=g, dtype=torch.int32).cuda()
    wq, wk = ((1 + 0.1 * torch.randn(D, generator=g)).to(torch.bfloat16).cuda() for _ in range(2))
    slots = (torch.randperm(T + 40, generator=g)[:T] - 1).cuda()
    whole, parts = (w4.kv4_cache((T + 40) // 64 + 1, Hkv, 64, D) for _ in range(2))
    args = dict(q_weight=wq, k_weight=wk, cos_sin=cs, interleaved=inter)
    qa = w4.kv4_append(k, v, whole, slots, q=q, positions=pos, **args)
    qn, kn = w4.w4a16_qk_norm_rope(q, k, wq, wk, cs, pos, interleaved=inter)
    ka, va = w4.kv4_gather(whole, slots)
    for i in range(0, T, 200):
        s = slice(i, i + 200)
        assert torch.equal(qa[s], w4.kv4_append(k[s], v[s], parts, slots[s], q=q[s], positions=pos[s], **args))
        a, b = w4.w4a16_qk_norm_rope(q[s], k[s], wq, wk, cs, pos[s], interleaved=inter)
        assert torch.equal(qn[s], a) and torch.equal(kn[s], b)
        a, b = w4.kv4_gather(whole, slots[s])
        assert torch.equal(ka[s], a) and torch.equal(va[s], b)
    assert torch.equal(whole, parts)
    assert w4.w4a16_check_device_error() == 0


@pytest.mark.parametrize("Hq,Hkv,D,new", [(2, 1, 256, 1), (4, 1, 128, 1), (8, 1, 64, 1), (8, 1, 256, 1), (7, 1, 128, 1),
                                          (9, 1, 256, 1), (5, 1, 128, 3), (12, 1, 64, 1)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (20, 3)])
def test_a_warp_for_each_share(Hq, Hkv, D, new, window, sinks):
    torch, w4 = cuda_or_skip()
    rng = np.random.default_rng(D + Hq + window)
    ends = rng.integers(1, 30, 640)
    ends[[5, 100, 319]] = 700, 333, 512
    ends[[6, 7, 200]] = 16, 17, 0
    n = np.minimum(rng.integers(1, new + 1, 640), np.maximum(ends, 1))
    n[[9, 10, 639]] = 0
    dev, host = _problem(torch, [int(e) for e in ends], [int(v) for v in n], Hq, Hkv, D, 16, D)
    scratch = w4.kv4_attention_scratch(Hq, Hkv, D)
    out = w4.kv4_attention(**dev, scratch=scratch, window=window, sinks=sinks, max_new=new)
    _check(w4, out, host, D ** -0.5, window, sinks)
    assert torch.equal(out, w4.kv4_attention(**dev, scratch=scratch, window=window, sinks=sinks, max_new=new))


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 256), (8, 2, 128), (6, 2, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 20)])
def test_one_piece_in_many_blocks(Hq, Hkv, D, window, sinks):
    # one request with few heads: its rows are streamed in blocks of 16
    torch, w4 = cuda_or_skip()
    dev, host = _problem(torch, [143], [101], Hq, Hkv, D, 32, D)
    out = w4.kv4_attention(**dev, scratch=w4.kv4_attention_scratch(Hq, Hkv, D), window=window, sinks=sinks, max_new=101)
    _check(w4, out, host, D ** -0.5, window, sinks)


# enough heads that pieces of more than 16 rows leave the streaming form
PIECES = [(32, 16, 256), (32, 16, 128), (48, 24, 64)]
ENDS, NEW = [90, 300, 2, 0, 41, 130, 17, 129, 64], [20, 130, 40, 30, 41, 129, 17, 1, 33]


@pytest.mark.parametrize("Hq,Hkv,D", PIECES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (30, 5), (128, 128), (500, 1)])
def test_pieces_of_many_heads(Hq, Hkv, D, window, sinks):
    # rows that see nothing among them, and rows past the last request
    torch, w4 = cuda_or_skip()
    dev, host = _problem(torch, ENDS, NEW, Hq, Hkv, D, 16, D + window, gap=3)
    out = torch.full((sum(NEW) + 3, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    w4.kv4_attention(**dev, scratch=w4.kv4_attention_scratch(Hq, Hkv, D), window=window, sinks=sinks, out=out, max_new=130)
    _check(w4, out, host, D ** -0.5, window, sinks)
    assert not out[150:188].any() and not out[190:220].any() and not out[-3:].any()


@pytest.mark.parametrize("Hq,Hkv,D", PIECES)
@pytest.mark.parametrize("scale", [0.002, -0.002])
def test_pieces_with_scores_and_scales_far_apart(Hq, Hkv, D, scale):
    torch, w4 = cuda_or_skip()
    dev, host = _problem(torch, ENDS, NEW, Hq, Hkv, D, 64, 21, spread=100.0)
    host[0][:, ::2] *= 2.0 ** 9
    host[0][:, 1::4] *= 2.0 ** -40
    host[0][:, 3] = 0
    dev["q"] = torch.tensor(host[0], device="cuda").to(torch.bfloat16)
    out = w4.kv4_attention(**dev, scratch=w4.kv4_attention_scratch(Hq, Hkv, D), scale=scale, max_new=130)
    _check_far(w4, out, host, scale)


@pytest.mark.parametrize("Hq,Hkv,D", [(16, 8, 256), (8, 2, 128), (12, 3, 64)])
@pytest.mark.parametrize("new", [1, 3])
def test_tokens_with_scores_and_scales_far_apart(Hq, Hkv, D, new):
    # the same for the streaming form, rows that see one or two keys among them
    torch, w4 = cuda_or_skip()
    dev, host = _problem(torch, [3, 300, 4, 70], [new] * 4, Hq, Hkv, D, 16, 22, spread=100.0)
    host[0][:, ::2] *= 2.0 ** 9
    dev["q"] = torch.tensor(host[0], device="cuda").to(torch.bfloat16)
    out = w4.kv4_attention(**dev, scratch=w4.kv4_attention_scratch(Hq, Hkv, D), scale=0.002, max_new=new)
    _check_far(w4, out, host, 0.002)


@pytest.mark.parametrize("Hq,Hkv,D", PIECES)
def test_pieces_with_unknown_blocks(Hq, Hkv, D):
    torch, w4 = cuda_or_skip()
    dev, host = _problem(torch, ENDS, NEW, Hq, Hkv, D, 16, 5)
    host[2][0, 2], host[2][1, 0], host[2][1, 12], host[2][5, 7], host[2][6, :] = -1, 10 ** 6, -7, -1, -1
    dev["block_table"] = torch.tensor(host[2], dtype=torch.int32, device="cuda")
    out = w4.kv4_attention(**dev, scratch=w4.kv4_attention_scratch(Hq, Hkv, D), max_new=130)
    torch.cuda.synchronize()
    assert w4.w4a16_check_device_error() == 6
    _check(w4, out, host, D ** -0.5)


@pytest.mark.parametrize("Hq,Hkv,D", PIECES)
def test_pieces_repeat_bit_for_bit_in_a_graph(Hq, Hkv, D):
    torch, w4 = cuda_or_skip()
    dev, host = _problem(torch, ENDS, NEW, Hq, Hkv, D, 32, 7)
    T = dev["q"].shape[0]
    wide = torch.zeros(T, (Hq + 2) * D + 8, dtype=torch.bfloat16, device="cuda")
    wide[:, :Hq * D] = dev["q"].flatten(1)
    dev["q"] = wide[:, :Hq * D].unflatten(1, (Hq, D))
    scratch = w4.kv4_attention_scratch(Hq, Hkv, D)
    first = w4.kv4_attention(**dev, scratch=scratch, max_new=130)
    _check(w4, first, host, D ** -0.5)
    out = torch.empty_like(first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(4):
            w4.kv4_attention(**dev, scratch=scratch, out=out, max_new=130)
    for _ in range(5):
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, out)
    assert w4.w4a16_check_device_error() == 0


@pytest.mark.parametrize("Hq,Hkv,D", [(2, 1, 256), (4, 1, 128), (8, 1, 64), (16, 1, 128)])
def test_step_of_tokens_short_and_long_pieces(Hq, Hkv, D):
    # one call with requests for each of the three forms it launches
    torch, w4 = cuda_or_skip()
    rng = np.random.default_rng(D)
    new = rng.choice([0, 1, 1, 1, 2, 3], 90)
    new[[3, 50, 89]] = 300, 61, 170
    ends = new + rng.integers(0, 60, 90)
    ends[80] = 900
    dev, host = _problem(torch, [int(e) for e in ends], [int(v) for v in new], Hq, Hkv, D, 32, D + 1, gap=2)
    out = torch.full((int(new.sum()) + 2, Hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    w4.kv4_attention(**dev, scratch=w4.kv4_attention_scratch(Hq, Hkv, D), max_new=300, out=out)
    _check(w4, out, host, D ** -0.5)


@pytest.mark.parametrize("R,V", [(40, 32000), (300, 65536), (7, 65537), (1000, 700)])
@pytest.mark.parametrize("bf16", [True, False])
def test_sample_rows_alone_and_together(R, V, bf16):
    # a row's token does not depend on how many rows, and so how many blocks, there are
    torch, w4 = cuda_or_skip()
    g = torch.Generator(device="cuda").manual_seed(V)
    x = (torch.randn(R, V, device="cuda", generator=g) * 2).to(torch.bfloat16 if bf16 else torch.float32)
    u = torch.rand(R, device="cuda", generator=g)
    T = 0.3 + torch.rand(R, device="cuda", generator=g)
    k = torch.randint(0, 400, (R,), device="cuda", generator=g, dtype=torch.int32)
    p = 0.5 + 0.5 * torch.rand(R, device="cuda", generator=g)
    m = torch.rand(R, device="cuda", generator=g) * 0.01
    got = w4.w4a16_sample(x, u, T, k, p, m)
    for r in list(range(0, R, max(1, R // 6))) + [R - 1]:
        s = slice(r, r + 1)
        assert torch.equal(got[s], w4.w4a16_sample(x[s], u[s], T[s], k[s], p[s], m[s]))


@pytest.mark.parametrize("T", [3, 1400])
def test_append_with_queries_and_nothing_to_turn(T):
    # q comes out as it is, k and v are stored as without it
    torch, w4 = cuda_or_skip()
    (q, k, v), _ = _qkv(torch, T, 12, 4, 256, T)
    a, b = (w4.kv4_cache(T // 16 + 1, 4, 16, 256) for _ in range(2))
    slots = torch.arange(T, device="cuda")
    out = w4.kv4_append(k, v, a, slots, q=q)
    w4.kv4_append(k, v, b, slots)
    assert torch.equal(out, q) and torch.equal(a, b)
    assert w4.w4a16_check_device_error() == 0


def test_sample_settings_that_are_no_numbers_are_off():
    torch, w4 = cuda_or_skip()
    x = torch.randn(6, 3000, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    u = torch.linspace(0, 0.99, 6, device="cuda")
    nan = torch.full((6,), float("nan"), device="cuda")
    off = w4.w4a16_sample(x, u)
    assert torch.equal(off, w4.w4a16_sample(x, u, min_p=nan))
    assert torch.equal(off, w4.w4a16_sample(x, u, min_p=-torch.ones_like(u)))
    assert torch.equal(off, w4.w4a16_sample(x, u, top_p=nan))
