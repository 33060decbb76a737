"""Edges of the KV4 operators: what lies outside a window, lengths out of
range, references that move far, values that are no numbers."""
import numpy as np
import pytest

from tests import kv4_helpers as ref
from tests.gpu_helpers import cuda_or_skip
from tests.test_gpu_kv4_attention import _check, _problem
from tests.test_gpu_kv4_cache import _i32, _qkv

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 16, 256), (32, 16, 128), (48, 24, 64)])
@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("window,sinks", [(1, 0), (30, 0), (30, 5), (100, 20)])
@pytest.mark.parametrize("new", [1, 20, 130])
def test_pages_that_no_query_sees_may_be_gone(Hq, Hkv, D, bs, window, sinks, new):
    # given back by the caller, or given to somebody else (the spare pages hold NaN
    # and infinite parameters): the same bits, and no error
    torch, w4 = cuda_or_skip()
    ends = [300, 190, 131, 20]
    n = [min(new, e) for e in ends]
    dev, host = _problem(torch, ends, n, Hq, Hkv, D, bs, D + window)
    kw = dict(scratch=w4.kv4_attention_scratch(Hq, Hkv, D), window=window, sinks=sinks, max_new=new)
    whole = w4.kv4_attention(**dev, **kw)
    gone, spare = [], (set(range(host[1].blocks)) - set(host[2].ravel().tolist())).pop()
    for b, (e, m) in enumerate(zip(ends, n)):
        first = max(0, e - m - window + 1)            # the first key in the first query's window
        for i in range(host[2].shape[1]):
            if i * bs >= sinks and (i + 1) * bs <= first:
                gone.append((b, i))
    assert gone
    for page in (-1, spare):
        for at in gone:
            host[2][at] = page
        dev["block_table"] = _i32(torch, host[2])
        out = w4.kv4_attention(**dev, **kw)
        torch.cuda.synchronize()
        assert w4.w4a16_check_device_error() == 0
        assert torch.equal(out, whole)


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 16, 256), (32, 16, 128), (48, 24, 64)])
@pytest.mark.parametrize("new", [1, 140])
@pytest.mark.parametrize("jump", [20, 26, 27, 32, 40])
@pytest.mark.parametrize("at", [64, 97, 130])
def test_weights_before_a_far_move_of_the_reference_count(Hq, Hkv, D, new, jump, at):
    # Keys of log2 score 0, then 7, then one of `jump` whose values are all zero:
    # the output is what the others add.  In the bound: the result's rounding
    # (2^-8), weights and values rounded to binary16 (2^-11 each), the scores'
    # binary32 steps (2^-16), and weights kept to 2^-30 of the largest.
    torch, w4 = cuda_or_skip()
    rng = np.random.default_rng(jump)
    end, bs = 160, 16
    c = ref.Cache(end // bs, Hkv, bs, D)
    score = np.zeros(end)
    score[32:64], score[at] = 7, jump
    one, zero = np.full(D // 64, 1.0, np.float16), rng.integers(1, 15, (end, Hkv, D // 64))
    V = np.zeros((end, Hkv, D))
    for j in range(end):
        for h in range(Hkv):
            kc = np.zeros(D, np.uint8)
            kc[0] = score[j] > 0
            c.put(0, j, h, kc, one * max(score[j], 1), one * 0)
            z = np.repeat(zero[j, h], 64)
            codes = z if j == at else rng.integers(0, 16, D)
            c.put(1, j, h, codes.astype(np.uint8), one, zero[j, h].astype(np.float16))
            V[j, h] = codes - z
    q = torch.zeros(new, Hq, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 1
    ln2 = float(np.float32(np.log(2)))
    out = w4.kv4_attention(q, torch.tensor(c.raw, device="cuda"), _i32(torch, [list(range(end // bs))]),
                           _i32(torch, [end]), _i32(torch, [0, new]), w4.kv4_attention_scratch(Hq, Hkv, D), scale=ln2,
                           max_new=new).double().cpu().numpy()
    for t in range(new):
        see = end - new + t + 1
        w = np.exp(ln2 * (score[:see] - score[:see].max()))
        w /= w.sum()
        o, size = np.einsum("j,jhd->hd", w, V[:see]), np.einsum("j,jhd->hd", w, np.abs(V[:see]))
        tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -10 + 2.0 ** -16) * (1 + 2.0 ** -8) * size + \
            2.0 ** -30 * w.max() * np.abs(V[:see]).sum(0)
        got = out[t].reshape(Hkv, Hq // Hkv, D)
        assert (np.abs(got - o[:, None]) <= tol[:, None]).all(), t
    assert w4.w4a16_check_device_error() == 0


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 16, 256), (32, 16, 128), (48, 24, 64)])
@pytest.mark.parametrize("new", [1, 90])
def test_scores_of_keys_at_the_middle_between_two_numbers(Hq, Hkv, D, new):
    # 3 * 1370 and 3 * 1374 lie half a unit of binary16 from its numbers, the first
    # is rounded up and the second down: each by 2^-11 of itself, the most there is.
    # Scores of 2055 and 2061, so the smaller weights grow by up to exp(2 * 2^-11 *
    # 2061) where keys are rounded; the streaming kernel takes them as they are.
    torch, w4 = cuda_or_skip()
    end, bs = 100, 16
    c = ref.Cache(-(-end // bs), Hkv, bs, D)
    one, rng = np.ones(D // 64, np.float16), np.random.default_rng(D)
    V = np.zeros((end, Hkv, D))
    for j in range(end):
        for h in range(Hkv):
            kc = np.zeros(D, np.uint8)
            kc[0] = 3
            c.put(0, j, h, kc, one * np.float16((1374 if j % 2 else 1370) / 1024), one * 0)
            V[j, h] = 0 if j % 2 else rng.integers(0, 16, D)
            c.put(1, j, h, V[j, h].astype(np.uint8), one, one * 0)
    score = 512.0 * 3 / 1024 * np.where(np.arange(end) % 2, 1374, 1370)
    q = torch.zeros(new, Hq, D, dtype=torch.bfloat16, device="cuda")
    q[..., 0] = 512
    out = w4.kv4_attention(q, torch.tensor(c.raw, device="cuda"), _i32(torch, [list(range(-(-end // bs)))]),
                           _i32(torch, [end]), _i32(torch, [0, new]), w4.kv4_attention_scratch(Hq, Hkv, D), scale=1.0,
                           max_new=new).double().cpu().numpy()
    e = ((2.0 ** -11 if new > 1 else 0) + 2.0 ** -20) * score.max()
    for t in range(new):
        see = end - new + t + 1
        w = np.exp(score[:see] - score[:see].max())
        o = np.einsum("j,jhd->hd", w / w.sum(), V[:see])[:, None]
        got = out[t].reshape(Hkv, Hq // Hkv, D)
        # (values and weights to binary16, the result to BF16)
        assert (np.abs(got - o) <= (np.expm1(2 * e) + 2.0 ** -10 + 2.0 ** -8 * np.exp(2 * e)) * o + 1e-30).all()
    assert w4.w4a16_check_device_error() == 0


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 16, 256), (4, 2, 128), (48, 24, 64)])
@pytest.mark.parametrize("new", [1, 130])
def test_lengths_out_of_range_are_reported(Hq, Hkv, D, new):
    torch, w4 = cuda_or_skip()
    ends, n = [170, 140, 135], [new] * 3
    dev, host = _problem(torch, ends, n, Hq, Hkv, D, 16, D)
    width = host[2].shape[1]
    kw = dict(scratch=w4.kv4_attention_scratch(Hq, Hkv, D), max_new=new)
    whole = w4.kv4_attention(**dev, **kw)
    torch.cuda.synchronize()
    assert w4.w4a16_check_device_error() == 0

    def status(lens=ends, cu=(0, new, 2 * new, 3 * new), T=3 * new):
        args = dict(dev, seq_lens=_i32(torch, lens), cu_new=_i32(torch, cu), q=dev["q"][:T])
        out = w4.kv4_attention(**args, **kw)
        torch.cuda.synchronize()
        return w4.w4a16_check_device_error(), out

    full = width * 16
    assert status()[0] == 0
    assert status([170, full + 1, 135])[0] == 6
    assert status([170, 140, 2 ** 31 - 1])[0] == 6
    assert status([-1, 140, 135])[0] == 6
    # a request without new tokens is not looked at
    for unused in (-5, 2 ** 31 - 1):
        assert status([170, unused, 135], (0, new, new, 2 * new), 2 * new)[0] == 0
    # fewer tokens in all than new ones: rows that see nothing, no error
    assert status([0, 140, 135])[0] == 0
    assert status(cu=(0, new, 2 * new, 3 * new + 1))[0] == 6
    assert status(cu=(0, 2 * new, new, 3 * new))[0] == 6
    assert status(cu=(-1, new, 2 * new, 3 * new))[0] == 6
    assert status()[0] == 0 and torch.equal(status()[1], whole)


@pytest.mark.parametrize("T,Hkv,D", [(5, 2, 128), (9, 1, 64), (3, 2, 256), (2000, 8, 256), (1200, 16, 128), (5000, 8, 64)])
@pytest.mark.parametrize("norm", [False, True])
def test_nan_keys_and_values_count_as_zero(T, Hkv, D, norm):
    torch, w4 = cuda_or_skip()
    (q, k, v), _ = _qkv(torch, T, Hkv, Hkv, D, T)
    g = torch.Generator(device="cuda").manual_seed(D)
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda") if norm else None
    slots = torch.arange(T, device="cuda")
    a, b = (w4.kv4_cache(T // 16 + 1, Hkv, 16, D) for _ in range(2))
    nan = torch.rand(v.shape, device="cuda", generator=g) < 0.02
    nan[0, 0, :64] = True                                    # a whole group
    v[1, 0, 3], v[2, 0, 5] = 3e38, float("inf")              # scales at their limit
    nan[1, 0, 4] = nan[2, 0, 4] = True
    sign = torch.where(torch.rand(v.shape, device="cuda", generator=g) < 0.5, -1.0, 1.0).to(torch.bfloat16)
    bad = torch.full_like(sign, float("nan")).copysign(sign)
    if norm:      # one NaN makes its head's norm NaN: all of it counts as zero
        head = nan[..., :1] & (torch.arange(T, device="cuda") % 3 == 0)[:, None, None]
        k1, k0 = torch.where(head & (torch.arange(D, device="cuda") == 7), bad, k), torch.where(head, 0, k)
    else:
        k1, k0 = torch.where(nan, bad, k), torch.where(nan, 0, k)
    w4.kv4_append(k1, torch.where(nan, bad, v), a, slots, q=q if norm else None, k_weight=w)
    w4.kv4_append(k0, torch.where(nan, 0, v), b, slots, q=q if norm else None, k_weight=w)
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    assert torch.isfinite(w4.kv4_gather(a, slots)[1].float()).all()
    assert w4.w4a16_check_device_error() == 0


def test_flags_that_have_no_truth_value_are_refused():
    torch, w4 = cuda_or_skip()
    (q, k, v), _ = _qkv(torch, 2, 2, 2, 64, 1)
    two = np.array([True, False])
    with pytest.raises(ValueError, match="truth value"):
        w4.w4a16_qk_norm_rope(q, k, None, None, None, None, interleaved=two)
    with pytest.raises(ValueError, match="truth value"):
        w4.kv4_append(k, v, w4.kv4_cache(1, 2, 16, 64), torch.arange(2, device="cuda"), interleaved=two)


@pytest.mark.parametrize("Hq,Hkv,D", [(32, 16, 256), (32, 16, 128), (48, 24, 64)])
def test_any_upper_bound_of_new_tokens_chooses_alike(Hq, Hkv, D):
    # no more than there are rows of q: the same bits for bounds past that
    torch, w4 = cuda_or_skip()
    dev, host = _problem(torch, [140, 60], [130, 30], Hq, Hkv, D, 16, D)
    kw = dict(scratch=w4.kv4_attention_scratch(Hq, Hkv, D))
    want = w4.kv4_attention(**dev, **kw, max_new=160)
    for most in (1 << 20, 1 << 31, 1 << 62, (1 << 63) - 1):
        assert torch.equal(want, w4.kv4_attention(**dev, **kw, max_new=most))


@pytest.mark.parametrize("requests,Hq,Hkv,D", [(700, 4, 1, 256), (700, 4, 1, 128), (700, 4, 2, 64), (4096, 4, 1, 256),
                                               (4096, 8, 1, 64)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (30, 2)])
def test_pieces_of_many_requests(requests, Hq, Hkv, D, window, sinks):
    # more than are put in order of their length, and as many as a call takes
    torch, w4 = cuda_or_skip()
    rng = np.random.default_rng(requests + D)
    g = torch.Generator(device="cuda").manual_seed(D)
    new = rng.integers(0, 9, requests)
    new[[3, requests - 1]] = 150, 70
    ends = new + rng.integers(0, 90, requests)
    held = -(-ends // 16)
    blocks = int(held.sum())
    cache = torch.randint(0, 256, (blocks, Hkv, 1, 18 * D), device="cuda", generator=g, dtype=torch.uint8)
    shape = (blocks, Hkv, 1, D // 2)
    par = torch.stack([(0.05 + 0.2 * torch.rand(shape, device="cuda", generator=g)).half(),
                       torch.randint(0, 16, shape, device="cuda", generator=g).half()], -1)
    cache[..., 16 * D:] = par.flatten(-2).view(torch.uint8)
    ids = rng.permutation(blocks)
    table = np.full((requests, int(held.max())), -1)
    table[np.arange(table.shape[1])[None] < held[:, None]] = ids
    cu = np.concatenate([[0], np.cumsum(new)])
    q = torch.randn(int(cu[-1]), Hq, D, device="cuda", generator=g).to(torch.bfloat16)
    out = w4.kv4_attention(q, cache, _i32(torch, table), _i32(torch, ends), _i32(torch, cu),
                           w4.kv4_attention_scratch(Hq, Hkv, D), window=window, sinks=sinks, max_new=150)
    # some of them against the reference
    pick = sorted({0, 1, 3, requests - 1, *rng.integers(0, requests, 25).tolist()})
    c = ref.Cache(blocks, Hkv, 16, D)
    c.raw = cache.cpu().numpy()
    rows = np.concatenate([np.arange(cu[b], cu[b + 1]) for b in pick])
    host = (q.double().cpu().numpy()[rows], c, table[pick], ends[pick], np.concatenate([[0], np.cumsum(new[pick])]))
    _check(w4, out[torch.tensor(rows, device="cuda")], host, D ** -0.5, window, sinks)
    assert torch.isfinite(out).all()
