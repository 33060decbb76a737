"""Bounds of pages, the choice of pages by their scores and attention over
them.  The first two are defined step by step and match bit for bit; attention
is within the bound of kv4_helpers.attention."""
import numpy as np
import pytest

from tests import kv4_helpers as ref
from tests import kv4_long_helpers as lh
from tests.gpu_helpers import cuda_or_skip

pytestmark = pytest.mark.gpu

HEADS = [(16, 8, 256), (8, 1, 128), (4, 4, 64), (14, 2, 128), (16, 1, 64), (3, 3, 256), (5, 1, 256)]


@pytest.mark.parametrize("H,D,bs", [(8, 256, 16), (1, 256, 64), (3, 128, 32), (9, 64, 16), (2, 128, 256), (17, 64, 128)])
def test_bounds_of_the_pages_that_a_step_fills(H, D, bs):
    torch, w4 = cuda_or_skip()
    rng = np.random.default_rng(D + bs)
    blocks = 7
    c = lh.poisoned(blocks, H, bs, D, rng)
    full = [5, 0, 2]
    for page in full:
        for i in range(bs):
            lh.fill(c, rng, page * bs + i, 50.0)
    c.raw[2, 0, :, 16 * D:] = 0                     # a page of zeros
    slots = np.arange(5 * bs - 3, 6 * bs).tolist() + [-1, 2 * bs + bs - 1, 3 * bs, bs - 1, 6 * bs + bs - 2, -5]
    slots += [1 * bs] * 40 + [6 * bs]
    out = torch.full((blocks, H, 2 * D + 16), 77, dtype=torch.uint8, device="cuda")
    got = w4.kv4_bounds(torch.tensor(c.raw, device="cuda"), torch.tensor(slots, device="cuda"), out)
    assert got is out
    raw = out.cpu().numpy()
    for page in range(blocks):
        if page not in full:
            # (the last slot of page 4 is among them: its poison is no key of a cache)
            assert page == 4 or (raw[page] == 77).all()
            continue
        high, low, step = lh.bounds(c, page)
        assert np.array_equal(raw[page, :, :D].view(np.int8), high)
        assert np.array_equal(raw[page, :, D:2 * D].view(np.int8), low)
        assert np.array_equal(raw[page, :, 2 * D:].view(np.float32)[:, :D // 64], step)
    assert w4.w4a16_check_device_error() == 0
    again = out.clone()
    w4.kv4_bounds(torch.tensor(c.raw, device="cuda"), torch.tensor([blocks * bs, blocks * bs + bs - 1, -1], device="cuda"), out)
    torch.cuda.synchronize()
    assert w4.w4a16_check_device_error() == 6 and torch.equal(out, again)
    w4.kv4_bounds(torch.tensor(c.raw, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda"), out)
    assert torch.equal(out, again)


def test_bounds_hold_every_key():
    torch, w4 = cuda_or_skip()
    rng = np.random.default_rng(1)
    k = torch.tensor(rng.normal(0, 3, (64, 2, 128)) * np.exp(rng.normal(0, 2, (64, 2, 1))), device="cuda").to(torch.bfloat16)
    cache, slots = w4.kv4_cache(2, 2, 32, 128), torch.arange(64, device="cuda")
    w4.kv4_append(k, k, cache, slots)
    raw = w4.kv4_bounds(cache, slots, w4.kv4_bounds_buffer(2, 2, 128)).cpu().numpy()
    step = raw[..., 256:].view(np.float32)[..., :2].astype(np.float64).repeat(64, -1)
    high, low = raw[..., :128].view(np.int8) * step, raw[..., 128:256].view(np.int8) * step
    c = ref.Cache(2, 2, 32, 128)
    c.raw = cache.cpu().numpy()
    for slot in range(64):
        for h in range(2):
            v = c.values(0, slot, h)
            slack = 2.0 ** -23 * np.abs(v)      # of the quotient's rounding
            assert (v <= high[slot // 32, h] + slack).all() and (v >= low[slot // 32, h] - slack).all()


def _batch(torch, ends, new, Hq, Hkv, D, bs, seed, gap=0):
    rng = np.random.default_rng(seed)
    held = [max(0, -(-e // bs)) for e in ends]
    blocks = sum(held) + 2
    ids = rng.permutation(blocks)
    table = np.full((len(ends), max(held + [1]) + 1), -1)
    at = 0
    for b, n in enumerate(held):
        table[b, :n] = ids[at:at + n]
        at += n
    cu = np.concatenate([[0], np.cumsum(new)])
    q = ref.bf16(rng.normal(0, 1, (cu[-1] + gap, Hq, D)))
    raw = lh.packed_bounds(rng, blocks, Hkv, D)
    return q, raw, table, ends, cu


def _select(torch, w4, q, raw, table, ends, cu, bs, top, first, recent):
    i32 = dict(dtype=torch.int32, device="cuda")
    x = torch.tensor(q, device="cuda").to(torch.bfloat16)
    Hkv = raw.shape[1]
    tables = torch.full((len(q), Hkv, top), 12345, **i32)
    lens = torch.full((len(q),), 12345, **i32)
    got = w4.kv4_select(x, torch.tensor(raw, device="cuda"), torch.tensor(table, **i32), torch.tensor(ends, **i32),
                        torch.tensor(cu, **i32), bs, top, first=first, recent=recent, tables=tables, lens=lens)
    assert got[0] is tables and got[1] is lens
    return tables.cpu().numpy(), lens.cpu().numpy()


def _same(got, want):
    assert np.array_equal(got[1], want[1]), np.argwhere(got[1] != want[1])[:5]
    assert np.array_equal(got[0], want[0]), np.argwhere(got[0] != want[0])[:5]


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("top,first,recent", [(1, 0, 1), (2, 1, 1), (5, 0, 1), (7, 2, 3), (9, 3, 6), (40, 1, 2)])
def test_select(Hq, Hkv, D, top, first, recent):
    # fewer pages than `top`, as many, one more, many; several new tokens, idle requests, rows of none
    torch, w4 = cuda_or_skip()
    bs = 16
    ends = [1, 16, 17, top * bs, top * bs + 1, 640, 0, 1000, 333, 90]
    new = [1, 1, 3, 1, 1, 1, 0, 2, 19, 0]
    p = _batch(torch, ends, new, Hq, Hkv, D, bs, D + top, gap=2)
    _same(_select(torch, w4, *p, bs, top, first, recent), lh.select(*p, bs, top, first, recent))
    assert w4.w4a16_check_device_error() == 0


@pytest.mark.parametrize("Hq,Hkv,D", [(16, 16, 128), (24, 12, 64), (18, 9, 256), (6, 2, 128), (7, 1, 64), (8, 2, 256), (8, 1, 256),
                                      (18, 2, 64)])
@pytest.mark.parametrize("top,first,recent", [(1, 0, 1), (6, 1, 2), (33, 0, 4)])
def test_select_for_many_tokens(Hq, Hkv, D, top, first, recent):
    # tokens of a request together (and 9 query heads, which are too many for that); rows of no
    # request, requests that end inside such a team, scores that are equal
    torch, w4 = cuda_or_skip()
    ends, new = [700, 90, 30, 0, 401], [101, 1, 30, 0, 3]
    q, raw, table, ends, cu = _batch(torch, ends, new, Hq, Hkv, D, 16, D + top, gap=5)
    raw[table[0, 4:30]] = raw[table[0, 4]]
    q[20] = 0
    _same(_select(torch, w4, q, raw, table, ends, cu, 16, top, first, recent),
          lh.select(q, raw, table, ends, cu, 16, top, first, recent))
    assert w4.w4a16_check_device_error() == 0


@pytest.mark.parametrize("Hq,Hkv,D,T", [(40, 10, 64, 140), (48, 12, 256, 140), (70, 70, 64, 145), (34, 17, 256, 300), (96, 12, 128, 140),
                                        (64, 8, 64, 470), (30, 10, 256, 750), (24, 8, 128, 960)])
def test_select_for_so_many_tokens_that_a_wave_does_not_take_them(Hq, Hkv, D, T):
    torch, w4 = cuda_or_skip()
    p = _batch(torch, [T + 150, 130, 0], [T - 9, 7, 0], Hq, Hkv, D, 16, T, gap=2)
    _same(_select(torch, w4, *p, 16, 6, 1, 1), lh.select(*p, 16, 6, 1, 1))
    assert w4.w4a16_check_device_error() == 0


@pytest.mark.parametrize("Hq,Hkv,D", [(20, 20, 64), (30, 10, 128), (40, 20, 256)])
def test_select_for_many_requests(Hq, Hkv, D):
    # more requests than the order by length and a first wave of CTAs take
    torch, w4 = cuda_or_skip()
    rng = np.random.default_rng(D)
    ends = [int(e) for e in rng.integers(1, 500, 130)]
    q, raw, table, ends, cu = _batch(torch, ends, [1] * 130, Hq, Hkv, D, 16, D)
    _same(_select(torch, w4, q, raw, table, ends, cu, 16, 9, 1, 2), lh.select(q, raw, table, ends, cu, 16, 9, 1, 2))


def test_largest_whole_numbers():
    # every product at its largest, of either sign: the sums are exact in both forms
    torch, w4 = cuda_or_skip()
    for new in (1, 30):
        q, raw, table, ends, cu = _batch(torch, [1500], [new], 2, 1, 256, 16, new)
        q[:] = np.where(np.random.default_rng(1).random(q.shape) < 0.5, 1.0, -1.0)
        raw[..., :256] = np.int8(127).view(np.uint8)
        raw[..., 256:512] = np.random.default_rng(2).integers(-127, -120, raw[..., 256:512].shape).astype(np.int8).view(np.uint8)
        _same(_select(torch, w4, q, raw, table, ends, cu, 16, 20, 1, 1), lh.select(q, raw, table, ends, cu, 16, 20, 1, 1))


@pytest.mark.parametrize("Hq,Hkv,D,ends,bs", [(2, 1, 256, [70000], 16), (4, 1, 128, [40001, 3, 9000], 32), (2, 2, 64, [33000] * 5, 16)])
def test_select_of_many_pages(Hq, Hkv, D, ends, bs):
    torch, w4 = cuda_or_skip()
    p = _batch(torch, ends, [1] * len(ends), Hq, Hkv, D, bs, D)
    for top in (33, 700):
        _same(_select(torch, w4, *p, bs, top, 1, 2), lh.select(*p, bs, top, 1, 2))


def test_equal_scores_go_to_the_lower_page():
    # a query of zeros, pages that are the same, and scores one rounding apart
    torch, w4 = cuda_or_skip()
    q, raw, table, ends, cu = _batch(torch, [1600, 1600, 1600], [1, 1, 1], 4, 2, 128, 16, 9)
    q[0] = 0
    raw[table[1, 3:90]] = raw[table[1, 3]]
    raw[table[2, 1:99]] = raw[table[2, 1]]
    step = raw[table[2, 50:60], :, 256:].view(np.float32)
    raw[table[2, 50:60], :, 256:] = np.nextafter(step, np.float32(9)).view(np.uint8)
    for top in (4, 13, 60):
        _same(_select(torch, w4, q, raw, table, ends, cu, 16, top, 1, 1), lh.select(q, raw, table, ends, cu, 16, top, 1, 1))


def test_queries_of_any_size_and_no_numbers():
    torch, w4 = cuda_or_skip()
    q, raw, table, ends, cu = _batch(torch, [900] * 7, [1] * 7, 6, 2, 64, 16, 2)
    q[0, :, ::3], q[1, 0], q[2, 3, 5], q[3, :, 1], q[4] = np.nan, np.nan, np.inf, -np.inf, q[4] * 2.0 ** -130
    q[5] *= 2.0 ** 120
    q[6, :, ::2] = 0
    q = ref.bf16(q)
    q[0, :, ::3], q[1, 0] = np.nan, np.nan
    _same(_select(torch, w4, q, raw, table, ends, cu, 16, 9, 0, 1), lh.select(q, raw, table, ends, cu, 16, 9, 0, 1))
    assert w4.w4a16_check_device_error() == 0


def test_select_with_bad_lengths_and_ids():
    torch, w4 = cuda_or_skip()
    q, raw, table, ends, cu = _batch(torch, [500, 500, 500, 500], [1, 1, 2, 1], 4, 2, 128, 16, 3, gap=1)
    table[0, 7], table[1, 0], table[2, 31], table[1, 12] = -9, 10 ** 6, -1, raw.shape[0]
    ends = [500, 500, 500, table.shape[1] * 16 + 40]
    for top in (6, 30, 40):
        got = _select(torch, w4, q, raw, table, ends, cu, 16, top, 1, 1)
        _same(got, lh.select(q, raw, table, ends, cu, 16, top, 1, 1))
        assert w4.w4a16_check_device_error() == 6
    for bad in ([0, 1, 2, 4, 90], [0, 2, 1, 4, 5], [-4, 1, 2, 4, 5]):
        _select(torch, w4, q, raw, table, ends, np.array(bad), 16, 6, 1, 1)
        assert w4.w4a16_check_device_error() == 6
    _same(_select(torch, w4, q, raw, table, [-1, 500, 0, 500], cu, 16, 6, 1, 1)[1:] * 2,
          lh.select(q, raw, table, [-1, 500, 0, 500], cu, 16, 6, 1, 1)[1:] * 2)
    assert w4.w4a16_check_device_error() == 6


def _tables(rng, c, T, top, lens):
    """Random pages for each token and head, filled as far as lens says."""
    tables = np.full((T, c.H, top), -1)
    for t in range(T):
        for h in range(c.H):
            n = -(-max(0, int(lens[t])) // c.bs)
            tables[t, h, :n] = rng.permutation(c.blocks)[:n]
    return tables


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("bs", [16, 64])
def test_sparse_attention(Hq, Hkv, D, bs):
    torch, w4 = cuda_or_skip()
    rng = np.random.default_rng(D + bs)
    c = ref.Cache(12, Hkv, bs, D)
    for slot in range(12 * bs):
        lh.fill(c, rng, slot)
    lens = np.array([1, 15, 16, 17, 0, bs, bs + 1, 5 * bs - 3, 5 * bs, 33])
    tables = _tables(rng, c, len(lens), 5, lens)
    q = ref.bf16(rng.normal(0, 1, (len(lens), Hq, D)))
    i32 = dict(dtype=torch.int32, device="cuda")
    x, raw = torch.tensor(q, device="cuda").to(torch.bfloat16), torch.tensor(c.raw, device="cuda")
    scratch = w4.kv4_attention_scratch(Hq, Hkv, D)
    out = torch.full_like(x, float("nan"))
    got = w4.kv4_sparse_attention(x, raw, torch.tensor(tables, **i32), torch.tensor(lens, **i32), scratch, out=out, scale=0.1)
    assert got is out
    want, tol = lh.sparse(q, c, tables, lens, 0.1)
    lh.check(w4, out, want, tol)
    # pages and lengths that are not there
    tables[7, :, 1], tables[8, 0, 0], lens[3] = -1, 99, -2
    out = w4.kv4_sparse_attention(x, raw, torch.tensor(tables, **i32), torch.tensor(lens, **i32), scratch, scale=0.1)
    torch.cuda.synchronize()
    assert w4.w4a16_check_device_error() == 6
    want, tol = lh.sparse(q, c, tables, lens, 0.1)
    lh.check(w4, out, want, tol)
    lens[3] = 5 * bs + 7        # past the table
    out = w4.kv4_sparse_attention(x, raw, torch.tensor(tables, **i32), torch.tensor(lens, **i32), scratch, scale=0.1)
    torch.cuda.synchronize()
    assert w4.w4a16_check_device_error() == 6


@pytest.mark.parametrize("T,Hq,Hkv,D", [(1, 8, 1, 128), (3, 8, 1, 256), (7, 24, 1, 64), (9, 20, 10, 64), (14, 28, 4, 128), (40, 8, 4, 64),
                                        (30, 16, 8, 64)])
@pytest.mark.parametrize("even", [True, False])
def test_sparse_attention_with_rows_split_into_parts(T, Hq, Hkv, D, even):
    # as many tiles for every token, or some of none and some of one beside long ones; fewer and
    # more segments than CTAs
    torch, w4 = cuda_or_skip()
    rng = np.random.default_rng(T * D)
    c = ref.Cache(40, Hkv, 16, D)
    for slot in range(640):
        lh.fill(c, rng, slot)
    lens = np.full(T, 630) if even else np.where(rng.random(T) < 0.3, rng.integers(0, 3, T), rng.integers(3, 641, T))
    tables = _tables(rng, c, T, 40, lens)
    q = ref.bf16(rng.normal(0, 1, (T, Hq, D)))
    i32 = dict(dtype=torch.int32, device="cuda")
    x, raw = torch.tensor(q, device="cuda").to(torch.bfloat16), torch.tensor(c.raw, device="cuda")
    scratch = w4.kv4_attention_scratch(Hq, Hkv, D)
    want, tol = lh.sparse(q, c, tables, lens, D ** -0.5)
    for _ in range(2):
        lh.check(w4, w4.kv4_sparse_attention(x, raw, torch.tensor(tables, **i32), torch.tensor(lens, **i32), scratch), want, tol)


def test_sparse_attention_of_more_tokens_than_a_launch_takes():
    torch, w4 = cuda_or_skip()
    rng = np.random.default_rng(8)
    c = ref.Cache(6, 1, 16, 64)
    for slot in range(96):
        lh.fill(c, rng, slot)
    T = 4096 + 37
    lens = rng.integers(0, 33, T)
    tables = _tables(rng, c, T, 2, lens)
    q = ref.bf16(rng.normal(0, 1, (T, 2, 64)))
    i32 = dict(dtype=torch.int32, device="cuda")
    wide = torch.zeros(T, 200, dtype=torch.bfloat16, device="cuda")
    wide[:, 8:136] = torch.tensor(q, device="cuda").to(torch.bfloat16).flatten(1)
    out = w4.kv4_sparse_attention(wide[:, 8:136].unflatten(1, (2, 64)), torch.tensor(c.raw, device="cuda"), torch.tensor(tables, **i32),
                                  torch.tensor(lens, **i32), w4.kv4_attention_scratch(2, 1, 64))
    some = np.r_[0:50, 4060:T]
    want, tol = lh.sparse(q[some], c, tables[some], lens[some], 64 ** -0.5)
    lh.check(w4, out[torch.tensor(some, device="cuda")], want, tol)


@pytest.mark.parametrize("Hq,Hkv,D", [(16, 8, 256), (8, 2, 128)])
def test_a_step_over_selected_pages(Hq, Hkv, D):
    # a prompt, then steps of one token through append, bounds, select and attention in one captured graph
    torch, w4 = cuda_or_skip()
    g = torch.Generator("cuda").manual_seed(D)
    B, bs, top = 3, 16, 6
    i32 = dict(dtype=torch.int32, device="cuda")
    cache, bounds = w4.kv4_cache(B * 20, Hkv, bs, D), w4.kv4_bounds_buffer(B * 20, Hkv, D)
    scratch = w4.kv4_attention_scratch(Hq, Hkv, D)
    table, free = torch.full((B, 20), -1, **i32), torch.randperm(B * 20, device="cuda", generator=g).to(torch.int32)
    ctx, ones = torch.zeros(B, **i32), torch.ones(B, **i32)
    rows = lambda n, h: torch.randn(n, h, D, device="cuda", generator=g).to(torch.bfloat16)
    prompt = torch.tensor([150, 95, 30], **i32)
    plan = w4.kv4_plan(ctx, prompt, table, free, bs, num_tokens=275)
    w4.kv4_append(rows(275, Hkv), rows(275, Hkv), cache, plan.slots)
    w4.kv4_bounds(cache, plan.slots, bounds)
    ctx.copy_(plan.seq_lens)
    free = free[int(plan.taken):].clone()
    q, k, v = rows(B, Hq), rows(B, Hkv), rows(B, Hkv)
    seen = {}

    def step():
        plan = w4.kv4_plan(ctx, ones, table, free, bs, num_tokens=B)
        w4.kv4_append(k, v, cache, plan.slots)
        w4.kv4_bounds(cache, plan.slots, bounds)
        tables, lens = w4.kv4_select(q, bounds, table, plan.seq_lens, plan.cu_new, bs, top, first=1, recent=2)
        out = w4.kv4_sparse_attention(q, cache, tables, lens, scratch)
        ctx.copy_(plan.seq_lens)
        free.copy_(free[(torch.arange(free.numel(), device="cuda") + plan.taken) % free.numel()])
        seen.update(tables=tables, lens=lens, out=out, ends=plan.seq_lens, cu=plan.cu_new)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(20):
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, device="cuda", generator=g))
        graph.replay()
        raw, ends, cu = bounds.cpu().numpy(), seen["ends"].cpu().numpy(), seen["cu"].cpu().numpy()
        host_q, host_table = q.double().cpu().numpy(), table.cpu().numpy()
        tables, lens = seen["tables"].cpu().numpy(), seen["lens"].cpu().numpy()
        _same((tables, lens), lh.select(host_q, raw, host_table, ends, cu, bs, top, 1, 2))
        c = ref.Cache(B * 20, Hkv, bs, D)
        c.raw = cache.cpu().numpy()
        want, tol = lh.sparse(host_q, c, tables, lens, D ** -0.5)
        lh.check(w4, seen["out"], want, tol)
    # the bounds of every full page are those of its keys
    for b in range(B):
        for i in range(int(ends[b]) // bs):
            high, low, unit = lh.bounds(c, int(host_table[b, i]))
            page = raw[host_table[b, i]]
            assert np.array_equal(page[:, :D].view(np.int8), high) and np.array_equal(page[:, D:2 * D].view(np.int8), low)
            assert np.array_equal(page[:, 2 * D:].view(np.float32)[:, :D // 64], unit)


def test_few_pages_are_all_of_attention():
    # where every page is taken the result is kv4_attention's bit for bit
    torch, w4 = cuda_or_skip()
    dev, host = lh.grouped(torch, [(0, [(40, 1), (9, 1), (100, 1)])], 8, 4, 128, 16, 11)
    scratch = w4.kv4_attention_scratch(8, 4, 128)
    bounds = w4.kv4_bounds_buffer(dev["cache"].shape[0], 4, 128)
    tables, lens = w4.kv4_select(dev["q"], bounds, dev["block_table"], dev["seq_lens"], dev["cu_new"], 16, 8)
    assert lens.tolist() == [41, 10, 101]
    a = w4.kv4_sparse_attention(dev["q"], dev["cache"], tables, lens, scratch)
    b = w4.kv4_attention(dev["q"], dev["cache"], dev["block_table"], dev["seq_lens"], dev["cu_new"], scratch, max_new=1)
    want, tol = ref.attention(*host, 128 ** -0.5)
    lh.check(w4, a, want, tol)
    assert torch.equal(a, b)


@pytest.mark.parametrize("T,D", [(3, 256), (700, 64)])
def test_copies_that_never_come(T, D):
    # test-only injection, as in the waits of kv4_attention
    torch, w4 = cuda_or_skip()
    rng = np.random.default_rng(D)
    c = ref.Cache(9, 2, 16, D)
    for slot in range(9 * 16):
        lh.fill(c, rng, slot)
    lens = rng.integers(1, 65, T)
    tables = _tables(rng, c, T, 4, lens)
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.tensor(ref.bf16(rng.normal(0, 1, (T, 4, D))), device="cuda").to(torch.bfloat16)
    args = (q, torch.tensor(c.raw, device="cuda"), torch.tensor(tables, **i32), torch.tensor(lens, **i32), w4.kv4_attention_scratch(4, 2, D))
    first = w4.kv4_sparse_attention(*args)
    w4.w4a16_debug_inject(w4.INJECT_STALL_PIPELINE)
    try:
        w4.kv4_sparse_attention(*args)
        status = w4.w4a16_check_device_error()
    finally:
        w4.w4a16_debug_inject(0)
    assert status == 5
    for _ in range(3):
        assert torch.equal(first, w4.kv4_sparse_attention(*args))
    assert w4.w4a16_check_device_error() == 0


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 2)])
@pytest.mark.parametrize("new", [1, 30])
def test_steps_that_are_not_finite(Hq, Hkv, new):
    # products of 0 and infinity, sums of infinities of both signs, NaN
    torch, w4 = cuda_or_skip()
    rng = np.random.default_rng(new)
    q, raw, table, ends, cu = _batch(torch, [1500], [new], Hq, Hkv, 256, 16, new)
    steps = raw[..., 512:].view(np.float32)
    for value in (np.nan, np.inf):
        steps[rng.random(steps.shape) < 0.1] = value
    _same(_select(torch, w4, q, raw, table, ends, cu, 16, 20, 1, 1), lh.select(q, raw, table, ends, cu, 16, 20, 1, 1))


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 2)])
@pytest.mark.parametrize("new", [1, 30])
def test_scores_that_vanish(Hq, Hkv, new):
    # zeros of either sign are equal scores
    torch, w4 = cuda_or_skip()
    q, raw, table, ends, cu = _batch(torch, [1500], [new], Hq, Hkv, 128, 16, new)
    q *= 2.0 ** -110
    raw[..., 256:].view(np.float32)[...] *= np.float32(2.0 ** -40)
    _same(_select(torch, w4, q, raw, table, ends, cu, 16, 20, 1, 1), lh.select(q, raw, table, ends, cu, 16, 20, 1, 1))
