"""Attention of requests that share a prefix, against binary64 over each
request's whole context, with the error bound of kv4_helpers.attention (what the
join adds, a binary32 rounding of each part, is within its 2^-16)."""
import numpy as np
import pytest

from tests import kv4_helpers as ref
from tests import kv4_long_helpers as lh
from tests.gpu_helpers import cuda_or_skip
from tests.test_gpu_kv4_forms import _check_far

pytestmark = pytest.mark.gpu

HEADS = [(16, 8, 256), (8, 1, 128), (4, 4, 64), (14, 2, 128), (16, 1, 64), (3, 3, 256)]
# (prefix, [(past, new) of each request]) of each group
SMALL = [(48, [(0, 1), (5, 1), (17, 1)]),          # ends and lengths around a tile
         (16, [(1, 1), (0, 2)]),
         (32, [(3, 1)]),                           # a group of one
         (0, [(20, 1), (7, 3)]),                   # nothing shared
         (64, [(0, 0), (9, 1), (0, 0), (31, 4)])]  # some sit the step out


def _run(w4, dev, scratch=None, **kw):
    return w4.kv4_prefix_attention(**dev, scratch=lh.scratch(w4, dev) if scratch is None else scratch, **kw)


def _check(w4, out, host, scale):
    want, tol = ref.attention(*host, scale)
    lh.check(w4, out, want, tol)


@pytest.mark.parametrize("Hq,Hkv,D", HEADS)
@pytest.mark.parametrize("bs", [16, 32])
def test_small_groups(Hq, Hkv, D, bs):
    torch, w4 = cuda_or_skip()
    dev, host = lh.grouped(torch, SMALL, Hq, Hkv, D, bs, Hq * D + bs, gap=2)
    out = torch.full_like(dev["q"], float("nan"))
    _run(w4, dev, out=out, max_new=4, max_group=5)
    _check(w4, out, host, D ** -0.5)


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 256), (8, 2, 128), (4, 2, 64), (10, 1, 256), (9, 3, 128)])
def test_many_rows_behind_one_prefix(Hq, Hkv, D):
    # more rows than a tile of queries has, prefixes that end inside a tile of keys
    torch, w4 = cuda_or_skip()
    rng = np.random.default_rng(D)
    groups = [(208, [(int(rng.integers(0, 40)), 1) for _ in range(150)]),
              (400, [(int(rng.integers(0, 9)), int(rng.integers(1, 4))) for _ in range(20)])]
    dev, host = lh.grouped(torch, groups, Hq, Hkv, D, 16, D)
    scratch = lh.scratch(w4, dev)
    out = _run(w4, dev, scratch=scratch, max_new=3, max_group=150)
    _check(w4, out, host, D ** -0.5)
    assert torch.equal(out, _run(w4, dev, scratch=scratch, max_new=3, max_group=150))


@pytest.mark.parametrize("Hq,Hkv,D", [(4, 2, 256), (4, 1, 128), (6, 2, 64)])
def test_prompts_behind_one_prefix(Hq, Hkv, D):
    # pieces of many new tokens, beside requests of one
    torch, w4 = cuda_or_skip()
    groups = [(128, [(0, 150), (3, 33), (0, 1), (0, 70)]), (64, [(0, 5), (40, 1)]), (16, [(0, 140)])]
    dev, host = lh.grouped(torch, groups, Hq, Hkv, D, 32, D, gap=1)
    for widest in (254, None, 1):       # bounds are hints
        out = _run(w4, dev, max_new=150 if widest else None, max_group=widest)
        _check(w4, out, host, D ** -0.5)


@pytest.mark.parametrize("Hq,Hkv,D", [(16, 8, 256), (8, 2, 128), (6, 2, 64)])
@pytest.mark.parametrize("rows", [2, 90])
def test_scores_and_scales_far_apart(Hq, Hkv, D, rows):
    # the parts of a row have maxima far from each other
    torch, w4 = cuda_or_skip()
    dev, host = lh.grouped(torch, [(160, [(i % 30, 1) for i in range(rows)])], Hq, Hkv, D, 16, 3, spread=100.0)
    host[0][:, ::2] *= 2.0 ** 9
    host[0][:, 1::4] *= 2.0 ** -40
    host[0][1] = 0
    dev["q"] = torch.tensor(host[0], device="cuda").to(torch.bfloat16)
    for scale in (0.002, -0.002):
        _check_far(w4, _run(w4, dev, scale=scale, max_new=1, max_group=rows), host, scale)


def test_prefixes_that_say_too_much_or_too_little():
    # what is shared ends with the shortest context; a prefix inside a page, inside a tile
    torch, w4 = cuda_or_skip()
    groups = [(96, [(0, 1), (40, 2), (64, 1)]), (64, [(1, 1), (3, 1)])]
    dev, host = lh.grouped(torch, groups, 8, 4, 128, 32, 4)
    want, tol = ref.attention(*host, 128 ** -0.5)
    for lens in ([96, 64], [95, 63], [33, 17], [15, 1], [0, 0]):
        dev["prefix_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        lh.check(w4, _run(w4, dev, max_new=2, max_group=4), want, tol)
    # every page of these two is the same, their last tokens as well
    dev["block_table"][4] = dev["block_table"][3]
    dev["seq_lens"][4] = dev["seq_lens"][3]
    dev["prefix_lens"] = torch.tensor([10 ** 9, 10 ** 9], dtype=torch.int32, device="cuda")
    table, ends = host[2].copy(), list(host[3])
    table[4], ends[4] = table[3], ends[3]
    dev["cu_groups"] = torch.tensor([3, 3, 5], dtype=torch.int32, device="cuda")
    want, tol = ref.attention(host[0], host[1], table, ends, host[4], 128 ** -0.5)
    lh.check(w4, _run(w4, dev, max_new=2, max_group=4), want, tol)


def test_lengths_and_groups_out_of_range():
    # neither read nor written through; the status is set, and rows of good requests are right
    torch, w4 = cuda_or_skip()
    dev, host = lh.grouped(torch, [(48, [(0, 1), (9, 1)]), (32, [(2, 1), (4, 1)])], 8, 4, 128, 16, 5)
    good, tol = ref.attention(*host, 128 ** -0.5)
    i32 = dict(dtype=torch.int32, device="cuda")
    bad = [("cu_groups", [0, 2, 9]), ("cu_groups", [-3, 2, 4]), ("cu_groups", [0, 4, 2]), ("prefix_lens", [-5, 32]),
           ("cu_new", [0, 1, 2, 3, 700]), ("cu_new", [0, 3, 1, 2, 4]), ("seq_lens", [49, 58, 35, 10 ** 6]),
           ("seq_lens", [-4, 58, 35, 37])]
    for name, value in bad:
        out = _run(w4, dict(dev, **{name: torch.tensor(value, **i32)}), scratch=lh.scratch(w4, dev), max_new=1, max_group=2)
        torch.cuda.synchronize()
        assert w4.w4a16_check_device_error() == 6, (name, value)
        if name == "prefix_lens" or value == [0, 2, 9]:
            assert (np.abs(out.double().cpu().numpy() - good) <= tol).all()
    # a page of the prefix that is not there hides its tokens
    dev["block_table"][:2, 1] = -1
    table = host[2].copy()
    table[:2, 1] = -1
    out = _run(w4, dev, max_new=1, max_group=2)
    torch.cuda.synchronize()
    assert w4.w4a16_check_device_error() == 6
    want, tol = ref.attention(host[0], host[1], table, host[3], host[4], 128 ** -0.5)
    lh.check(w4, out, want, tol)


@pytest.mark.parametrize("Hq,Hkv,D", [(16, 8, 256), (8, 1, 128)])
def test_captured_with_other_lengths_and_strided_rows(Hq, Hkv, D):
    # one graph for steps of different lengths; q is a slice of a fused row
    torch, w4 = cuda_or_skip()
    steps = [lh.grouped(torch, [(p, [(a, 1) for a in past]), (32, [(1, 1)] * 3)], Hq, Hkv, D, 16, p, gap=0)
             for p, past in ((64, range(40)), (224, range(50, 90)))]
    width = max(s[0]["block_table"].shape[1] for s in steps)
    blocks = max(s[0]["cache"].shape[0] for s in steps)
    T = steps[0][0]["q"].shape[0]
    now = {k: v.clone() for k, v in steps[0][0].items()}
    now["cache"] = torch.zeros(blocks, *now["cache"].shape[1:], dtype=torch.uint8, device="cuda")
    now["block_table"] = torch.full((43, width), -1, dtype=torch.int32, device="cuda")
    wide = torch.zeros(T, (Hq + 2) * D + 8, dtype=torch.bfloat16, device="cuda")
    now["q"] = wide[:, :Hq * D].unflatten(1, (Hq, D))
    scratch, out = lh.scratch(w4, now), torch.empty(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    kw = dict(scratch=scratch, out=out, max_new=1, max_group=40)

    def load(dev):
        for k, v in dev.items():
            now[k][tuple(slice(0, n) for n in v.shape)] = v
    load(steps[0][0])
    _run(w4, now, **kw)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _run(w4, now, **kw)
        _run(w4, now, **kw)
    for dev, host in steps * 2:
        load(dev)
        out.zero_()
        g.replay()
        _check(w4, out, host, D ** -0.5)


@pytest.mark.parametrize("Hq,Hkv,D", [(16, 8, 256), (8, 1, 128), (4, 4, 64)])
def test_caches_too_small_to_share(Hq, Hkv, D):
    torch, w4 = cuda_or_skip()
    dev, host = lh.grouped(torch, SMALL + [(32, [(0, 70), (3, 1)])], Hq, Hkv, D, 16, D, gap=1, wide=False)
    out = torch.full_like(dev["q"], float("nan"))
    _run(w4, dev, out=out, max_new=70, max_group=71)
    _check(w4, out, host, D ** -0.5)
    dev["cu_groups"][1] = 10 ** 6
    _run(w4, dev, out=out, max_new=70, max_group=71)
    torch.cuda.synchronize()
    assert w4.w4a16_check_device_error() == 6
    _check(w4, out, host, D ** -0.5)


@pytest.mark.parametrize("groups", [1500, 40])
def test_many_groups(groups):
    # more groups than a warp has lanes, more stretches than a launch has workers
    torch, w4 = cuda_or_skip()
    rng = np.random.default_rng(groups)
    some = [(int(rng.integers(0, 4)) * 16 if groups > 40 else int(rng.integers(1, 12)) * 16,
             [(int(rng.integers(0, 9)), 1) for _ in range(rng.integers(1, 4 if groups > 40 else 40))]) for _ in range(groups)]
    dev, host = lh.grouped(torch, some, 2, 1, 64, 16, groups)
    out = _run(w4, dev, max_new=1, max_group=40)
    _check(w4, out, host, 64 ** -0.5)


@pytest.mark.parametrize("requests,Hq,D", [(540, 20, 64), (270, 40, 128)])
def test_a_prefix_of_requests_that_fill_the_gpu(requests, Hq, D):
    # their own items fill it several times over
    torch, w4 = cuda_or_skip()
    dev, host = lh.grouped(torch, [(1040, [(i % 5, 1) for i in range(requests)])], Hq, 1, D, 16, D)
    out = _run(w4, dev, max_new=1, max_group=requests)
    _check(w4, out, host, D ** -0.5)


def test_a_prefix_with_more_items_than_pieces_may_have():
    # it stays whole.  Against kv4_attention, each of them within the bound of kv4_helpers.attention
    # of the exact result, with the largest |k| and |v| for every one
    torch, w4 = cuda_or_skip()
    n, H, D, pages = 4096, 20, 64, 20
    i32 = dict(dtype=torch.int32, device="cuda")
    g = torch.Generator("cuda").manual_seed(1)
    rows = lambda m: torch.randn(m, H, D, device="cuda", generator=g).to(torch.bfloat16).clamp(-4, 4)
    cache = w4.kv4_cache(pages + n, H, 16, D)
    lead = torch.randperm(pages + n, device="cuda", generator=g).to(torch.int32)
    own = lead[pages:]
    slots = torch.cat([(lead[:pages].long()[:, None] * 16 + torch.arange(16, device="cuda")).flatten(), own.long() * 16])
    w4.kv4_append(rows(len(slots)), rows(len(slots)), cache, slots)
    table = torch.cat([lead[:pages].expand(n, pages), own[:, None]], 1).contiguous()
    q, ends, cu = rows(n), torch.full((n,), 16 * pages + 1, **i32), torch.arange(n + 1, **i32)
    one = lambda x: torch.tensor(x, **i32)
    got = w4.kv4_prefix_attention(q, cache, table, ends, cu, one([16 * pages]), one([0, n]),
                                  w4.kv4_prefix_attention_scratch(n, n, 1, H, H, D), max_new=1, max_group=n).double()
    want = w4.kv4_attention(q, cache, table, ends, cu, w4.kv4_attention_scratch(H, H, D), max_new=1).double()
    largest = 4 + 8 / 15               # a rounding of 4 bits off the values written
    e = (2.0 ** -12 + 2.0 ** -20) * D ** -0.5 * largest * q.double().abs().sum(-1, keepdim=True)
    tol = 2 * (2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -12 + 2.0 ** -16 + torch.expm1(2 * e)) * largest * (1 + 2.0 ** -8))
    assert w4.w4a16_check_device_error() == 0
    assert ((got - want).abs() <= tol).all()


@pytest.mark.parametrize("D,members", [(64, 1), (256, 2)])
def test_most_requests_and_groups(D, members):
    torch, w4 = cuda_or_skip()
    some = [(16, [(j, 1) for j in range(members)]) for _ in range(4096 // members)]
    dev, host = lh.grouped(torch, some, 2, 1, D, 16, D)
    out = _run(w4, dev, max_new=1, max_group=members)
    _check(w4, out, host, D ** -0.5)


@pytest.mark.parametrize("rows,Hq,Hkv,D", [(30, 16, 8, 256), (30, 8, 2, 128), (60, 8, 2, 64), (3, 4, 1, 128)])
@pytest.mark.parametrize("flag", [1, 2])
def test_waits_that_run_out(rows, Hq, Hkv, D, flag):
    # test-only injection: no copy is issued and no item announced, or no product issued; the call
    # ends, reports it and leaves its scratch fit
    torch, w4 = cuda_or_skip()
    dev, host = lh.grouped(torch, [(160, [(i % 20, 1) for i in range(rows)])], Hq, Hkv, D, 16, D)
    scratch = lh.scratch(w4, dev)
    kw = dict(scratch=scratch, max_new=1, max_group=rows)
    first = _run(w4, dev, **kw)
    _check(w4, first, host, D ** -0.5)
    if flag == 2 and rows * Hq // Hkv <= 32:
        return                         # streamed: its warps copy for themselves
    w4.w4a16_debug_inject(flag)
    try:
        _run(w4, dev, **kw)
        status = w4.w4a16_check_device_error()
    finally:
        w4.w4a16_debug_inject(0)
    assert status == 5
    for _ in range(3):
        assert torch.equal(first, _run(w4, dev, **kw))
    assert w4.w4a16_check_device_error() == 0


@pytest.mark.parametrize("Hq,Hkv,D", [(16, 8, 256), (8, 2, 128)])
def test_a_server_with_one_prompt_for_all(Hq, Hkv, D):
    # the shared prompt is appended once; every request's table begins with its pages
    torch, w4 = cuda_or_skip()
    g = torch.Generator("cuda").manual_seed(D)
    B, bs, pages = 20, 16, 12
    i32 = dict(dtype=torch.int32, device="cuda")
    width = (65 << 20) // (B * bs * Hkv * 18 * D // 16) + 1
    blocks = pages + B * 6
    cache = w4.kv4_cache(blocks, Hkv, bs, D)
    rows = lambda n, h: torch.randn(n, h, D, device="cuda", generator=g).to(torch.bfloat16)
    ids = torch.randperm(blocks, device="cuda", generator=g).to(torch.int32)
    lead = ids[:pages]
    slots = (lead.long()[:, None] * bs + torch.arange(bs, device="cuda")).flatten()
    w4.kv4_append(rows(pages * bs, Hkv), rows(pages * bs, Hkv), cache, slots)
    table = torch.full((B, width), -1, **i32)
    table[:, :pages] = lead
    free, ctx = ids[pages:].clone(), torch.full((B,), pages * bs, **i32)
    prefix, groups = torch.tensor([pages * bs], **i32), torch.tensor([0, B], **i32)
    scratch = w4.kv4_prefix_attention_scratch(3 * B, B, 1, Hq, Hkv, D)
    plain = w4.kv4_attention_scratch(Hq, Hkv, D)
    for step in range(6):
        new = torch.randint(1, 4, (B,), device="cuda", generator=g, dtype=torch.int32)
        T = int(new.sum())
        plan = w4.kv4_plan(ctx, new, table, free, bs, num_tokens=T)
        q = rows(T, Hq)
        w4.kv4_append(rows(T, Hkv), rows(T, Hkv), cache, plan.slots)
        a = w4.kv4_prefix_attention(q, cache, table, plan.seq_lens, plan.cu_new, prefix, groups, scratch, max_new=3, max_group=T)
        b = w4.kv4_attention(q, cache, table, plan.seq_lens, plan.cu_new, plain, max_new=3)
        c = ref.Cache(blocks, Hkv, bs, D)
        c.raw = cache.cpu().numpy()
        want, tol = ref.attention(q.double().cpu().numpy(), c, table.cpu().numpy(), plan.seq_lens.tolist(), plan.cu_new.cpu().numpy(),
                                  D ** -0.5)
        lh.check(w4, a, want, tol)
        lh.check(w4, b, want, tol)
        ctx, free = plan.seq_lens, free[int(plan.taken):]


def test_on_another_stream_beside_another_call():
    # two calls at once, each with scratch of its own
    torch, w4 = cuda_or_skip()
    work = []
    for seed in (1, 2):
        dev, host = lh.grouped(torch, [(112, [(i, 1) for i in range(20)])], 8, 4, 128, 16, seed)
        work.append((dev, host, lh.scratch(w4, dev), torch.empty_like(dev["q"]), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for dev, _, scratch, out, stream in work:
            w4.kv4_prefix_attention(**dev, scratch=scratch, out=out, max_new=1, max_group=20, stream=stream)
    torch.cuda.synchronize()
    for _, host, _, out, _ in work:
        _check(w4, out, host, 128 ** -0.5)
