"""Attention of requests that share a prefix, where something of it is no
number, too long or not there: the rows that it concerns answer as
kv4_attention does, and the others are right."""
import numpy as np
import pytest

from tests import kv4_helpers as ref
from tests import kv4_long_helpers as lh
from tests.gpu_helpers import cuda_or_skip

pytestmark = pytest.mark.gpu


def _run(w4, dev, scratch=None, **kw):
    return w4.kv4_prefix_attention(**dev, scratch=lh.scratch(w4, dev) if scratch is None else scratch, **kw)


def _plain(w4, dev, most):
    Hq, Hkv, D = dev["q"].shape[1], dev["cache"].shape[1], dev["q"].shape[2]
    return w4.kv4_attention(dev["q"], dev["cache"], dev["block_table"], dev["seq_lens"], dev["cu_new"],
                            w4.kv4_attention_scratch(Hq, Hkv, D), max_new=most)


def _check_rows(out, want, tol, rows):
    got = out.double().cpu().numpy()[rows]
    bad = ~(np.abs(got - want[rows]) <= tol[rows])
    assert not bad.any(), "%d of %d off, first %s: %r" % (bad.sum(), bad.size, np.argwhere(bad)[0], got[bad][0])


# groups, heads, the most new tokens of a request and of a group
SHARED = {
    "tensor cores": ([(160, [(i % 20, 1) for i in range(30)])], 16, 8, 256, 1, 30),
    "tensor cores, one head": ([(400, [(i % 9, 1 + i % 3) for i in range(60)])], 8, 2, 64, 3, 119),
    "two forms": ([(320, [(i, 1) for i in range(40)]), (96, [(3, 1), (40, 1), (0, 1)])], 8, 2, 128, 1, 40),
    "streamed": ([(64 + 16 * (i % 3), [(i % 5, 1), (7, 1), (30, 1)]) for i in range(50)], 8, 8, 64, 1, 3),
    "streamed, split": ([(2000, [(i, 1) for i in range(6)])], 8, 4, 128, 1, 6),
    "prompts": ([(128, [(0, 150), (3, 33), (0, 1), (0, 70)] + [(i, 1) for i in range(30)]), (64, [(0, 5), (40, 1)])], 4, 1, 128, 150, 284),
}


@pytest.mark.parametrize("name", SHARED)
@pytest.mark.parametrize("wide", [True, False])
def test_queries_that_are_no_numbers(name, wide):
    # rows of them are NaN whatever the split, and no others
    torch, w4 = cuda_or_skip()
    groups, Hq, Hkv, D, most, widest = SHARED[name]
    dev, host = lh.grouped(torch, groups, Hq, Hkv, D, 16, D + len(groups), wide=wide)
    want, tol = ref.attention(*host, D ** -0.5)
    T = len(want)
    for value in (float("nan"), float("inf"), -float("inf")):
        here = {(0, 0): slice(None), (1, Hq - 1): 5, (T - 1, 1): slice(D - 1, None), (T // 2, 0): slice(1, None, 3)}
        rows = np.ones((T, Hq), bool)
        x = dict(dev, q=dev["q"].clone())
        for (t, h), d in here.items():
            x["q"][t, h, d] = value
            rows[t, h] = False
        out = _run(w4, x, max_new=most, max_group=widest)
        assert torch.equal(out.isnan(), _plain(w4, x, most).isnan())
        assert out.isnan().all(-1).cpu().numpy()[~rows].all()
        _check_rows(out, want, tol, rows)
        assert w4.w4a16_check_device_error() == 0


@pytest.mark.parametrize("name", ["tensor cores", "two forms", "streamed", "streamed, split"])
@pytest.mark.parametrize("where", ["shared", "own"])
def test_a_key_that_is_no_number(name, where):
    # in what is shared: all rows of its group and head; in what a request has of its own: that request's
    torch, w4 = cuda_or_skip()
    groups, Hq, Hkv, D, most, widest = SHARED[name]
    dev, host = lh.grouped(torch, groups, Hq, Hkv, D, 16, D + len(groups))
    q, c, table, ends, cu = host
    want, tol = ref.attention(*host, D ** -0.5)
    last = len(groups[0][1])                       # requests of the first group
    b = 0 if where == "shared" else 2
    slot = int(table[b, 1 if where == "shared" else (ends[b] - 1) // 16])
    cache = dev["cache"].clone()
    cache[slot, 0, 0].view(torch.float16)[8 * D] = float("nan")    # the scale of token 0, group 0 of K in head 0
    rows = np.ones((len(q), Hq), bool)
    first, end = (0, last) if where == "shared" else (b, b + 1)
    rows[cu[first]:cu[end], :Hq // Hkv] = False
    x = dict(dev, cache=cache)
    out = _run(w4, x, max_new=most, max_group=widest)
    assert torch.equal(out.isnan(), _plain(w4, x, most).isnan())
    assert out.isnan().all(-1).cpu().numpy()[~rows].all()
    _check_rows(out, want, tol, rows)


@pytest.mark.parametrize("name", SHARED)
def test_scratch_is_left_fit_for_the_next_call(name):
    # counters, and the word that tells of a plan; results as from a fresh one
    torch, w4 = cuda_or_skip()
    groups, Hq, Hkv, D, most, widest = SHARED[name]
    dev, host = lh.grouped(torch, groups, Hq, Hkv, D, 16, D + len(groups))
    scratch = lh.scratch(w4, dev)
    first = _run(w4, dev, scratch=scratch, max_new=most, max_group=widest)
    for _ in range(20):
        assert torch.equal(first, _run(w4, dev, scratch=scratch, max_new=most, max_group=widest))
    torch.cuda.synchronize()
    assert not scratch[:13312].any()
    # behind a call of fewer tokens, whose plan and parts lie elsewhere in the scratch
    few = dict(dev, q=dev["q"][:2].contiguous(), cu_new=dev["cu_new"].clamp(max=2))
    _run(w4, few, scratch=scratch, max_new=most, max_group=widest)
    torch.cuda.synchronize()
    w4.w4a16_check_device_error()
    assert not scratch[:13312].any()
    assert torch.equal(first, _run(w4, dev, scratch=scratch, max_new=most, max_group=widest))


def _idle_and_short(torch, active, idle, Hq, Hkv, D, seed):
    """A group whose first requests have no new tokens, and tables and lengths of theirs that are no longer
    anything; one whose context ends inside the prefix that is said to be shared by 640 tokens."""
    members = [(0, 0)] * idle + [(1 + i % 40, 1) for i in range(active)]
    dev, host = lh.grouped(torch, [(640, members), (0, [(9, 1), (3, 2)])], Hq, Hkv, D, 16, seed)
    q, c, table, ends, cu = host
    table, ends = table.copy(), list(ends)
    ends[idle + 1] = 422            # 421 tokens before the step: 416 are shared
    junk = np.random.default_rng(seed).choice([-1, 10 ** 8, c.blocks, -2 ** 31], (idle, table.shape[1]))
    i32 = dict(dtype=torch.int32, device="cuda")
    dev["seq_lens"] = torch.tensor([10 ** 9 if b % 2 else -7 for b in range(idle)] + ends[idle:], **i32)
    dev["block_table"][:idle] = torch.tensor(junk, **i32)
    return dev, (q, c, table, ends, cu), idle


@pytest.mark.parametrize("active,Hq,Hkv,D", [(12, 8, 8, 64), (6, 8, 2, 128), (7, 16, 8, 256), (50, 8, 2, 128), (40, 16, 8, 256), (90, 8, 2, 64)])
@pytest.mark.parametrize("said", [640, 10 ** 9])
def test_idle_requests_first_and_a_context_that_ends_inside_the_prefix(active, Hq, Hkv, D, said):
    # few rows, streamed, and many, on the tensor cores
    torch, w4 = cuda_or_skip()
    dev, host, idle = _idle_and_short(torch, active, 3, Hq, Hkv, D, D + active)
    dev["prefix_lens"][0] = said
    if said > 640:
        # the tables agree for ever: one context for all, and their own tokens too
        i32 = dict(dtype=torch.int32, device="cuda")
        q, c, table, ends, cu = host
        rows = slice(idle, idle + active)
        table[rows] = table[idle]
        ends[rows] = [min(e, ends[idle]) for e in ends[rows]]
        dev["block_table"][rows], dev["seq_lens"][rows] = torch.tensor(table[rows], **i32), torch.tensor(ends[rows], **i32)
    want, tol = ref.attention(*host, D ** -0.5)
    scratch = lh.scratch(w4, dev)
    out = _run(w4, dev, scratch=scratch, max_new=2, max_group=active)
    lh.check(w4, out, want, tol)
    # shared it is, and read by the first request with new tokens: the others' entries are not looked at
    dev["block_table"][idle + 1:idle + active, :416 // 16] = -1
    assert torch.equal(out, _run(w4, dev, scratch=scratch, max_new=2, max_group=active))
    torch.cuda.synchronize()
    assert w4.w4a16_check_device_error() == 0


# numbers that are out of range, and the requests that they concern
BAD = [("cu_groups", {2: 9000}, []), ("cu_groups", {0: -3}, []), ("cu_groups", {1: 10 ** 9}, []), ("prefix_lens", {0: -5}, []),
       ("cu_new", {-1: 70000}, [-1]), ("seq_lens", {-1: 10 ** 6}, [-1]), ("seq_lens", {0: -4}, [0]), ("seq_lens", {5: 2 ** 31 - 1}, [5])]


@pytest.mark.parametrize("active,Hq,Hkv,D", [(12, 8, 8, 64), (6, 8, 2, 128), (50, 8, 2, 128), (40, 16, 8, 256)])
def test_requests_beside_numbers_out_of_range(active, Hq, Hkv, D):
    # every row of the others is right
    torch, w4 = cuda_or_skip()
    groups = [(320, [(1 + i % 40, 1) for i in range(active)]), (48, [(9, 1), (3, 2)])]
    dev, host = lh.grouped(torch, groups, Hq, Hkv, D, 16, D + active)
    want, tol = ref.attention(*host, D ** -0.5)
    cu = host[4]
    for name, values, concerned in BAD:
        x = dict(dev, **{name: dev[name].clone()})
        for i, v in values.items():
            x[name][i] = v
        out = _run(w4, x, max_new=2, max_group=active)
        torch.cuda.synchronize()
        assert w4.w4a16_check_device_error() == 6, (name, values)
        rows = np.ones(len(want), bool)
        for b in concerned:
            b %= len(cu) - 1
            rows[cu[b]:cu[b + 1]] = False
        _check_rows(out, want, tol, rows)
