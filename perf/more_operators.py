"""What is measured of long contexts in the 4-bit key/value cache: cases, inputs and plain forms.

Two ways of not reading all of a long cache for every request of a decode step:

* prefix   attention of requests that share the first tokens of their contexts, in the same pages of the cache: these
           tokens are attended to once for all of a group's rows (kv4_prefix_attention);
* sparse   attention over pages that a cheap score selects for every new token and key head (kv4_sparse_attention), with
  bounds   the smallest and the largest key of a page in 8 bits, written when its last token is (kv4_bounds), and
  select   the score of a page, the most that any query head of the group could get from a key within its bounds, and the
           choice of the highest (kv4_select).

`own` chooses between the plain forms (elementary torch operations in 32 bits) and the library's kernels.

The cache is uint8 [blocks, kv heads, block / 16, 18 D]: tiles of 16 tokens x D elements, each holding the codes of K
[D / 64, 16, 32] (two per byte, the even element in the low nibble), those of V, then (scale, zero) in binary16 of K
[D / 64, 16, 2] and of V.  A value is (code - zero) * scale, with one scale and zero for 64 elements of a token's head.

The bounds are uint8 [blocks, kv heads, 2 D + 16]: D whole numbers in 8 bits (high), D more (low), and up to four
binary32 steps, one for 64 elements: a key of the page lies between low * step and high * step.
"""
import math

import torch

own = False

DEV = "cuda"
GROUP = 64   # elements of a head that share a scale, a zero and a step
TILE = 16    # tokens of a cache tile
STEP = 65 / 8192   # of a group's largest magnitude: whole numbers to 127 at most, and the factor is exact


# ------------------------------------------------------------------ cases

def listed():
    heads = {"hq": 16, "hkv": 8, "d": 256}
    small = {"hq": 32, "hkv": 8, "d": 128}
    return [
        # one decode step of 64 requests: four of them fill a page; launch latency is all there is
        {"name": "bounds decode", "op": "bounds", "tokens": 64, "in_order": False, **heads, "block": 16},
        # a long prompt just written, from inside a page to inside another
        {"name": "bounds prompt", "op": "bounds", "tokens": 65519, "in_order": True, **heads, "block": 64},
        # one request's decode step after a long context: few rows, many pages
        {"name": "select one", "op": "select", "requests": 1, "ctx_lo": 131071, "ctx_hi": 131071, "new": 1, **heads, "block": 64, "top": 64, "first": 1, "recent": 2},
        # a served batch of ragged contexts in small pages
        {"name": "select batch", "op": "select", "requests": 64, "ctx_lo": 2000, "ctx_hi": 120000, "new": 1, **heads, "block": 32, "top": 64, "first": 1, "recent": 4},
        # a further piece of a prompt, grouped by four, each of its tokens with pages of its own
        {"name": "select piece", "op": "select", "requests": 1, "ctx_lo": 30001, "ctx_hi": 30001, "new": 301, **small, "block": 64, "top": 17, "first": 0, "recent": 1},
        # one request's step over 2048 selected tokens
        {"name": "sparse one", "op": "sparse", "requests": 1, "ctx_lo": 40000, "ctx_hi": 40000, "new": 1, **heads, "block": 64, "top": 32},
        # a served batch, the same number of tokens in small pages; short contexts have fewer
        {"name": "sparse batch", "op": "sparse", "requests": 128, "ctx_lo": 700, "ctx_hi": 16000, "new": 1, **heads, "block": 16, "top": 128},
        # every token of a prompt piece over pages of its own
        {"name": "sparse piece", "op": "sparse", "requests": 1, "ctx_lo": 20001, "ctx_hi": 20001, "new": 301, **small, "block": 64, "top": 17},
        # four samples of one short prompt
        {"name": "prefix few", "op": "prefix", "groups": 1, "members_lo": 4, "members_hi": 4, "prefix_lo": 2048, "prefix_hi": 2048, "past_lo": 3, "past_hi": 200, "new_lo": 1, "new_hi": 1, **heads, "block": 16},
        # a served batch behind one long system prompt
        {"name": "prefix batch", "op": "prefix", "groups": 1, "members_lo": 128, "members_hi": 128, "prefix_lo": 32768, "prefix_hi": 32768, "past_lo": 1, "past_hi": 2000, "new_lo": 1, "new_hi": 1, **heads, "block": 64},
        # several groups of different size behind prompts of different length, a few drafted tokens a request
        {"name": "prefix groups", "op": "prefix", "groups": 7, "members_lo": 1, "members_hi": 30, "prefix_lo": 333, "prefix_hi": 24000, "past_lo": 0, "past_hi": 3001, "new_lo": 1, "new_hi": 4, **small, "block": 16},
        # new prompts behind one shared one
        {"name": "prefix prompts", "op": "prefix", "groups": 1, "members_lo": 12, "members_hi": 12, "prefix_lo": 6016, "prefix_hi": 6016, "past_lo": 0, "past_hi": 0, "new_lo": 101, "new_hi": 700, **heads, "block": 64},
    ]


def draw(rng):
    def log_int(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    hq, hkv = rng.choice([(16, 8), (32, 8), (8, 1), (12, 12), (28, 4), (20, 10), (64, 4)])
    heads = {"hq": hq, "hkv": hkv, "d": rng.choice([64, 128, 256, 256])}
    block = rng.choice([16, 32, 64, 128])
    wide = max(1, -(-hkv * heads["d"] // 2048))   # the listed cases have 2048 elements of K a token
    op = rng.choice(["bounds", "select", "select", "sparse", "sparse", "prefix", "prefix", "prefix"])
    if op == "bounds":
        in_order = rng.random() < 0.6
        return {"op": op, "tokens": log_int(1, 65519 // wide if in_order else 1000), "in_order": in_order, **heads, "block": block}
    if op in ("select", "sparse"):
        rows = log_int(1, 96)
        piece = rng.random() < 0.3
        top = log_int(3, 128)
        new = rows if piece else rng.choice([1, 1, 1, 2])
        if op == "sparse":
            tokens = rows if piece else rows * new
            top = max(2, min(top, 4096 // block, 200000 * 8 // (tokens * block * max(hkv, 8) * wide)))
        hi = log_int(200, max(300, min(120000, (130000 if op == "select" else 40000) * block // (rows * wide * 4 // 3 + 1))) if not piece else 30000)
        c = {"op": op, "requests": 1 if piece else rows, "ctx_lo": max(1, hi // 30), "ctx_hi": hi, "new": new, **heads, "block": block, "top": top}
        return dict(c, first=rng.randint(0, 1), recent=rng.randint(1, 2)) if op == "select" else c
    groups = log_int(1, 8)
    most = log_int(1, 96 // groups)
    prompts = rng.random() < 0.25
    new = log_int(5, max(5, 1500 // (groups * most))) if prompts else rng.choice([1, 1, 1, 2, 5])
    prefix = log_int(block, 24000 // max(1, groups * wide // 2))
    return {"op": op, "groups": groups, "members_lo": max(1, most // 5), "members_hi": most, "prefix_lo": max(block, prefix // 10), "prefix_hi": max(block, prefix),
            "past_lo": rng.choice([0, 1, 40]), "past_hi": log_int(40, 2000), "new_lo": max(1, new // 3), "new_hi": new, **heads, "block": block}


def _spread(lo, hi, n, turn):
    """n whole numbers from lo to hi, spread evenly over their logarithm in a fixed scattered order; the ends are among
    them."""
    if n == 1:
        return [hi]
    step = next(s for s in (turn, turn + 2, turn + 4, 1) if math.gcd(s, n) == 1)
    a, b = math.log(lo + 1), math.log(hi + 1)
    return [int(round(math.exp(a + (b - a) * ((i * step) % n) / (n - 1)))) - 1 for i in range(n)]


def _requests(case):
    """Of each request: tokens in the cache before the step, new ones, shared ones; and the groups' borders."""
    if case["op"] != "prefix":
        n = case["requests"]
        return _spread(case["ctx_lo"], case["ctx_hi"], n, 7), [case["new"]] * n, [0] * n, None
    b, groups = case["block"], case["groups"]
    members = _spread(case["members_lo"], case["members_hi"], groups, 3)
    shared = [max(1, p // b) * b for p in _spread(case["prefix_lo"], case["prefix_hi"], groups, 5)]   # whole pages
    n = sum(members)
    prefix = [p for m, p in zip(members, shared) for _ in range(m)]
    borders = [0]
    for m in members:
        borders.append(borders[-1] + m)
    ctx = [p + o for p, o in zip(prefix, _spread(case["past_lo"], case["past_hi"], n, 7))]
    return ctx, _spread(case["new_lo"], case["new_hi"], n, 11), prefix, borders


def _pages_filled(case):
    t, b = case["tokens"], case["block"]
    return (t + 5) // b if case["in_order"] else sum(i * 7 % b == b - 1 for i in range(t))


def work(case):
    op, hq, hkv, d, b = case["op"], case["hq"], case["hkv"], case["d"], case["block"]
    half = d // 2 + d // GROUP * 4         # bytes of a token's key in one head; its value takes as many
    row = 2 * d + d // GROUP * 4           # bytes of a page's bounds in one head
    if op == "bounds":
        n = _pages_filled(case) * hkv
        return {"bytes": n * (b * half + row) + 8 * case["tokens"], "flops": 4 * n * b * d}
    ctx, new, shared, borders = _requests(case)
    t = sum(new)
    if op == "select":
        # of a request whose pages are all taken nothing needs to be scored
        scored = [(c + n - 1) // b * (c + n > case["top"] * b) for c, n in zip(ctx, new)]
        return {"bytes": sum(scored) * hkv * row + 2 * t * hq * d + 4 * t * (hkv * case["top"] + 1) + 4 * sum(-(-(c + n) // b) for c, n in zip(ctx, new)),
                "flops": 2 * d * hq * sum(s * n for s, n in zip(scored, new))}
    if op == "sparse":
        keys = 0
        for c, n in zip(ctx, new):
            for p in range(c, c + n):
                keys += (min(case["top"], p // b + 1) - 1) * b + p % b + 1
        return {"bytes": keys * hkv * 2 * half + 4 * t * hq * d + 4 * t * (hkv * case["top"] + 1), "flops": 4 * keys * hq * d}
    tokens = sum(c + n - s for c, n, s in zip(ctx, new, shared)) + sum(shared[r] for r in borders[:-1])
    pairs = sum(n * c + n * (n + 1) // 2 for c, n in zip(ctx, new))
    return {"bytes": tokens * hkv * 2 * half + 4 * t * hq * d, "flops": 4 * pairs * hq * d}


# ----------------------------------------------------------------- inputs

def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return {"bounds": _prepare_bounds, "select": _prepare_select, "sparse": _prepare_sparse, "prefix": _prepare_prefix}[case["op"]](case, g)


def _cache(case, blocks, g):
    # codes and parameters as quantised normal values have them: a bell over the 16 codes, zeros near the middle
    d, hkv, b = case["d"], case["hkv"], case["block"]
    tiles = blocks * hkv * (b // TILE)
    cache = torch.empty(tiles, 18 * d, dtype=torch.uint8, device=DEV)
    count = torch.tensor([1, 2, 4, 7, 12, 19, 26, 31, 33, 31, 26, 19, 12, 7, 4, 2], device=DEV)
    level = torch.repeat_interleave(torch.arange(16, device=DEV, dtype=torch.uint8), count)
    level = torch.cat([level, torch.full((256 - level.numel(),), 8, dtype=torch.uint8, device=DEV)])
    pair = (level[:, None] | (level[None] << 4)).reshape(-1)
    step = max(1, (1 << 28) // (16 * d))
    for i in range(0, tiles, step):   # in pieces: the random words of the codes take more room than the codes
        n = min(step, tiles - i)
        cache[i:i + n, :16 * d] = pair[torch.randint(0, 65536, (n, 16 * d), device=DEV, generator=g, dtype=torch.int32)]
    scale = (0.25 + 0.2 * torch.rand(tiles, 2, d // GROUP, TILE, device=DEV, generator=g)).half()
    zero = torch.randint(6, 10, scale.shape, device=DEV, generator=g).half()
    cache[:, 16 * d:] = torch.stack([scale, zero], -1).reshape(tiles, -1).view(torch.uint8)
    return cache.view(blocks, hkv, b // TILE, 18 * d)


def _prepare_bounds(case, g):
    t, b = case["tokens"], case["block"]
    # pages in any order; a prompt's tokens follow each other from inside a page on, those of a decode step each have a page
    at = torch.arange(t, device=DEV) + 5 if case["in_order"] else torch.arange(t, device=DEV) * b + torch.arange(t, device=DEV) * 7 % b
    blocks = (t + 5) // b + 3 if case["in_order"] else t + 2
    pages = torch.randperm(blocks, device=DEV, generator=g)
    return {"case": case, "cache": _cache(case, blocks, g), "slots": pages[at // b] * b + at % b, "filled": _pages_filled(case),
            "bounds": torch.zeros(blocks, case["hkv"], 2 * case["d"] + 16, dtype=torch.uint8, device=DEV)}


def _batch(case, g):
    """Queries, block table (shared pages first), lengths and running sums of a step; and the number of blocks."""
    ctx, new, shared, borders = _requests(case)
    b, n = case["block"], len(ctx)
    ends = [c + k for c, k in zip(ctx, new)]
    lead = [s // b for s in shared]
    tail = [-(-e // b) - k for e, k in zip(ends, lead)]
    firsts = borders[:-1] if borders else []
    blocks = sum(tail) + sum(lead[r] for r in firsts) + 3
    ids = torch.randperm(blocks, device=DEV, generator=g).to(torch.int32)
    table = torch.full((n, max(k + t for k, t in zip(lead, tail)) + 1), -1, dtype=torch.int32, device=DEV)
    at = 0
    for i, r in enumerate(firsts):
        table[r:borders[i + 1], :lead[r]] = ids[at:at + lead[r]]
        at += lead[r]
    column = torch.arange(table.shape[1], device=DEV)[None]
    first, last = _i32(lead)[:, None], _i32([k + t for k, t in zip(lead, tail)])[:, None]
    table[(column >= first) & (column < last)] = ids[at:at + sum(tail)]
    cu = [0]
    for k in new:
        cu.append(cu[-1] + k)
    q = torch.randn(cu[-1], case["hq"], case["d"], device=DEV, generator=g).to(torch.bfloat16)
    return {"case": case, "q": q, "table": table, "ends": _i32(ends), "cu": _i32(cu)}, blocks


def _owner(cu, tokens):
    """Request of each new token."""
    return torch.searchsorted(cu, torch.arange(tokens, device=DEV, dtype=torch.int32), right=True) - 1


def _prepare_select(case, g):
    s, blocks = _batch(case, g)
    shape = (blocks, case["hkv"], case["d"])
    middle = 12 * torch.randn(shape, device=DEV, generator=g)
    reach = 40 + 60 * torch.rand(shape, device=DEV, generator=g)   # of a few dozen normal keys, either way
    step = 0.01 + 0.02 * torch.rand(blocks, case["hkv"], 4, device=DEV, generator=g)
    whole = torch.cat([(middle + reach).clamp(-127, 127), (middle - reach).clamp(-127, 127)], -1).to(torch.int8)
    s["bounds"] = torch.cat([whole.view(torch.uint8), step.view(torch.uint8)], -1)
    t = s["q"].shape[0]
    s["tables"] = torch.empty(t, case["hkv"], case["top"], dtype=torch.int32, device=DEV)
    s["lens"] = torch.empty(t, dtype=torch.int32, device=DEV)
    return s


def _prepare_sparse(case, g):
    s, blocks = _batch(case, g)
    b, top, hkv, t = case["block"], case["top"], case["hkv"], s["q"].shape[0]
    own_row = _owner(s["cu"], t)
    p = s["ends"][own_row] - s["cu"][own_row + 1] + torch.arange(t, device=DEV, dtype=torch.int32)
    seen = p // b + 1
    # any pages for each token and head, its own among them, in order
    weight = torch.rand(t, hkv, max(s["table"].shape[1], top), device=DEV, generator=g)
    column = torch.arange(weight.shape[2], device=DEV)
    weight = weight.masked_fill((column >= seen[:, None])[:, None], -1).masked_fill((column == seen[:, None] - 1)[:, None], 2)
    pages = weight.topk(top, -1).indices
    pages = torch.where(pages < seen[:, None, None], pages, weight.shape[2]).sort(-1).values
    known = pages < seen[:, None, None]
    ids = s["table"][own_row[:, None, None], pages.clamp(max=s["table"].shape[1] - 1)]
    s["tables"] = torch.where(known, ids, -1).contiguous()
    s["lens"] = ((seen.clamp(max=top) - 1) * b + p % b + 1).to(torch.int32)
    s["cache"] = _cache(case, blocks, g)
    s["out"] = torch.empty_like(s["q"])
    return s


def _prepare_prefix(case, g):
    s, blocks = _batch(case, g)
    ctx, new, shared, borders = _requests(case)
    s["prefix"], s["groups"] = _i32([shared[r] for r in borders[:-1]]), _i32(borders)
    s["cache"] = _cache(case, blocks, g)
    s["out"] = torch.empty_like(s["q"])
    # what the host of a serving loop knows of its step
    s["most"], s["widest"] = max(new), max(sum(new[a:e]) for a, e in zip(borders, borders[1:]))
    s["sizes"] = list(zip(borders, borders[1:], (shared[r] for r in borders[:-1])))
    s["lengths"], s["counts"] = [c + n for c, n in zip(ctx, new)], new
    return s


# -------------------------------------------------------------------- run

def run(state):
    return (_run_own if own else _run_plain)(state)


def _codes(bounds, d):
    """The bounds' parts: whole numbers and steps."""
    return {"high": bounds[..., :d].view(torch.int8), "low": bounds[..., d:2 * d].view(torch.int8), "step": bounds[..., 2 * d:].view(torch.float32)[..., :d // GROUP]}


def _run_own(s):
    import gemm_w4a16_gemv_gb300 as w4
    c = s["case"]
    op = c["op"]
    if op == "bounds":
        return _codes(w4.kv4_bounds(s["cache"], s["slots"], s["bounds"]), c["d"])
    if op == "select":
        tables, lens = w4.kv4_select(s["q"], s["bounds"], s["table"], s["ends"], s["cu"], c["block"], c["top"], first=c["first"], recent=c["recent"],
                                     tables=s["tables"], lens=s["lens"])
        return {"tables": tables, "lens": lens}
    if "scratch" not in s:   # kept by the user's program between calls
        s["scratch"] = (w4.kv4_attention_scratch(c["hq"], c["hkv"], c["d"], device=DEV) if op == "sparse" else
                        w4.kv4_prefix_attention_scratch(s["q"].shape[0], len(s["counts"]), len(s["sizes"]), c["hq"], c["hkv"], c["d"], device=DEV))
    if op == "sparse":
        return w4.kv4_sparse_attention(s["q"], s["cache"], s["tables"], s["lens"], s["scratch"], out=s["out"], scale=c["d"] ** -0.5)
    return w4.kv4_prefix_attention(s["q"], s["cache"], s["table"], s["ends"], s["cu"], s["prefix"], s["groups"], s["scratch"], out=s["out"],
                                   scale=c["d"] ** -0.5, max_new=s["most"], max_group=s["widest"])


def _run_plain(s):
    return {"bounds": _plain_bounds, "select": _plain_select, "sparse": _plain_sparse, "prefix": _plain_prefix}[s["case"]["op"]](s)


def _cells(tiles, d, part):
    """K (part 0) or V (1) as 32-bit values [..., 16 n, D] of tiles [..., n, 18 D]."""
    codes = tiles[..., part * 8 * d:(part + 1) * 8 * d].unflatten(-1, (d // GROUP, TILE, GROUP // 2))
    para = tiles[..., (16 + part) * d:(17 + part) * d].contiguous().view(torch.float16).unflatten(-1, (d // GROUP, TILE, 2)).float()
    x = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()   # [..., n, groups, 16, 64]
    x = (x - para[..., 1:]) * para[..., :1]
    return x.transpose(-3, -2).flatten(-2).flatten(-3, -2)


def _plain_bounds(s):
    d, b, bounds, slots = s["case"]["d"], s["case"]["block"], s["bounds"], s["slots"]
    last = torch.sort(slots % b != b - 1, stable=True).indices[:s["filled"]]   # tokens that fill their pages
    page = slots[last] // b
    k = _cells(s["cache"][page], d, 0)                                         # [pages, heads, block, D]
    high, low = k.amax(2).unflatten(-1, (-1, GROUP)), k.amin(2).unflatten(-1, (-1, GROUP))
    step = torch.maximum(high.abs(), low.abs()).amax(-1) * STEP
    safe = torch.where(step > 0, step, torch.ones_like(step))[..., None]
    whole = torch.cat([(high / safe).ceil().flatten(-2), (low / safe).floor().flatten(-2)], -1).to(torch.int8)
    bounds[page, :, :2 * d] = whole.view(torch.uint8)
    bounds[page, :, 2 * d:2 * d + d // 16] = step.view(torch.uint8)
    return _codes(bounds, d)


def _plain_select(s):
    c = s["case"]
    d, hkv, b, top = c["d"], c["hkv"], c["block"], c["top"]
    q = s["q"].float()
    t = q.shape[0]
    r = _owner(s["cu"], t)
    p = s["ends"][r] - s["cu"][r + 1] + torch.arange(t, device=DEV, dtype=torch.int32)
    seen = p // b + 1
    # queries as whole numbers in 8 bits: sums of products of whole numbers do not depend on their order
    unit = q.abs().amax(-1) * STEP                                                  # [T, heads]
    whole = (q / torch.where(unit > 0, unit, torch.ones_like(unit))[..., None]).round().view(t, hkv, -1, d // GROUP, GROUP)
    table = s["table"][r]                                                           # [T, pages]
    part = _codes(s["bounds"][table.clamp(min=0).long()], d)                        # [T, pages, heads, D]
    high, low = (part[name].float().unflatten(-1, (-1, GROUP)) for name in ("high", "low"))
    dot = torch.einsum("thgnd,tphnd->thgnp", whole.clamp(min=0), high) + torch.einsum("thgnd,tphnd->thgnp", whole.clamp(max=0), low)
    dot = dot * part["step"].permute(0, 2, 3, 1)[:, :, None]
    while dot.shape[3] > 1:                                                         # neighbouring groups of 64 first
        dot = dot[:, :, :, 0::2] + dot[:, :, :, 1::2]
    score = (dot[:, :, :, 0] * unit.view(t, hkv, -1, 1)).amax(2)                    # [T, heads, pages]
    page = torch.arange(table.shape[1], device=DEV)
    score = score.masked_fill(((page < c["first"]) | (page >= seen[:, None] - c["recent"]))[:, None], math.inf)
    score = score.masked_fill((page >= seen[:, None])[:, None], -math.inf)
    order = torch.sort(score, dim=-1, descending=True, stable=True).indices[..., :top]
    order = torch.nn.functional.pad(order, (0, top - order.shape[-1]), value=page.numel())
    taken = seen.clamp(max=top)
    order = torch.where((torch.arange(top, device=DEV) < taken[:, None])[:, None], order, page.numel()).sort(-1).values
    ids = table[torch.arange(t, device=DEV)[:, None, None], order.clamp(max=page.numel() - 1)]
    return {"tables": torch.where(order < page.numel(), ids, -1), "lens": ((taken - 1) * b + p % b + 1).to(torch.int32)}


def _plain_sparse(s):
    c = s["case"]
    d, h, t = c["d"], c["hkv"], s["q"].shape[0]
    tiles = s["cache"][s["tables"].clamp(min=0).long(), torch.arange(h, device=DEV)[None, :, None]].flatten(2, 3)   # [T, heads, tiles, bytes]
    k, v = _cells(tiles, d, 0), _cells(tiles, d, 1)
    x = (s["q"].float().view(t, h, -1, d) * d ** -0.5) @ k.transpose(-1, -2)
    x = x.masked_fill((torch.arange(x.shape[-1], device=DEV) >= s["lens"][:, None])[:, None, None], -math.inf)
    x = (x - x.amax(-1, keepdim=True)).exp()
    return ((x @ v) / x.sum(-1, keepdim=True)).flatten(1, 2).to(torch.bfloat16)


def _plain_prefix(s):
    c = s["case"]
    d, h, b = c["d"], c["hkv"], c["block"]
    g = c["hq"] // h
    q, table, cache = s["q"], s["table"], s["cache"]
    out = torch.empty_like(q)
    token = 0
    for first, last, prefix in s["sizes"]:
        counts, ends = s["counts"][first:last], s["lengths"][first:last]
        n, most, pages = last - first, max(counts), -(-max(ends) // b)
        rows = sum(counts)
        i = torch.arange(most, device=DEV)
        at = s["cu"][first:last, None] + i[None]                                      # [n, most]
        here = i[None] < (s["cu"][first + 1:last + 1] - s["cu"][first:last])[:, None]
        x = q.float()[at.clamp(max=q.shape[0] - 1).long()] * d ** -0.5                # [n, most, heads, D]
        x = x.view(n, most, h, g, d).permute(0, 2, 3, 1, 4)                           # [n, h, g, most, D]
        lead = cache[table[first, :prefix // b].long()].transpose(0, 1).flatten(1, 2)             # [h, tiles, bytes]
        tail = cache[table[first:last, prefix // b:pages].clamp(min=0).long()].transpose(1, 2).flatten(2, 3)   # [n, h, tiles, bytes]
        shared = x.transpose(0, 1).reshape(h, n * g * most, d) @ _cells(lead, d, 0).transpose(-1, -2)
        own_part = (x.reshape(n, h, g * most, d) @ _cells(tail, d, 0).transpose(-1, -2)).view(n, h, g, most, -1)
        position = (s["ends"][first:last] - s["cu"][first + 1:last + 1] + s["cu"][first:last])[:, None] + i
        j = prefix + torch.arange(own_part.shape[-1], device=DEV)
        own_part = own_part.masked_fill((j > position[..., None])[:, None, None], -math.inf)
        shared = shared.view(h, n, g, most, -1).transpose(0, 1)                       # [n, h, g, most, prefix]
        peak = torch.maximum(shared.amax(-1, keepdim=True), own_part.amax(-1, keepdim=True))
        shared, own_part = (shared - peak).exp(), (own_part - peak).exp()
        total = shared.sum(-1, keepdim=True) + own_part.sum(-1, keepdim=True)
        o = (shared.transpose(0, 1).reshape(h, n * g * most, -1) @ _cells(lead, d, 1)).view(h, n, g, most, d).transpose(0, 1)
        o = o + (own_part.reshape(n, h, g * most, -1) @ _cells(tail, d, 1)).view(n, h, g, most, d)
        o = (o / total).permute(0, 3, 1, 2, 4).reshape(n, most, h * g, d)
        out[token:token + rows] = o[here].to(torch.bfloat16) if min(counts) < most else o.flatten(0, 1).to(torch.bfloat16)
        token += rows
    return out


# ------------------------------------------------------------------ exact

def exact(case, seed):
    """What run() returns, in 64 bits from the definitions, one row of pages at a time."""
    op = case["op"]
    if op == "select":
        return None   # whole numbers
    s = prepare(case, seed)
    if op == "bounds":
        return _exact_bounds(s)
    c = s["case"]
    d, h = c["d"], c["hkv"]
    g = c["hq"] // h
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    if op == "sparse":
        lens = s["lens"].tolist()
        pages = -(-s["lens"] // c["block"])
        for t in range(len(lens)):
            ids = s["tables"][t, :, :int(pages[t])].long()
            for head in range(h):
                out[t, head * g:(head + 1) * g] = _exact_rows(s["q"][t:t + 1, head * g:(head + 1) * g], s["cache"][ids[head], head], lens[t] - 1, lens[t], d)[0]
        return out
    # as if nothing were shared
    cu, ends = s["cu"].tolist(), s["ends"].tolist()
    for r, end in enumerate(ends):
        ids = s["table"][r, :-(-end // c["block"])].long()
        for head in range(h):
            rows = slice(cu[r], cu[r + 1])
            out[rows, head * g:(head + 1) * g] = _exact_rows(s["q"][rows, head * g:(head + 1) * g], s["cache"][ids, head], end - (cu[r + 1] - cu[r]), end, d)
    return out


def _exact_values(raw, d, part):
    """[tokens, D] of one head's tiles [n, 18 D], in 64 bits."""
    codes = raw[:, part * 8 * d:(part + 1) * 8 * d].reshape(-1, d // GROUP, TILE, GROUP // 2)
    para = raw[:, (16 + part) * d:(17 + part) * d].contiguous().view(torch.float16).reshape(-1, d // GROUP, TILE, 2).double()
    x = torch.empty(*codes.shape[:-1], GROUP, dtype=torch.float64, device=DEV)
    x[..., 0::2], x[..., 1::2] = (codes % 16).double(), (codes // 16).double()
    x = (x - para[..., 1:2]) * para[..., 0:1]
    return x.transpose(1, 2).reshape(-1, d)


def _exact_rows(q, pages, first, end, d):
    """Attention of queries [n, g, D] at positions first, first + 1, ... over the first `end` tokens of pages [P, tiles, 18 D]."""
    raw = pages.reshape(-1, 18 * d)
    k, v = _exact_values(raw, d, 0)[:end], _exact_values(raw, d, 1)[:end]
    w = torch.einsum("tgd,jd->gtj", q.double(), k) / math.sqrt(d)
    hidden = torch.arange(end, device=DEV)[None] > first + torch.arange(q.shape[0], device=DEV)[:, None]
    return torch.einsum("gtj,jd->tgd", torch.softmax(w.masked_fill(hidden[None], -math.inf), -1), v)


def _exact_bounds(s):
    c = s["case"]
    d, b = c["d"], c["block"]
    step = torch.zeros(s["bounds"].shape[0], c["hkv"], d // GROUP, dtype=torch.float64, device=DEV)
    at = s["slots"][s["slots"] % b == b - 1] // b
    chunk = max(1, (1 << 27) // (c["hkv"] * b * d))
    for i in range(0, at.numel(), chunk):
        page = at[i:i + chunk]
        k = _exact_values(s["cache"][page].reshape(-1, 18 * d), d, 0).view(page.numel(), c["hkv"], b, d // GROUP, GROUP)
        step[page] = k.abs().amax((2, 4)) * STEP
    return {"high": None, "low": None, "step": step}   # whole numbers, and what they are whole numbers of
