"""What is measured of the 4-bit key/value cache, the attention over it and the sampler: cases, inputs and plain forms.

The operators are those of a decode step around the quantised linears:

* plan       block tables, positions and cache slots from the requests' lengths (kv4_plan);
* norm_rope  RMS norm of every query and key head with the position rotation (w4a16_qk_norm_rope);
* append     keys and values quantised to 4 bits into their cache slots, and read back (kv4_append, kv4_gather);
* attention  attention over the paged 4-bit cache, with a sliding window and first tokens that stay visible
             (kv4_attention);
* sample     temperature, top-k, top-p and min-p from given uniform numbers (w4a16_sample).

`own` chooses between the plain forms (elementary torch operations in 32 bits) and the library's kernels.

The cache is uint8 [blocks, kv heads, block / 16, 18 D]: tiles of 16 tokens x D elements, each holding the codes of K
[D / 64, 16, 32] (two per byte, the even element in the low nibble), those of V, then (scale, zero) in binary16 of K
[D / 64, 16, 2] and of V.  A value is (code - zero) * scale, with one scale and zero for 64 elements of a token's head.
"""
import math

import torch

own = False

DEV = "cuda"
GROUP = 64   # elements of a head that share a scale and a zero point
TILE = 16    # tokens of a cache tile
UNIT = 2.0 ** 40   # integer mass of the most likely token in the sampler


# ------------------------------------------------------------------ cases

def listed():
    heads = {"hq": 16, "hkv": 8, "d": 256}
    return [
        # the tables of one decode step of a served batch: launch latency is all there is
        {"name": "plan decode", "op": "plan", "requests": 64, "ctx_lo": 1, "ctx_hi": 8000, "new_lo": 1, "new_hi": 1, "block": 16},
        # a step that mixes decoding requests with long prompt pieces
        {"name": "plan mixed", "op": "plan", "requests": 511, "ctx_lo": 1, "ctx_hi": 120000, "new_lo": 1, "new_hi": 1000, "block": 32},
        # one token of one request, the model's 16 query and 8 key heads of 256
        {"name": "norm rope token", "op": "norm_rope", "tokens": 1, **heads, "rot": 256, "interleaved": False},
        # a prompt piece with another head layout: grouped by four, interleaved pairs
        {"name": "norm rope prompt", "op": "norm_rope", "tokens": 4099, "hq": 32, "hkv": 8, "d": 128, "rot": 128, "interleaved": True},
        # a decode step of 64 requests into the cache
        {"name": "append decode", "op": "append", "tokens": 64, **heads, "block": 16},
        # a long prompt into the cache, ending inside a page
        {"name": "append prompt", "op": "append", "tokens": 8191, **heads, "block": 64},
        # one request's decode step over a cache of ordinary length: split over the length, or nothing runs in parallel
        {"name": "attention one", "op": "attention", "requests": 1, "ctx_lo": 8200, "ctx_hi": 8200, "new_lo": 1, "new_hi": 1, **heads, "block": 16, "window": 0, "sinks": 0},
        # a served batch, lengths spread over two decades, in a layer that sees everything
        {"name": "attention ragged", "op": "attention", "requests": 64, "ctx_lo": 255, "ctx_hi": 32767, "new_lo": 1, "new_hi": 1, **heads, "block": 64, "window": 0, "sinks": 0},
        # the same step in a sliding-window layer of 1024 with four first tokens kept
        {"name": "attention window", "op": "attention", "requests": 128, "ctx_lo": 500, "ctx_hi": 20000, "new_lo": 1, "new_hi": 1, **heads, "block": 16, "window": 1024, "sinks": 4},
        # prompt pieces that attend to their own past in the cache
        {"name": "attention prompt", "op": "attention", "requests": 3, "ctx_lo": 1, "ctx_hi": 6000, "new_lo": 701, "new_hi": 4096, **heads, "block": 64, "window": 0, "sinks": 0},
        # one row of logits of the 262144-token vocabulary
        {"name": "sample one", "op": "sample", "rows": 1, "vocab": 262144, "dtype": "bfloat16"},
        # a batch, each row with its own settings
        {"name": "sample batch", "op": "sample", "rows": 128, "vocab": 262144, "dtype": "bfloat16"},
    ]


def draw(rng):
    def log_int(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    hq, hkv = rng.choice([(16, 8), (32, 8), (8, 1), (12, 12), (28, 4), (20, 10), (64, 4)])
    heads = {"hq": hq, "hkv": hkv, "d": rng.choice([64, 128, 256, 256])}
    block = rng.choice([16, 32, 64, 128])
    op = rng.choice(["plan", "norm_rope", "append", "attention", "attention", "prompt", "sample"])
    if op == "plan":
        n = log_int(1, 511)
        return {"op": op, "requests": n, "ctx_lo": 1, "ctx_hi": log_int(20, 120000), "new_lo": 1, "new_hi": log_int(1, 1000), "block": block}
    if op in ("norm_rope", "append"):
        d = heads["d"]
        c = {"op": op, "tokens": log_int(1, 8191 if d * (hq + hkv) <= 6144 else 3000), **heads}
        return dict(c, block=block) if op == "append" else dict(c, rot=rng.choice([d, d, d // 2]), interleaved=rng.random() < 0.4)
    if op == "attention":
        n = log_int(1, 64)
        room = min(32767, 900000 // (n * max(1, hkv // 8)))
        hi = log_int(100, room)
        window = rng.choice([0, 0, rng.randint(1, 1500)])
        return {"op": "attention", "requests": n, "ctx_lo": max(1, hi // 20), "ctx_hi": hi, "new_lo": 1, "new_hi": rng.choice([1, 1, 1, 3]), **heads, "block": block, "window": window, "sinks": rng.choice([0, 4, 17]) if window else 0}
    if op == "prompt":
        window = rng.choice([0, 0, rng.randint(100, 1500)])
        new = log_int(30, 1500)
        return {"op": "attention", "requests": rng.randint(1, 3), "ctx_lo": 1, "ctx_hi": log_int(2, 5000), "new_lo": max(1, new // 3), "new_hi": new, **heads, "block": block, "window": window, "sinks": rng.choice([0, 4, 17]) if window else 0}
    return {"op": "sample", "rows": log_int(1, 128), "vocab": log_int(1000, 262144), "dtype": rng.choice(["bfloat16", "bfloat16", "float32"])}


def _spread(lo, hi, n, turn):
    """n whole numbers from lo to hi, spread evenly over their logarithm in a fixed scattered order; the ends are among
    them."""
    if n == 1:
        return [hi]
    step = next(s for s in (turn, turn + 2, turn + 4, 1) if math.gcd(s, n) == 1)
    return [int(round(math.exp(math.log(lo) + (math.log(hi) - math.log(lo)) * ((i * step) % n) / (n - 1)))) for i in range(n)]


def _lengths(case):
    """Tokens in the cache before the step, and new ones, for each request: of the case alone."""
    n = case["requests"]
    return _spread(case["ctx_lo"], case["ctx_hi"], n, 7), _spread(case["new_lo"], case["new_hi"], n, 11)


def _pairs(case):
    """(query, key) pairs that are visible, and cache tokens that any query of a request sees, over all requests."""
    pairs = tokens = 0
    w, s = case["window"], case["sinks"]
    for c, n in zip(*_lengths(case)):
        end = c + n
        if w <= 0:
            pairs += n * c + n * (n + 1) // 2
            tokens += end
            continue
        for p in range(c, end):
            low = max(0, p - w + 1)
            pairs += p + 1 - low + min(s, low)
        low = max(0, c - w + 1)
        tokens += end - low + min(s, low)
    return pairs, tokens


def work(case):
    op = case["op"]
    if op == "plan":
        b = case["block"]
        ctx, new = _lengths(case)
        t = sum(new)
        blocks = sum(-(-(c + n) // b) - -(-c // b) for c, n in zip(ctx, new))
        return {"bytes": 4 * (4 * len(ctx) + 2) + 12 * t + 8 * blocks, "flops": 0}
    if op == "sample":
        n = case["rows"] * case["vocab"]
        return {"bytes": n * (2 if case["dtype"] == "bfloat16" else 4) + 24 * case["rows"], "flops": 4 * n}
    hq, hkv, d = case["hq"], case["hkv"], case["d"]
    cell = 2 * (d // 2 + d // GROUP * 4)   # bytes of a token's key and value in one head
    if op == "attention":
        pairs, tokens = _pairs(case)
        return {"bytes": tokens * hkv * cell + 4 * sum(_lengths(case)[1]) * hq * d, "flops": 4 * pairs * hq * d}
    t = case["tokens"]
    if op == "norm_rope":
        return {"bytes": t * (4 * (hq + hkv) * d + 4 * case["rot"] + 4) + 4 * d, "flops": 8 * t * (hq + hkv) * d}
    # bfloat16 in, cells out, cells in, bfloat16 out
    return {"bytes": t * (2 * 4 * hkv * d + 2 * hkv * cell + 16), "flops": 12 * t * hkv * d}


# ----------------------------------------------------------------- inputs

def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return {"plan": _prepare_plan, "sample": _prepare_sample, "attention": _prepare_attention}.get(case["op"], _prepare_rope)(case, g)


def _prepare_plan(case, g):
    b = case["block"]
    ctx, new = _lengths(case)
    held = [-(-c // b) for c in ctx]
    more = sum(-(-(c + n) // b) - h for c, n, h in zip(ctx, new, held))
    width = max(-(-(c + n) // b) for c, n in zip(ctx, new)) + 3
    ids = torch.randperm(sum(held) + more + 50, device=DEV, generator=g).to(torch.int32)
    order = torch.randperm(len(ctx), device=DEV, generator=g)
    table = torch.full((len(ctx), width), -1, dtype=torch.int32, device=DEV)
    held_t = _i32(held)[order]
    at = torch.arange(width, device=DEV)[None] < held_t[:, None]
    table[at] = ids[:sum(held)]
    return {"case": case, "ctx": _i32(ctx)[order].contiguous(), "new": _i32(new)[order].contiguous(), "table": table,
            "free": ids[sum(held):].contiguous(), "tokens": sum(new)}


def _rope_table(positions, rot):
    i = torch.arange(rot // 2, device=DEV, dtype=torch.float64)
    a = torch.arange(positions, device=DEV, dtype=torch.float64)[:, None] * 10000.0 ** (-2 * i / rot)
    return torch.cat([a.cos(), a.sin()], 1).float().contiguous()


def _prepare_rope(case, g):
    t, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
    # one row of q | k | v for a token, as a fused projection writes it
    qkv = (torch.randn(t, (hq + 2 * hkv) * d, device=DEV, generator=g) * 1.5).to(torch.bfloat16)
    s = {"case": case, "q": qkv[:, :hq * d].view(t, hq, d), "k": qkv[:, hq * d:(hq + hkv) * d].view(t, hkv, d)}
    if case["op"] == "norm_rope":
        rows = 16384
        s["cos_sin"] = _rope_table(rows, case["rot"])
        s["positions"] = torch.randint(0, rows, (t,), device=DEV, generator=g, dtype=torch.int32)
        for name in ("wq", "wk"):
            s[name] = (1 + 0.2 * torch.randn(d, device=DEV, generator=g)).to(torch.bfloat16)
        s["q_out"] = torch.empty(t, hq, d, dtype=torch.bfloat16, device=DEV)
        s["k_out"] = torch.empty(t, hkv, d, dtype=torch.bfloat16, device=DEV)
        return s
    b = case["block"]
    blocks = -(-t // b) + 2
    s["v"] = qkv[:, (hq + hkv) * d:].view(t, hkv, d)
    # pages in any order, tokens of a page in order; the first ones start inside a page
    pages = torch.randperm(blocks, device=DEV, generator=g)
    at = torch.arange(t, device=DEV) + 5
    s["slots"] = pages[at // b] * b + at % b
    s["cache"] = torch.zeros(blocks, hkv, b // TILE, 18 * d, dtype=torch.uint8, device=DEV)
    s["k_back"] = torch.empty(t, hkv, d, dtype=torch.bfloat16, device=DEV)
    s["v_back"] = torch.empty_like(s["k_back"])
    return s


def _prepare_attention(case, g):
    hq, hkv, d, b = case["hq"], case["hkv"], case["d"], case["block"]
    ctx, new = _lengths(case)
    ends = [c + n for c, n in zip(ctx, new)]
    held = [-(-e // b) for e in ends]
    blocks = sum(held) + 1
    ids = torch.randperm(blocks, device=DEV, generator=g).to(torch.int32)
    table = torch.full((len(ctx), max(held) + 1), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(max(held) + 1, device=DEV)[None] < _i32(held)[:, None]] = ids[:sum(held)]
    # codes and parameters as quantised normal values have them: a bell over the 16 codes, zeros near the middle
    tiles = blocks * hkv * (b // TILE)
    cache = torch.empty(tiles, 18 * d, dtype=torch.uint8, device=DEV)
    two = torch.tensor([1, 2, 4, 7, 12, 19, 26, 31, 33, 31, 26, 19, 12, 7, 4, 2], device=DEV)
    level = torch.repeat_interleave(torch.arange(16, device=DEV, dtype=torch.uint8), two)
    level = torch.cat([level, torch.full((256 - level.numel(),), 8, dtype=torch.uint8, device=DEV)])
    pair = (level[:, None] | (level[None] << 4)).reshape(-1)
    step = max(1, (1 << 28) // (16 * d))
    i = 0
    while i < tiles:   # in pieces: the random words of the codes take more room than the codes
        n = min(step, tiles - i)
        cache[i:i + n, :16 * d] = pair[torch.randint(0, 65536, (n, 16 * d), device=DEV, generator=g, dtype=torch.int32)]
        i += n
    scale = (0.25 + 0.2 * torch.rand(tiles, 2, d // GROUP, TILE, device=DEV, generator=g)).half()
    zero = torch.randint(6, 10, scale.shape, device=DEV, generator=g).half()
    cache[:, 16 * d:] = torch.stack([scale, zero], -1).reshape(tiles, -1).view(torch.uint8)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    q = torch.randn(cu[-1], hq, d, device=DEV, generator=g).to(torch.bfloat16)
    return {"case": case, "q": q, "cache": cache.view(blocks, hkv, b // TILE, 18 * d), "table": table, "ends": _i32(ends), "cu": _i32(cu),
            "longest": max(ends), "most": max(new), "out": torch.empty_like(q)}


def _prepare_sample(case, g):
    n, v = case["rows"], case["vocab"]
    # logits of a model: a wide bulk and a few that stand out
    x = 2.2 * torch.randn(n, v, device=DEV, generator=g) - 4
    x.scatter_add_(1, torch.randint(0, v, (n, 40), device=DEV, generator=g), 9 * torch.rand(n, 40, device=DEV, generator=g) + 2)
    r = torch.arange(n, device=DEV)
    # settings by row: plain sampling, top-k and top-p, min-p, a cool and a greedy row
    kind = r % 5
    return {"case": case, "logits": x.to(getattr(torch, case["dtype"])), "u": torch.rand(n, device=DEV, generator=g),
            "temperature": torch.where(kind == 4, 0.0, torch.where(kind == 3, 0.6, 1.0)),
            "top_k": torch.where((kind == 0) | (kind == 3), 64, 0).to(torch.int32),
            "top_p": torch.where((kind == 0) | (kind == 1), 0.92, 1.0), "min_p": torch.where((kind == 2) | (kind == 3), 0.02, 0.0),
            "tokens": torch.empty(n, dtype=torch.int32, device=DEV)}


# -------------------------------------------------------------------- run

def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import gemm_w4a16_gemv_gb300 as w4
    c = s["case"]
    op = c["op"]
    if op == "plan":
        if "buffers" not in s:   # a serving loop keeps its step's buffers
            s["buffers"] = w4.kv4_plan_buffers(c["requests"], s["tokens"], device=DEV)
        p = w4.kv4_plan(s["ctx"], s["new"], s["table"], s["free"], c["block"], out=s["buffers"])
        return {"seq_lens": p.seq_lens, "cu_new": p.cu_new, "positions": p.positions, "slots": p.slots, "taken": p.taken, "table": s["table"]}
    if op == "norm_rope":
        q, k = w4.w4a16_qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], s["cos_sin"], s["positions"], q_out=s["q_out"], k_out=s["k_out"],
                                     interleaved=c["interleaved"])
        return {"q": q, "k": k}
    if op == "append":
        w4.kv4_append(s["k"], s["v"], s["cache"], s["slots"])
        k, v = w4.kv4_gather(s["cache"], s["slots"], k=s["k_back"], v=s["v_back"])
        return {"k": k, "v": v}
    if op == "attention":
        if "scratch" not in s:   # kept by the user's program between calls
            s["scratch"] = w4.kv4_attention_scratch(c["hq"], c["hkv"], c["d"], device=DEV)
        return w4.kv4_attention(s["q"], s["cache"], s["table"], s["ends"], s["cu"], out=s["out"], scratch=s["scratch"], scale=c["d"] ** -0.5,
                                window=c["window"], sinks=c["sinks"], max_new=s["most"])
    return w4.w4a16_sample(s["logits"], s["u"], s["temperature"], s["top_k"], s["top_p"], s["min_p"], out=s["tokens"])


def _run_plain(s):
    return {"plan": _plain_plan, "norm_rope": _plain_norm_rope, "append": _plain_append, "attention": _plain_attention,
            "sample": _plain_sample}[s["case"]["op"]](s)


def _plain_plan(s):
    b, ctx, new, table, free = s["case"]["block"], s["ctx"], s["new"], s["table"], s["free"]
    t = s["tokens"]
    ends = ctx + new
    held = (ctx + b - 1) // b
    need = (ends + b - 1) // b - held
    cu = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0, dtype=torch.int32)])
    first = need.cumsum(0, dtype=torch.int32) - need          # place in the free list of a request's first new block
    column = torch.arange(table.shape[1], device=DEV, dtype=torch.int32)[None]
    at = column - held[:, None]
    fresh = (at >= 0) & (at < need[:, None])
    table = torch.where(fresh, free[(first[:, None] + at).clamp(0, free.numel() - 1).long()], table)
    token = torch.arange(t, device=DEV, dtype=torch.int32)
    request = (torch.searchsorted(cu, token, right=True) - 1)
    positions = ctx[request] + token - cu[request]
    slots = table[request, (positions // b).long()].long() * b + positions % b
    return {"seq_lens": ends, "cu_new": cu, "positions": positions, "slots": slots, "taken": need.sum(dtype=torch.int32).reshape(1), "table": table}


def _plain_norm_rope(s):
    c = s["case"]
    half = c["rot"] // 2
    row = s["cos_sin"][s["positions"].long()]
    cos, sin = row[:, None, :half], row[:, None, half:]

    def one(x, w):
        x = x.float()
        x = x * (x.square().mean(-1, keepdim=True) + 1e-6).rsqrt() * w.float()
        r = x[..., :2 * half]
        if c["interleaved"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = r[..., :half], r[..., half:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([r, x[..., 2 * half:]], -1).to(torch.bfloat16)

    return {"q": one(s["q"], s["wq"]), "k": one(s["k"], s["wk"])}


def _quantise(x):
    """Codes [T, H, D], scales and zeros [T, H, D / 64] of the 64-element groups of x."""
    g = x.float().unflatten(-1, (-1, GROUP))
    low, high = g.amin(-1).clamp(max=0), g.amax(-1).clamp(min=0)
    scale = ((high - low) / 15).clamp(max=65504.0).half()
    s = scale.float()
    safe = torch.where(s > 0, s, torch.ones_like(s))
    zero = (-low / safe).round().clamp(0, 15)
    codes = (g / safe[..., None]).round() + zero[..., None]
    codes = codes.clamp(0, 15) * (s > 0)[..., None]
    return codes.flatten(-2).to(torch.uint8), scale, (zero * (s > 0)).half()


def _plain_append(s):
    cache, slots, d = s["cache"], s["slots"], s["case"]["d"]
    b = s["case"]["block"]
    groups = d // GROUP
    block, tile, row = slots // b, slots % b // TILE, slots % TILE
    view = cache.transpose(1, 2)   # [blocks, tiles, heads, bytes]
    col = torch.arange(GROUP // 2, device=DEV)
    group = torch.arange(groups, device=DEV)
    back = []
    for part, x in ((0, s["k"]), (1, s["v"])):
        codes, scale, zero = _quantise(x)
        packed = (codes[..., 0::2] | (codes[..., 1::2] << 4)).unflatten(-1, (groups, GROUP // 2))
        code_at = part * 8 * d + (group[:, None] * TILE + row[:, None, None]) * (GROUP // 2) + col   # [T, groups, 32]
        para_at = (16 + part) * d + (group * TILE + row[:, None]) * 4                                # [T, groups]
        heads = torch.arange(x.shape[1], device=DEV)
        where = (block[:, None, None, None], tile[:, None, None, None], heads[None, :, None, None])
        view[where + (code_at[:, None],)] = packed
        para = torch.stack([scale, zero], -1).view(torch.uint8)      # [T, heads, groups, 4]
        view[where + ((para_at[..., None] + torch.arange(4, device=DEV))[:, None],)] = para
        c = view[where + (code_at[:, None],)]
        p = view[where + ((para_at[..., None] + torch.arange(4, device=DEV))[:, None],)].view(torch.float16).float()
        value = torch.stack([c & 15, c >> 4], -1).flatten(-2).float()
        back.append(((value - p[..., 1:]) * p[..., :1]).flatten(-2).to(torch.bfloat16))
    return {"k": back[0], "v": back[1]}


def _cells(pages, d):
    """K and V as 32-bit values [B, heads, tokens, D] of pages [B, P, heads, tiles, 18 D]."""
    b, p, h, t = pages.shape[:4]
    out = []
    for part in (0, 1):
        codes = pages[..., part * 8 * d:(part + 1) * 8 * d].unflatten(-1, (d // GROUP, TILE, GROUP // 2))
        para = pages[..., (16 + part) * d:(17 + part) * d].contiguous().view(torch.float16).unflatten(-1, (d // GROUP, TILE, 2)).float()
        x = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float()   # [B, P, h, t, groups, 16, 64]
        x = (x - para[..., 1:]) * para[..., :1]
        out.append(x.permute(0, 2, 1, 3, 5, 4, 6).reshape(b, h, p * t * TILE, d))
    return out


def _plain_attention(s):
    c = s["case"]
    d, h, g = c["d"], c["hkv"], c["hq"] // c["hkv"]
    q, ends, cu = s["q"], s["ends"], s["cu"]
    n, most, pages = ends.numel(), s["most"], -(-s["longest"] // c["block"])
    k, v = _cells(s["cache"][s["table"][:, :pages].clamp(min=0).long()], d)
    new = cu[1:] - cu[:-1]
    i = torch.arange(most, device=DEV)
    here = i[None] < new[:, None]                                     # [B, most]
    at = (cu[:-1, None] + i[None]).clamp(max=q.shape[0] - 1).long()
    x = q.float()[at].view(n, most, h, g, d).permute(0, 2, 3, 1, 4).reshape(n, h, g * most, d)
    x = (x * d ** -0.5) @ k.transpose(-1, -2)                         # [B, heads, g most, tokens]
    p = ((ends - new)[:, None] + i)[:, :, None]                       # positions of the queries
    j = torch.arange(k.shape[2], device=DEV)[None, None]
    seen = j <= p
    if c["window"] > 0:
        seen = seen & ((p - j < c["window"]) | (j < c["sinks"]))
    x = x.view(n, h, g, most, -1).masked_fill_(~seen[:, None, None], -math.inf).view(n, h, g * most, -1)
    x -= x.amax(-1, keepdim=True)
    x.exp_()
    o = (x @ v) / x.sum(-1, keepdim=True)
    o = o.view(n, h, g, most, d).permute(0, 3, 1, 2, 4).reshape(n, most, h * g, d)
    return o[here].to(torch.bfloat16)


def _mass(logits, temperature):
    """Whole-number masses of the tokens, 2^40 for the most likely: sums of them do not depend on the order."""
    x = logits.float() / torch.where(temperature > 0, temperature, torch.ones_like(temperature))[:, None]
    return ((x - x.amax(-1, keepdim=True)).exp().double() * UNIT).round().long()


def _plain_sample(s):
    x = s["logits"].float()
    rows, v = x.shape
    mass = _mass(x, s["temperature"])
    value, order = torch.sort(x, dim=-1, descending=True, stable=True)
    rank = torch.arange(v, device=DEV)[None]
    top = torch.where(s["top_k"] > 0, s["top_k"], v)[:, None]
    ordered = mass.gather(1, order) * (rank < top)
    before = ordered.cumsum(-1) - ordered
    # the shortest prefix that holds top_p of what is left
    goal = (ordered.sum(-1, keepdim=True).double() * s["top_p"].clamp(0, 1).double()[:, None]).long().clamp(min=1)
    ordered = ordered * ((before < goal) | (s["top_p"] >= 1)[:, None])
    ordered = ordered * (ordered.double() >= s["min_p"].double()[:, None] * UNIT)
    kept = torch.zeros_like(mass).scatter_(1, order, ordered)
    total = kept.sum(-1, keepdim=True)
    goal = (total.double() * s["u"].double()[:, None]).long().clamp(max=total - 1)
    token = (kept.cumsum(-1) <= goal).sum(-1)
    return torch.where(s["temperature"] > 0, token, order[:, 0]).to(torch.int32)


# ------------------------------------------------------------------ exact

def exact(case, seed):
    """What run() returns, in 64 bits from the definitions, one request and one head group at a time."""
    op = case["op"]
    if op in ("plan", "sample"):
        return None   # whole numbers
    s = prepare(case, seed)
    if op == "norm_rope":
        return {"q": _exact_rope(s, s["q"], s["wq"]), "k": _exact_rope(s, s["k"], s["wk"])}
    if op == "append":
        return {"k": _exact_cells(s["k"]), "v": _exact_cells(s["v"])}
    return _exact_attention(s)


def _exact_rope(s, x, w):
    # a rotation of a pair is a product of complex numbers
    c = s["case"]
    rot = c["rot"]
    x = x.double()
    x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / c["d"] + 1e-6) * w.double()
    at = s["positions"].long()
    turn = torch.complex(s["cos_sin"][at, :rot // 2].double(), s["cos_sin"][at, rot // 2:].double())[:, None]
    out = x.clone()
    if c["interleaved"]:
        z = torch.view_as_complex(x[..., :rot].reshape(*x.shape[:-1], rot // 2, 2).contiguous()) * turn
        out[..., :rot] = torch.view_as_real(z).reshape(*x.shape[:-1], rot)
    else:
        z = torch.complex(x[..., :rot // 2].contiguous(), x[..., rot // 2:rot].contiguous()) * turn
        out[..., :rot // 2], out[..., rot // 2:rot] = z.real, z.imag
    return out


def _exact_cells(x):
    # the nearest of the 16 levels that scale and zero span, found by comparing with all of them; of two as near, the one
    # an even number of steps from zero
    t, h, d = x.shape
    g = x.double().reshape(t * h * (d // GROUP), GROUP)
    low = torch.minimum(g.min(-1).values, g.new_zeros(()))
    high = torch.maximum(g.max(-1).values, g.new_zeros(()))
    scale = ((high - low) / 15).half().double()
    zero = torch.floor(-low / scale + 0.5).clamp(0, 15)
    best, far = torch.zeros_like(g), torch.full_like(g, math.inf)
    for code in range(16):
        steps = (code - zero)[:, None]
        off = (steps * scale[:, None] - g).abs()
        nearer = (off < far) | ((off == far) & (steps % 2 == 0))
        best, far = torch.where(nearer, steps * scale[:, None], best), torch.minimum(off, far)
    return best.reshape(t, h, d)


def _exact_attention(s):
    c = s["case"]
    d, h, b = c["d"], c["hkv"], c["block"]
    g = c["hq"] // h
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    cu, ends = s["cu"].tolist(), s["ends"].tolist()
    for r, end in enumerate(ends):
        pages = s["cache"][s["table"][r, :-(-end // b)].long()]       # [P, heads, tiles, bytes]
        first, last = cu[r], cu[r + 1]
        p = torch.arange(end - (last - first), end, device=DEV)[:, None]
        j = torch.arange(end, device=DEV)[None]
        hidden = (j > p) if c["window"] <= 0 else (j > p) | ((j <= p - c["window"]) & (j >= c["sinks"]))
        for head in range(h):
            kv = []
            for part in (0, 1):
                raw = pages[:, head].reshape(-1, 18 * d)
                codes = raw[:, part * 8 * d:(part + 1) * 8 * d].reshape(-1, d // GROUP, TILE, GROUP // 2)
                para = raw[:, (16 + part) * d:(17 + part) * d].contiguous().view(torch.float16).reshape(-1, d // GROUP, TILE, 2).double()
                x = torch.empty(*codes.shape[:-1], GROUP, dtype=torch.float64, device=DEV)
                x[..., 0::2], x[..., 1::2] = (codes % 16).double(), (codes // 16).double()
                x = (x - para[..., 1:2]) * para[..., 0:1]
                kv.append(x.transpose(1, 2).reshape(-1, d)[:end])
            q = s["q"][first:last, head * g:(head + 1) * g].double()
            w = torch.einsum("tgd,jd->gtj", q, kv[0]) / math.sqrt(d)
            w = torch.softmax(w.masked_fill(hidden[None], -math.inf), -1)
            out[first:last, head * g:(head + 1) * g] = torch.einsum("gtj,jd->tgd", w, kv[1])
    return out
