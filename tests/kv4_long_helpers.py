"""Plain references of the operators for long contexts in the 4-bit cache, in
binary64, or by the formula's binary32 steps one by one in numpy; and problems
for them."""
import numpy as np

from tests import kv4_helpers as ref

F = np.float32
POISON = np.array([0x7E00, 0xFC00, 0x7C00, 0x7BFF], np.uint16)   # NaN, -inf, inf, the largest


def fill(c, rng, slot, spread=1.0):
    """Random keys and values of every head into a slot."""
    for part in (0, 1):
        for h in range(c.H):
            s = rng.uniform(0.02, 0.3, c.D // 64) * spread ** rng.uniform(-1, 1)
            c.put(part, slot, h, rng.integers(0, 16, c.D).astype(np.uint8), s.astype(np.float16),
                  rng.integers(0, 16, c.D // 64))


def poisoned(blocks, Hkv, bs, D, rng):
    """A cache whose parameters are NaN, infinite or huge everywhere."""
    c = ref.Cache(blocks, Hkv, bs, D, 0xFF)
    par = c.raw[..., 16 * D:].view(np.uint16)
    par[...] = POISON[rng.integers(0, 4, par.shape)]
    return c


def grouped(torch, groups, Hq, Hkv, D, bs, seed, gap=0, spread=1.0, wide=True):
    """Requests in groups [(prefix, [(past, new), ...]), ...]: the first
    prefix // bs pages of a group's requests are the same ones.  `wide`: a table
    for so much cache that sharing is worth while by its width."""
    rng = np.random.default_rng(seed)
    ends = [p + past + n for p, members in groups for past, n in members]
    new = [n for _, members in groups for _, n in members]
    blocks = sum(-(-e // bs) for e in ends) + 3
    c = poisoned(blocks, Hkv, bs, D, rng)
    ids = list(rng.permutation(blocks))
    width = max(-(-e // bs) for e in ends) + 2
    if wide:
        width = max(width, (65 << 20) // (len(ends) * bs * Hkv * 18 * D // 16) + 1)
    table = np.full((len(ends), width), -1)
    b, borders = 0, [0]
    for prefix, members in groups:
        lead = [ids.pop() for _ in range(prefix // bs)]
        for j in range(len(lead) * bs):
            fill(c, rng, int(lead[j // bs]) * bs + j % bs, spread)
        for _ in members:
            more = [ids.pop() for _ in range(-(-ends[b] // bs) - len(lead))]
            table[b, :len(lead) + len(more)] = lead + more
            for j in range(len(lead) * bs, ends[b]):
                fill(c, rng, int(table[b, j // bs]) * bs + j % bs, spread)
            b += 1
        borders.append(b)
    cu = np.concatenate([[0], np.cumsum(new)])
    q = ref.bf16(rng.normal(0, 1, (cu[-1] + gap, Hq, D)))
    i32 = dict(dtype=torch.int32, device="cuda")
    dev = dict(q=torch.tensor(q, device="cuda").to(torch.bfloat16), cache=torch.tensor(c.raw, device="cuda"),
               block_table=torch.tensor(table, **i32), seq_lens=torch.tensor(ends, **i32), cu_new=torch.tensor(cu, **i32),
               prefix_lens=torch.tensor([p // bs * bs for p, _ in groups], **i32), cu_groups=torch.tensor(borders, **i32))
    return dev, (q, c, table, ends, cu)


def scratch(w4, dev):
    Hkv, D = dev["cache"].shape[1], dev["q"].shape[2]
    return w4.kv4_prefix_attention_scratch(dev["q"].shape[0], dev["seq_lens"].numel(), dev["prefix_lens"].numel(),
                                           dev["q"].shape[1], Hkv, D)


def check(w4, out, want, tol):
    got = out.double().cpu().numpy()
    assert np.isfinite(got).all()
    bad = np.abs(got - want) > tol
    assert not bad.any(), "%d of %d off, first %s: %r, want %r +- %r" % (
        bad.sum(), bad.size, np.argwhere(bad)[0], got[bad][0], want[bad][0], tol[bad][0])
    assert w4.w4a16_check_device_error() == 0


def bounds(c, block):
    """high, low [H, D] and steps [H, D / 64] of a page."""
    high, low, step = np.zeros((c.H, c.D), np.int64), np.zeros((c.H, c.D), np.int64), np.zeros((c.H, c.D // 64), F)
    for h in range(c.H):
        v = np.array([c.values(0, block * c.bs + i, h) for i in range(c.bs)], F)
        hi, lo = v.max(0).reshape(-1, 64), v.min(0).reshape(-1, 64)
        step[h] = np.maximum(np.abs(hi), np.abs(lo)).max(-1) * F(65 / 8192)
        by = np.where(step[h] > 0, step[h], F(1))[:, None]
        high[h], low[h] = np.ceil(hi / by).reshape(-1), np.floor(lo / by).reshape(-1)
    return high, low, step


def packed_bounds(rng, blocks, H, D):
    """Bounds of made-up pages as the library lays them out."""
    a, b = rng.integers(-127, 128, (2, blocks, H, D)).astype(np.int8)
    raw = np.zeros((blocks, H, 2 * D + 16), np.uint8)
    raw[..., :D], raw[..., D:2 * D] = np.maximum(a, b).view(np.uint8), np.minimum(a, b).view(np.uint8)
    raw[..., 2 * D:] = rng.uniform(0.01, 0.03, (blocks, H, 4)).astype(F).view(np.uint8)
    return raw


def scores(q, raw, ids, h):
    """Scores [pages] of head rows q [G, D] (binary32) against pages `ids` of
    key head h; -inf for ids outside the cache."""
    D = q.shape[1]
    q = np.clip(np.where(np.isnan(q), F(0), q), F(-3.3895314e38), F(3.3895314e38)).astype(F)
    with np.errstate(over="ignore", invalid="ignore"):
        u = np.abs(q).max(-1) * F(65 / 8192)
        c = np.rint(q / np.where(u > 0, u, F(1))[:, None]).astype(np.int64)
        out = np.full(len(ids), -np.inf, F)
        for i, page in enumerate(ids):
            if not 0 <= page < raw.shape[0]:
                continue
            row = raw[page, h]
            high, low = row[:D].view(np.int8).astype(np.int64), row[D:2 * D].view(np.int8).astype(np.int64)
            step = row[2 * D:].view(F)[:D // 64]
            dot = (c * np.where(c > 0, high, low)).reshape(len(q), -1, 64).sum(-1)
            t = dot.astype(F) * step
            while t.shape[1] > 1:
                t = t[:, 0::2] + t[:, 1::2]
            out[i] = np.fmax.reduce(t[:, 0] * u, initial=-np.inf)
    return out


def select(q, raw, table, seq_lens, cu, bs, top, first, recent):
    """tables [T, H, top], lens [T] by the definition."""
    T, H, blocks = q.shape[0], raw.shape[1], raw.shape[0]
    G = q.shape[1] // H
    tables, lens = np.full((T, H, top), -1), np.zeros(T, np.int64)
    for b in range(len(seq_lens)):
        for t in range(int(cu[b]), int(cu[b + 1])):
            p = min(int(seq_lens[b]) - int(cu[b + 1]) + t, table.shape[1] * bs - 1)
            if p < 0:
                continue
            seen = p // bs + 1
            n = min(seen, top)
            lens[t] = (n - 1) * bs + p % bs + 1
            for h in range(H):
                if seen <= top:
                    pages = list(range(seen))
                else:
                    middle = list(range(first, seen - recent))
                    s = scores(q[t, h * G:(h + 1) * G], raw, table[b, middle], h)
                    best = sorted(middle, key=lambda i: (-s[i - first], i))[:top - first - recent]
                    pages = list(range(first)) + sorted(best) + list(range(seen - recent, seen))
                ids = table[b, pages]
                tables[t, h, :n] = np.where((ids >= 0) & (ids < blocks), ids, -1)
    return tables, lens


def sparse(q, c, tables, lens, scale):
    """Attention over the tables' pages, and its bound, as kv4_helpers.attention."""
    out, tol = np.zeros(q.shape), np.zeros(q.shape)
    G = q.shape[1] // c.H
    for h in range(c.H):
        part = ref.Cache.__new__(ref.Cache)
        part.blocks, part.H, part.bs, part.D = c.blocks, 1, c.bs, c.D
        part.raw = c.raw[:, h:h + 1]
        rows = slice(h * G, (h + 1) * G)
        # a token is a request of one new token
        out[:, rows], tol[:, rows] = ref.attention(q[:, rows], part, tables[:, h], lens, np.arange(len(lens) + 1), scale)
    return out, tol
