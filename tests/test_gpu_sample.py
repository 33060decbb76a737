"""Sampling: every setting against the definition in binary64, at points whose
answer no binary32 rounding can change, and the exact whole-number rules."""
import numpy as np
import pytest

from tests.gpu_helpers import cuda_or_skip

pytestmark = pytest.mark.gpu


def _kept(logits, T, k, p, minp):
    """Probabilities (binary64, renormalised) of the kept tokens by index."""
    x = np.asarray(logits, np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    m = np.exp(x / T - (x / T).max())
    order = np.argsort(-x, kind="stable")
    w = m[order].copy()
    if k > 0:
        w[k:] = 0
    if p < 1:
        before = np.cumsum(w) - w
        w[~(before < max(p, 0) * w.sum())] = 0
        w[0] = m[order[0]]
    w[w < minp] = 0
    out = np.zeros_like(m)
    out[order] = w
    return out / out.sum()


def _run(torch, w4, logits, u, T=1.0, k=0, p=1.0, minp=0.0, dtype="float32"):
    n = len(u)
    f = lambda v: torch.full((n,), v, dtype=torch.float32, device="cuda")
    x = torch.tensor(np.asarray(logits), dtype=torch.float32).to(getattr(torch, dtype)).cuda()
    x = x[None].expand(n, -1).contiguous()
    out = w4.w4a16_sample(x, torch.tensor(u, dtype=torch.float32, device="cuda"), f(T),
                          torch.full((n,), k, dtype=torch.int32, device="cuda"), f(p), f(minp))
    torch.cuda.synchronize()
    return out.cpu().numpy()


def _sweep(torch, w4, logits, T, k, p, minp, dtype, most=200):
    """u in the middle of every kept token's interval (those wider than 1e-4):
    binary32 exponentials move a boundary by less than 1e-5 for |l / T| < 80."""
    w = _kept(logits, T, k, p, minp)
    edge = np.cumsum(w)
    wide = np.flatnonzero(w > 1e-4)[:most]
    assert len(wide)
    got = _run(torch, w4, logits, (edge - w / 2)[wide], T, k, p, minp, dtype)
    assert np.array_equal(got, wide)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("V", [1, 2, 31, 33, 1000, 4099, 262144])
def test_settings(V, dtype):
    torch, w4 = cuda_or_skip()
    rng = np.random.default_rng(V)
    x = rng.normal(-3, 2.0, V)
    at = rng.integers(0, V, 30)
    x[at] += rng.uniform(5, 12, 30)
    x = torch.tensor(x, dtype=torch.float32).to(getattr(torch, dtype)).float().numpy()
    for T, k, minp in [(1.0, 0, 0.0), (0.7, 0, 0.0), (1.3, 5, 0.0), (1.0, 64, 0.0), (1.0, 0, 0.03), (0.5, 40, 0.01),
                       (1.0, V + 5, 0.0), (1.0, 1, 0.0)]:
        w = _kept(x, T, k, 1.0, 0.0)
        top = np.sort(w)[::-1].cumsum()
        # top-p in the middle of a step of the sorted sums; min-p away from any mass
        ps = [1.0] + [float((top[i] + top[i - 1]) / 2) for i in (1, 3, 10) if i < (w > 0).sum() and w.max() < 0.999 and
                      top[i] - top[i - 1] > 1e-4]
        if minp:
            r = np.sort(w / w.max())
            i = np.searchsorted(r, minp)
            minp = float(r[i] + r[i - 1]) / 2 if 0 < i < V else minp
        for p in ps:
            _sweep(torch, w4, x, T, k, p, minp, dtype)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("V", [300, 5000, 262144])
def test_ties_go_to_the_lower_index(V, dtype):
    # all equal: masses are exact, so every cut falls where whole numbers put it
    torch, w4 = cuda_or_skip()
    x = np.full(V, 1.5)
    u = [0.0, 0.25, 0.5, 0.75, 0.999]
    assert np.array_equal(_run(torch, w4, x, u, dtype=dtype), [int(v * V) for v in np.float32(u).astype(float)])
    assert np.array_equal(_run(torch, w4, x, u, k=100, dtype=dtype), [0, 25, 50, 75, 99])
    # p = 0.5 keeps half of them, the first by index; of the first 100, 50
    assert np.array_equal(_run(torch, w4, x, [0.0, 0.5, 0.999999], p=0.5, dtype=dtype),
                          [0, V // 4, int(np.float64(np.float32(0.999999)) * (V // 2))])
    assert np.array_equal(_run(torch, w4, x, [0.0, 0.5, 0.99], k=100, p=0.5, dtype=dtype), [0, 25, 49])
    assert np.array_equal(_run(torch, w4, x, u, T=0.0, dtype=dtype), [0] * 5)
    # ties at the cut of top-k only: two above it, the rest equal
    x[[V - 1, 7]] = 4.0
    got = _run(torch, w4, x, np.linspace(0, 0.9999, 400), k=5, dtype=dtype)
    assert set(got) == {0, 1, 2, 7, V - 1}


@pytest.mark.parametrize("V", [50, 9000])
def test_signed_zeros_are_equal(V):
    torch, w4 = cuda_or_skip()
    x = np.zeros(V)
    x[::2] = -0.0
    x[3:] -= 40
    assert np.array_equal(_run(torch, w4, x, [0.1, 0.4, 0.9], k=2), [0, 0, 1])
    assert np.array_equal(_run(torch, w4, x, [0.1], T=0.0), [0])


def test_edge_numbers():
    torch, w4 = cuda_or_skip()
    x = np.array([0.5, -1.0, 2.0, 0.0, 1.0])
    # u of one or more gives the last kept token, a negative one or NaN the first
    assert np.array_equal(_run(torch, w4, x, [1.0, 7.0, -1.0, float("nan")]), [4, 4, 0, 0])
    # p of zero or less keeps the first in order
    assert np.array_equal(_run(torch, w4, x, [0.0, 0.99], p=0.0), [2, 2])
    assert np.array_equal(_run(torch, w4, x, [0.0, 0.99], p=-3.0), [2, 2])
    assert np.array_equal(_run(torch, w4, x, [0.99], k=-4), [4])
    # min-p of one keeps the largest
    assert np.array_equal(_run(torch, w4, x, [0.0, 0.99], minp=1.0), [2, 2])
    # a temperature that overflows the quotient is greedy; a negative one and NaN too
    for T in (1e-42, -1.0, float("nan"), 0.0):
        assert np.array_equal(_run(torch, w4, x, [0.9], T=T), [2])


@pytest.mark.parametrize("V", [40, 3000, 100000])
def test_infinite_nan_and_masked_logits(V):
    torch, w4 = cuda_or_skip()
    u = np.linspace(0, 0.999, 50)
    x = np.full(V, -np.inf)
    assert np.array_equal(_run(torch, w4, x, u), [-1] * 50)
    assert np.array_equal(_run(torch, w4, x, u, T=0.0), [-1] * 50)
    assert np.array_equal(_run(torch, w4, np.full(V, np.nan), u, k=3, p=0.5), [-1] * 50)
    x[V - 2] = -3.0   # one token left by the mask
    assert np.array_equal(_run(torch, w4, x, u, k=7, p=0.9), [V - 2] * 50)
    x[:] = torch.finfo(torch.float32).min   # masked with the lowest value
    x[5] = 0.0
    assert np.array_equal(_run(torch, w4, x, u), [5] * 50)
    x = np.where(np.arange(V) % 3 == 0, np.nan, 0.0)
    got = _run(torch, w4, x, u, k=20)
    assert set(got) <= set([i for i in range(V) if i % 3][:20])
    x[11], x[7] = np.inf, np.inf
    assert np.array_equal(_run(torch, w4, x, u), [7] * 50)


def test_rows_do_not_touch_each_other_and_strides():
    torch, w4 = cuda_or_skip()
    g = torch.Generator().manual_seed(2)
    for dtype in (torch.float32, torch.bfloat16):
        wide = (torch.randn(40, 5007, generator=g) * 3).to(dtype).cuda()
        x = wide[:, 3:5004]     # rows that start at odd addresses
        u = torch.rand(40, generator=g).cuda()
        T = torch.linspace(0.2, 2, 40).cuda()
        k = torch.randint(0, 90, (40,), generator=g, dtype=torch.int32).cuda()
        p = torch.rand(40, generator=g).cuda()
        m = (torch.rand(40, generator=g) * 0.1).cuda()
        all_rows = w4.w4a16_sample(x, u, T, k, p, m)
        for r in range(0, 40, 7):
            one = w4.w4a16_sample(x[r:r + 1].contiguous(), u[r:r + 1], T[r:r + 1].clone(), k[r:r + 1].clone(),
                                  p[r:r + 1].clone(), m[r:r + 1].clone())
            assert int(one) == int(all_rows[r])
        # settings left out are off
        off = w4.w4a16_sample(x, u)
        same = w4.w4a16_sample(x, u, torch.ones_like(u), torch.zeros_like(k), torch.ones_like(u), torch.zeros_like(u))
        assert torch.equal(off, same)
    assert w4.w4a16_sample(x[:0], u[:0]).numel() == 0


@pytest.mark.parametrize("V", [700, 262144])
def test_whole_number_rules_on_many_rows(V):
    # masses from binary32 exponentials, everything after them in whole numbers
    torch, w4 = cuda_or_skip()
    R = 60
    g = torch.Generator(device="cuda").manual_seed(V)
    x = (torch.randn(R, V, device="cuda", generator=g) * 2).to(torch.bfloat16)
    u = torch.rand(R, device="cuda", generator=g)
    T = 0.3 + torch.rand(R, device="cuda", generator=g)
    k = torch.randint(1, 200, (R,), device="cuda", generator=g, dtype=torch.int32)
    p = 0.5 + 0.5 * torch.rand(R, device="cuda", generator=g)
    got = w4.w4a16_sample(x, u, T, k, p).long()
    f = x.float()
    q = f / T[:, None]
    mass = ((q - q.amax(-1, keepdim=True)).exp().double() * 2.0 ** 40).round().long()
    v, order = torch.sort(f, dim=-1, descending=True, stable=True)
    o = mass.gather(1, order) * (torch.arange(V, device="cuda")[None] < k[:, None])
    before = o.cumsum(-1) - o
    goal = (o.sum(-1).double() * p.double()).long().clamp(min=1)
    o = o * (before < goal[:, None])
    kept = torch.zeros_like(mass).scatter_(1, order, o)
    tot = kept.sum(-1)
    # the chosen token is kept, and u lies in its interval (an exponential that
    # is an ulp off moves the edges by less than 2^-20 of the sum)
    m = kept.gather(1, got[:, None])[:, 0]
    hi = kept.cumsum(-1).gather(1, got[:, None])[:, 0]
    pos = u.double() * tot.double()
    slack = tot.double() * 2.0 ** -20
    assert (m > 0).all()
    assert ((hi - m).double() <= pos + slack).all() and (pos <= hi.double() + slack).all()
