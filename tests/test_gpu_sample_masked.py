"""Sampling over logits masked with the lowest finite number, where fewer
tokens are left than top-k asks for: every row gets one of the tokens left."""
import numpy as np
import pytest

from tests.gpu_helpers import cuda_or_skip
from tests.test_gpu_sample import _kept

pytestmark = pytest.mark.gpu


def _tokens(torch, w4, x, u, T, k, p):
    n = len(u)
    f = lambda v: torch.full((n,), v, dtype=torch.float32, device="cuda")
    out = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    w4.w4a16_sample(x[None].expand(n, -1).contiguous(), torch.tensor(u, dtype=torch.float32, device="cuda"), f(T),
                    torch.full((n,), k, dtype=torch.int32, device="cuda"), f(p), out=out)
    return out.cpu().numpy()


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("V", [40, 3000, 262144])
@pytest.mark.parametrize("left", [1, 5, 30])
@pytest.mark.parametrize("k", [7, 500])
@pytest.mark.parametrize("T,p", [(1.0, 1.0), (1.0, 0.8), (0.5, 1.0), (1e-4, 0.8), (3.0, 0.8)])
def test_fewer_tokens_left_than_top_k(V, dtype, left, k, T, p):
    torch, w4 = cuda_or_skip()
    low = torch.finfo(getattr(torch, dtype)).min
    x = torch.full((V,), low, dtype=getattr(torch, dtype), device="cuda")
    at = np.random.default_rng(V + left).permutation(V)[:left]
    x[torch.tensor(at, device="cuda")] = torch.tensor(0.5 - 0.25 * np.arange(left), device="cuda").to(x.dtype)
    w = _kept(x.double().cpu().numpy(), T, k, 1.0, 0.0)
    assert np.abs(np.sort(w)[::-1].cumsum() - p).min() > 1e-4 or p == 1.0     # no boundary at p
    w = _kept(x.double().cpu().numpy(), T, k, p, 0.0)
    wide = np.flatnonzero(w > 1e-4)   # u in the middle of each token's interval
    got = _tokens(torch, w4, x, (w.cumsum() - w / 2)[wide], T, k, p)
    assert np.array_equal(got, wide)


@pytest.mark.parametrize("V", [700, 262144])
def test_masked_rows_beside_others(V):
    # a mask of the lowest number, of -infinity and none, rows of one call
    torch, w4 = cuda_or_skip()
    g = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randn(3, V, device="cuda", generator=g)
    keep = torch.rand(V, device="cuda", generator=g) < 300 / V
    x[0].masked_fill_(~keep, torch.finfo(torch.float32).min)
    x[1] = x[0].masked_fill(~keep, -np.inf)
    u = torch.rand(3, device="cuda", generator=g)
    u[1] = u[0]
    for k in (0, 20, 301, 600):
        kt = torch.full((3,), k, dtype=torch.int32, device="cuda")
        for p in (0.5, 1.0):
            out = torch.full((3,), -7, dtype=torch.int32, device="cuda")
            got = w4.w4a16_sample(x, u, top_k=kt, top_p=torch.full((3,), p, device="cuda"), out=out).tolist()
            assert got[0] == got[1] and bool(keep[got[0]]) and 0 <= got[2] < V


@pytest.mark.parametrize("T", [1e-37, 1e-30])
def test_tiny_temperatures(T):
    # the largest wins, however far below it the rest is in units of T
    torch, w4 = cuda_or_skip()
    for V in (40, 3000, 100000):
        x = torch.full((V,), -1e9, device="cuda")
        x[2], x[7] = 0.0, 0.25
        for k in (3, 300):
            assert (_tokens(torch, w4, x, [0.0, 0.5, 0.99], T, k, 1.0) == 7).all()


@pytest.mark.parametrize("k", [0, 2, 300])
@pytest.mark.parametrize("T", [1e38, 2e38, 3.4e38, np.inf])
def test_temperatures_as_large_as_the_logits(T, k):
    # differences of logits past binary32's range, quotients of ordinary size
    torch, w4 = cuda_or_skip()
    x = np.zeros(1000)
    x[3], x[900], x[500] = 3e38, -3e38, -1e38
    x[1::2] = -np.inf
    x[3] = 3e38
    w = _kept(np.float32(x), float(np.float32(T)) if T < 1e39 else 1e300, k, 1.0, 0.0)
    wide = np.flatnonzero(w > 1e-4)
    got = _tokens(torch, w4, torch.tensor(x, dtype=torch.float32, device="cuda"), (w.cumsum() - w / 2)[wide], T, k, 1.0)
    assert np.array_equal(got, wide)


@pytest.mark.parametrize("V", [40, 3000, 262144])
@pytest.mark.parametrize("bits", [30, 100])
@pytest.mark.parametrize("T", [0.9, 0.95, 0.6])
@pytest.mark.parametrize("k,p", [(0, 1.0), (9, 1.0), (300, 1.0), (0, 0.5), (300, 0.5)])
def test_quotients_whose_rounding_is_wider_than_the_exponentials(V, bits, T, k, p):
    # logits just below a power of two, in steps of 64 and more: l / T lies above it,
    # where numbers are twice as far apart, so tokens of different logits have the
    # same mass and a step further they have none (whole numbers, exact)
    torch, w4 = cuda_or_skip()
    rng = np.random.default_rng(V)
    step = rng.integers(0, 12, V)
    step[:4] = 0, 1, 2, 3
    for top in range(2 ** 24 - 2 ** 17, 2 ** 24):     # the two largest have the same quotient
        x = ((top - step) * 2.0 ** (bits - 24)).astype(np.float32)
        q = x / np.float32(T)
        if q[0] == q[1]:
            break
    x[V // 2:] /= 2
    q = x / np.float32(T)
    mass = np.rint(2.0 ** 40 * np.exp((q - q.max()).astype(np.float64)))
    order = np.argsort(-x, kind="stable")
    w = mass[order]
    w[k if k else V:] = 0
    if p < 1:
        before = np.cumsum(w) - w
        w[before >= max(np.trunc(w.sum() * p), 1)] = 0
    kept = np.zeros(V)
    kept[order] = w
    edge = kept.cumsum()
    u = np.float32(np.linspace(0.0, 0.9999, 60))
    want = np.searchsorted(edge, np.trunc(edge[-1] * u.astype(np.float64)), side="right")
    assert np.array_equal(_tokens(torch, w4, torch.tensor(x, device="cuda"), u, T, k, p), want)
