"""The score of a page by its bounds is no less than what any key of the page
gives a query head, the query taken in its 8 bits (in numpy, whose bounds and
choices the library's match bit for bit)."""
import numpy as np
import pytest

from tests import kv4_helpers as ref
from tests import kv4_long_helpers as lh


@pytest.mark.parametrize("H,G,D,bs", [(2, 1, 64, 16), (1, 4, 128, 32), (2, 2, 256, 16)])
@pytest.mark.parametrize("kind", ["normal", "far apart", "one sign", "zeros"])
def test_no_key_of_a_page_is_above_its_score(H, G, D, bs, kind):
    rng = np.random.default_rng(D + bs)
    pages = 4
    k = rng.normal(0, 2, (pages * bs, H, D))
    q = rng.normal(0, 1, (5, H * G, D))
    if kind == "far apart":
        k *= np.exp(rng.normal(0, 3, (pages * bs, H, 1)))
        q *= np.exp(rng.normal(0, 3, (5, H * G, D)))
    elif kind == "one sign":
        k, q = np.abs(k), -np.abs(q)
    elif kind == "zeros":
        k[:bs], k[bs:, :, ::2], q[0], q[1:, :, 1::3] = 0, 0, 0, 0
    k, q = ref.bf16(k), ref.bf16(q)
    c = ref.Cache(pages, H, bs, D)
    c.append(k, k, np.arange(pages * bs))
    raw = np.zeros((pages, H, 2 * D + 16), np.uint8)
    for page in range(pages):
        high, low, step = lh.bounds(c, page)
        assert np.abs(high).max() <= 127 and np.abs(low).max() <= 127
        raw[page, :, :D], raw[page, :, D:2 * D] = high.astype(np.int8).view(np.uint8), low.astype(np.int8).view(np.uint8)
        raw[page, :, 2 * D:2 * D + D // 16] = step.view(np.uint8)
    u = np.abs(q).max(-1, keepdims=True) * 65 / 8192
    whole = np.rint(q / np.where(u > 0, u, 1)) * u           # the query as it is scored
    steps = raw[..., 2 * D:].view(np.float32)[..., :D // 64].astype(np.float64).repeat(64, -1)   # [pages, H, D]
    for t in range(len(q)):
        for h in range(H):
            rows = slice(h * G, (h + 1) * G)
            score = lh.scores(q[t, rows], raw, np.arange(pages), h)
            for page in range(pages):
                v = np.array([c.values(0, page * bs + i, h) for i in range(bs)])
                # binary32: the bounds' quotients 2^-23 of a key, the unit 2^-24, five operations 2^-24 of the
                # sum each; less than 2^-20 of the largest that the sum can be
                slack = 2.0 ** -20 * (np.abs(whole[t, rows]) @ (127 * steps[page, h])).max()
                assert (whole[t, rows] @ v.T).max() <= score[page] + slack
                # and not far above: by no more than the width of the bounds, and the two steps of rounding them
                span = v.max(0) - v.min(0) + 2 * steps[page, h]
                assert score[page] <= (whole[t, rows] @ v.T).max() + (np.abs(whole[t, rows]) @ span).max() + slack
