"""GPU tests of paged attention over caches that hold only what the new tokens see: pages that lie behind the
window (and past the sinks) are given back, and every other place that no token sees is NaN."""
import math

import pytest
import torch

from hybrid_checks import within
from test_gpu_paged import Cache, rsm  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def seen_places(n, L, W, S):
    """[L] truth values: some new token (at places L - n .. L - 1) sees the key."""
    j = torch.arange(L)
    return torch.ones(L, dtype=torch.bool) if not W else (j > L - n - W) | (j < S)


def release(c, W, S, fill, last=None):
    """Table entries without a seen place become `fill`, all rows without one NaN. last: new tokens that count."""
    page = c.k_cache.shape[1]
    keep = torch.zeros(c.k_cache.shape[:2], dtype=torch.bool)
    for b, (n, L) in enumerate(zip(c.new, c.lens)):
        seen = seen_places(n, L, W, S)
        if last is not None and n > last:
            seen[L - n + last:] = False
        for slot in range(c.table.shape[1]):
            part = seen[slot * page:(slot + 1) * page]
            if part.any():
                keep[c.table[b, slot], :len(part)] |= part
            else:
                c.table[b, slot] = fill
    for cache in (c.k_cache, c.v_cache):
        cache[~keep.cuda()] = float("nan")


# (new tokens, lengths, H, Hkv, D, window, sinks)
CASES = [([1], [700], 8, 2, 128, 100, 4), ([1] * 5, [5, 64, 90, 500, 1000], 4, 4, 64, 33, 0), ([2, 3], [900, 41], 10, 2, 80, 20, 1),
         ([40, 1, 0, 130], [500, 300, 9, 400], 4, 2, 64, 50, 4), ([200], [1000], 2, 2, 128, 150, 70), ([64, 33], [2100, 600], 8, 2, 72, 1, 0),
         ([1, 4], [3000, 800], 4, 1, 256, 100, 9), ([70], [400], 3, 3, 256, 90, 2), ([1], [9000], 2, 1, 128, 4000, 4),
         ([300], [300], 2, 1, 64, 64, 0), ([130], [4000], 4, 4, 64, 700, 130), ([1, 90], [300, 300], 4, 2, 64, 0, 0)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page", [1, 8, 16, 24, 64, 128])
@pytest.mark.parametrize("case", CASES)
def test_pages_that_nothing_sees(rsm, case, page, dtype):  # noqa: F811
    new, lens, H, Hkv, D, W, S = case
    c = Cache(new, lens, H, Hkv, D, page, dtype, seed=page + D)
    c.append(rsm)
    for fill in (-1, 2**31 - 1):
        release(c, W, S, fill)
        r = rsm.paged_forward(c.q, *c.args(), max(new), window=W, sinks=S, lse=True)
        torch.cuda.synchronize()
        assert rsm.device_status() == 0
        w = c.want(W, S, 1 / math.sqrt(D))
        within("o", r["o"], *w["o"])
        within("lse", r["lse"], *w["lse"], rms=False)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new,most", [([5, 7], 2), ([150, 40], 33)])
def test_tokens_past_the_limit(rsm, new, most, dtype):  # noqa: F811
    """Places of tokens past max_q are not computed, and not looked up by those that are."""
    c = Cache(new, [400, 90], 4, 2, 64, 16, dtype, seed=most)
    c.append(rsm)
    want = rsm.paged_forward(c.q, *c.args(), most, window=60)["o"].clone()
    release(c, 60, 0, -1, last=most)
    got = rsm.paged_forward(c.q, *c.args(), most, window=60)["o"]
    assert rsm.device_status() == 0
    for b, n in enumerate(new):
        rows = slice(c.cu[b], c.cu[b] + min(n, most))
        assert torch.isfinite(got[rows]).all() and torch.equal(got[rows], want[rows])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page", [8, 16, 24, 64])
@pytest.mark.parametrize("new", [1, 40])
def test_a_page_in_sight_is_still_reported(rsm, new, page, dtype):  # noqa: F811
    """The page with the window's first key, and the one with the last sink."""
    for slot in ((300 - new - 99) // page, 3 // page):
        c = Cache([new], [300], 4, 2, 64, page, dtype, seed=new)
        c.append(rsm)
        c.table[0, slot] = -1
        rsm.paged_forward(c.q, *c.args(), new, window=100, sinks=4)
        assert rsm.device_status() == 7 and rsm.device_status() == 0
