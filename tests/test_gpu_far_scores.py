"""GPU tests of attention whose scores climb or fall by far more than 2^32 along the keys, so that the references
of the running softmax move again and again and those of a row's warps, blocks and parts stand far apart.

Every element has its own first-order bound. The bound on the whole (rms) is for scores of a few units: a score of
1536 (0.75 x 2048 keys) is rounded by up to 1536 x 2^-24 = 2^-13.4 with each term that is added to it, and its
weight with it, where that bound is 2^-16 in fp32. It is left out here."""
import math

import pytest
import torch

from oracle import hybrid
from hybrid_checks import roundings, within
from test_gpu_paged import Cache, rsm  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def slope(q, k, per_key):
    """Adds `per_key` (natural units, at the default scale) times the key's place to every score, through the
    first column: the keys' are the places, rounded, the queries' all alike. q [.., n, H, D], k [.., L, Hkv, D]."""
    D = q.shape[-1]
    q[..., 0] = per_key * math.sqrt(D) * 4
    k[..., 0] = (torch.arange(k.shape[-3], device=k.device) / 4)[:, None]


# (T, H, Hkv, D, window, sinks): one query head per key/value head, whose two query tiles are two key tiles apart,
# and groups, whose tiles are closer; windows that start inside, at and past the first tiles
WINDOWS = [(512, 2, 2, 64, 100, 0), (2048, 2, 2, 128, 512, 4), (1100, 1, 1, 128, 64, 0), (700, 3, 3, 72, 129, 70),
           (512, 2, 2, 128, 512, 0), (900, 4, 2, 64, 100, 4), (600, 4, 1, 128, 65, 0), (400, 5, 1, 80, 191, 130)]


@pytest.mark.parametrize("per_key", [0.75, -0.75, 5.0])
@pytest.mark.parametrize("shape", WINDOWS)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_window(rsm, shape, per_key, dtype):  # noqa: F811
    T, H, Hkv, D, W, S = shape
    g = torch.Generator(device="cuda").manual_seed(T + D)
    q, k, v, do = (torch.randn(2, T, h, D, generator=g, device="cuda").to(dtype) for h in (H, Hkv, Hkv, H))
    slope(q, k, per_key)
    r = rsm.window_forward(q, k, v, W, S, lse=True)
    torch.cuda.synchronize()
    assert rsm.device_status() == 0
    want = hybrid.window(q, k, v, W, S, 1 / math.sqrt(D), do, *roundings(dtype))
    within("o", r["o"], *want["o"], rms=False)
    within("lse", r["lse"], *want["lse"], rms=False)
    grads = rsm.window_backward(q, k, v, r["o"], r["lse"], do, W, S)
    for n in ("dq", "dk", "dv"):
        within(n, grads[n], *want[n], rms=False)  # few keys per row: ds is a difference of like values


# (new tokens, lengths, H, Hkv, D, page, window, sinks): chunks, whole and cut; few rows in one block per sequence,
# in clusters, and in blocks that leave parts
PAGED = [([300], [300], 2, 2, 64, 16, 100, 0), ([300], [1000], 2, 2, 128, 64, 150, 4), ([513, 200], [2300, 700], 1, 1, 128, 16, 65, 0),
         ([140, 64], [900, 3000], 2, 2, 72, 32, 0, 0), ([260], [4000], 4, 4, 64, 64, 0, 0), ([70], [2000], 8, 2, 128, 24, 300, 4),
         ([1] * 80, [50 + 13 * i for i in range(80)], 8, 4, 128, 16, 0, 0), ([1, 1], [700, 1000], 8, 2, 64, 16, 0, 0),
         ([1], [9000], 2, 1, 128, 64, 0, 0), ([3, 2], [6000, 100], 10, 2, 80, 8, 0, 0), ([4], [5000], 4, 1, 256, 16, 1500, 4),
         ([1] * 3, [300, 128, 129], 8, 1, 128, 128, 100, 4)]


@pytest.mark.parametrize("per_key", [0.75, -0.75, 5.0])
@pytest.mark.parametrize("case", PAGED)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_paged(rsm, case, per_key, dtype):  # noqa: F811
    new, lens, H, Hkv, D, page, W, S = case
    c = Cache(new, lens, H, Hkv, D, page, dtype, seed=len(new) + D)
    c.q /= 2
    for b, (n, L) in enumerate(zip(new, lens)):
        slope(c.q[c.cu[b]:c.cu[b + 1]], c.keys[b], per_key)
        c.k[c.cu[b]:c.cu[b + 1]] = c.keys[b][L - n:]
        at = torch.arange(L - n, device="cuda")
        c.k_cache[c.table[b].long()[at // page], at % page] = c.keys[b][:L - n]
    c.append(rsm)
    r = rsm.paged_forward(c.q, *c.args(), max(new), window=W, sinks=S, lse=True)
    torch.cuda.synchronize()
    assert rsm.device_status() == 0
    want = c.want(W, S, 1 / math.sqrt(D))
    for n in ("o", "lse"):
        within(n, r[n], *want[n], rms=False)


@pytest.mark.parametrize("H", [2, 8])
def test_random_far_scores(rsm, H):  # noqa: F811
    """Scores of hundreds without an order, over windows of two query tiles."""
    g = torch.Generator(device="cuda").manual_seed(H)
    q, k, v = (torch.randn(1, 1500, h, 128, generator=g, device="cuda").to(BF16) for h in (H, 2, 2))
    q *= 40
    r = rsm.window_forward(q, k, v, 300, 4, lse=True)
    torch.cuda.synchronize()
    assert rsm.device_status() == 0
    want = hybrid.window(q, k, v, 300, 4, 1 / math.sqrt(128), None, *roundings(BF16))
    within("o", r["o"], *want["o"], rms=False)
    within("lse", r["lse"], *want["lse"], rms=False)
