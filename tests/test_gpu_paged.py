"""GPU tests of rsm_paged_append and rsm_paged_forward against the 64-bit form."""
import math
import random

import pytest
import torch

from oracle import hybrid
from hybrid_checks import roundings, within

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def rsm():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__
    __graft_entry__.build()
    import sparse_routed_slot_b200 as m
    return m


class Cache:
    """Sequences of the given lengths and new tokens, their rows scattered over shuffled pages; what no
    sequence holds is NaN."""

    def __init__(self, new, lens, H, Hkv, D, page, dtype, seed=0, spare=2, extra_width=1, behind=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.new, self.lens, self.dtype = new, lens, dtype
        B, N = len(new), sum(new)
        width = max([-(-x // page) for x in lens] + [0]) + extra_width
        pages = B * width + spare
        order = list(range(pages))
        random.Random(seed).shuffle(order)
        table = torch.full((B, width), -1, dtype=torch.int32)
        self.k_cache = torch.full((pages, page, Hkv, D), float("nan"), device="cuda", dtype=dtype)
        self.v_cache = self.k_cache.clone()
        self.q = (r(N + behind, H, D) * 2).to(dtype)
        self.k, self.v = r(N + behind, Hkv, D).to(dtype), r(N + behind, Hkv, D).to(dtype)
        self.keys, self.values = [], []
        cu = [0]
        for b, (n, L) in enumerate(zip(new, lens)):
            kk, vv = r(L, Hkv, D).to(dtype), r(L, Hkv, D).to(dtype)
            m = min(n, L)  # new tokens that have a place
            if m:
                kk[L - m:] = self.k[cu[-1] + n - m:cu[-1] + n]
                vv[L - m:] = self.v[cu[-1] + n - m:cu[-1] + n]
            for s in range(-(-L // page)):
                table[b, s] = order.pop()
                rows = slice(s * page, min(L - m, (s + 1) * page))  # the new ones are left to the append
                if rows.stop > rows.start:
                    self.k_cache[table[b, s], :rows.stop - rows.start] = kk[rows]
                    self.v_cache[table[b, s], :rows.stop - rows.start] = vv[rows]
            self.keys.append(kk)
            self.values.append(vv)
            cu.append(cu[-1] + n)
        self.cu = cu
        self.table = table.cuda()
        self.cu_q = torch.tensor(cu, dtype=torch.int32, device="cuda")
        self.kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def args(self):
        return self.k_cache, self.v_cache, self.table, self.cu_q, self.kv_len

    def append(self, rsm):
        rsm.paged_append(self.k, self.v, *self.args())

    def want(self, W, S, scale):
        u, uo = roundings(self.dtype)
        each = []
        for b, (n, L) in enumerate(zip(self.new, self.lens)):
            at = torch.arange(L - n, L, device="cuda")
            each.append(hybrid.attend(self.q[self.cu[b]:self.cu[b + 1]], self.keys[b], self.values[b], at, W, S, scale, None, u, uo))
        return {n: tuple(torch.cat([e[n][i] for e in each]) for i in (0, 1)) for n in ("o", "lse")}

    def check(self, rsm, W=0, S=0, max_q=None):
        D = self.q.shape[2]
        self.append(rsm)
        r = rsm.paged_forward(self.q, *self.args(), max(self.new) if max_q is None else max_q, window=W, sinks=S, lse=True)
        torch.cuda.synchronize()
        assert rsm.device_status() == 0
        N = self.cu[-1]
        w = self.want(W, S, 1 / math.sqrt(D))
        within("o", r["o"][:N], *w["o"])
        within("lse", r["lse"][:N], *w["lse"], rms=False)
        return r


# (new tokens, lengths, H, Hkv, D, page, window, sinks)
CASES = [([1], [1], 1, 1, 64, 16, 0, 0), ([1], [700], 16, 4, 128, 16, 0, 0), ([1] * 5, [1, 2, 63, 64, 65], 4, 4, 64, 64, 0, 0),
         ([1] * 3, [300, 128, 129], 8, 1, 128, 128, 100, 4), ([1] * 4, [17, 400, 255, 1000], 10, 2, 80, 8, 0, 0),
         ([3, 0, 1, 40], [3, 0, 200, 333], 4, 2, 64, 24, 0, 0), ([130, 1, 0, 77], [600, 5, 9, 77], 8, 2, 128, 16, 0, 0),
         ([200, 129], [1000, 129], 6, 2, 128, 32, 150, 4), ([64], [5000], 4, 1, 64, 64, 0, 0), ([5], [9000], 2, 2, 128, 256, 0, 0),
         ([16, 4], [500, 500], 4, 4, 72, 40, 37, 70), ([100], [260], 3, 3, 256, 16, 0, 0), ([2, 2], [50, 1], 4, 4, 64, 1, 0, 0),
         ([300], [300], 12, 4, 96, 7, 299, 0), ([33, 1], [2100, 2100], 64, 1, 128, 64, 512, 128), ([1], [20000], 8, 8, 128, 64, 0, 0)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", CASES)
def test_append_and_forward(rsm, case, dtype):
    new, lens, H, Hkv, D, page, W, S = case
    Cache(new, lens, H, Hkv, D, page, dtype, seed=len(new) + D).check(rsm, W, S)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_that_see_nothing(rsm, dtype):
    """More new tokens than the sequence holds: the first ones stand below place zero, see nothing, are
    written nowhere and get zeros."""
    c = Cache([5, 2, 3], [2, 0, 40], 4, 2, 64, 16, dtype, seed=3)
    r = c.check(rsm)
    assert (r["o"][:3] == 0).all() and (r["o"][5:7] == 0).all() and (r["lse"][:3] == float("-inf")).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new,lens", [([2, 1], [900, 40]), ([130, 64], [800, 64])])
def test_rows_behind_the_last_sequence_stay(rsm, dtype, new, lens):
    c = Cache(new, lens, 4, 2, 128, 16, dtype, seed=4, behind=7)
    N = sum(new)
    before = c.k_cache.clone()
    c.append(rsm)
    held = torch.zeros(c.k_cache.shape[:2], dtype=torch.bool, device="cuda")
    for b, (n, L) in enumerate(zip(new, lens)):
        for pos in range(L - n, L):
            held[c.table[b, pos // 16], pos % 16] = True
    same = lambda a, b: torch.equal(a.view(torch.uint8), b.view(torch.uint8))  # noqa: E731  (NaN compares too)
    assert same(c.k_cache[~held], before[~held])
    o = torch.full_like(c.q, 7.0)
    lse = torch.full((N + 7, 4), 7.0, device="cuda")
    rsm.paged_forward(c.q, *c.args(), max(new), lse=True, out={"o": o, "lse": lse})
    assert (o[N:] == 7).all() and (lse[N:] == 7).all() and torch.isfinite(o[:N]).all()
    # and rows past max_q
    o.fill_(7.0)
    rsm.paged_forward(c.q, *c.args(), 1, out={"o": o})
    assert (o[1:new[0]] == 7).all() and (o[new[0] + 1:] == 7).all()
    assert not (o[0] == 7).all() and not (o[new[0]] == 7).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_pages_and_lengths_outside_the_cache(rsm, dtype):
    """Left out and reported, for the write and for the read; nothing faults."""
    for new, lens in (([1, 1], [100, 90]), ([60, 40], [100, 90])):
        c = Cache(new, lens, 4, 2, 64, 16, dtype, seed=5)
        c.append(rsm)
        good = c.table.clone()
        for wrong in (-1, c.k_cache.shape[0], 2**31 - 1):
            c.table.copy_(good)
            c.table[0, 2] = wrong
            r = rsm.paged_forward(c.q, *c.args(), max(new))
            assert rsm.device_status() == 7 and rsm.device_status() == 0
            # the first sequence without keys 32..47, the second as before
            keep = [j for j in range(100) if not 32 <= j < 48]
            u, uo = roundings(dtype)
            places = torch.arange(100 - new[0], 100, device="cuda")
            # places counted among the keys that are left: the last row sees them all
            w = hybrid.attend(c.q[new[0] - 1:new[0]], c.keys[0][keep], c.values[0][keep],
                              torch.tensor([len(keep) - 1], device="cuda"), 0, 0, 1 / 8, None, u, uo)
            assert places[-1] == 99
            within("o", r["o"][new[0] - 1:new[0]], *w["o"])
        c.table[0, 99 // 16] = -5
        before = c.k_cache.clone()
        rsm.paged_append(c.k, c.v, *c.args())
        assert rsm.device_status() == 7
        assert torch.equal(c.k_cache.view(torch.uint8), before.view(torch.uint8))  # the same values again, or nothing
        c.table.copy_(good)
        c.kv_len[1] = 10**9
        rsm.paged_forward(c.q, *c.args(), max(new))
        rsm.paged_append(c.k, c.v, *c.args())
        assert rsm.device_status() == 7
        c.kv_len[1] = -3
        r = rsm.paged_forward(c.q, *c.args(), max(new))
        assert rsm.device_status() == 0 and (r["o"][new[0]:] == 0).all()
        # offsets out of order or past the tokens: clamped
        c.kv_len[1] = 90
        for cu in ([0, 10**9, 5], [5, 0, -1], [-4, 1, 2], [0, 0, 10**9]):
            c.cu_q.copy_(torch.tensor(cu, dtype=torch.int32))
            rsm.paged_forward(c.q, *c.args(), max(new))
            rsm.paged_append(c.k, c.v, *c.args())
        rsm.device_status()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_chunks_and_steps_match_one_window_call(rsm, dtype):
    """A prompt taken in by chunks and then token by token gives what one window call over it gives."""
    T, H, Hkv, D, W, S, page = 300, 4, 2, 64, 90, 3, 16
    g = torch.Generator(device="cuda").manual_seed(8)
    q, k, v = (torch.randn(1, T, h, D, generator=g, device="cuda").to(dtype) for h in (H, Hkv, Hkv))
    whole = rsm.window_forward(q, k, v, W, S)["o"][0]
    width = -(-T // page)
    kc = torch.full((width, page, Hkv, D), float("nan"), device="cuda", dtype=dtype)
    vc = kc.clone()
    table = torch.randperm(width, generator=torch.Generator().manual_seed(1)).to(torch.int32).view(1, width).cuda()
    at, got = 0, []
    for n in [130, 1, 64, 37] + [1] * 68:
        cu = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        ln = torch.tensor([at + n], dtype=torch.int32, device="cuda")
        rows = slice(at, at + n)
        rsm.paged_append(k[0, rows].contiguous(), v[0, rows].contiguous(), kc, vc, table, cu, ln)
        got.append(rsm.paged_forward(q[0, rows].contiguous(), kc, vc, table, cu, ln, n, window=W, sinks=S)["o"])
        at += n
    got = torch.cat(got)
    assert at == T
    u, uo = roundings(dtype)
    w = hybrid.attend(q[0], k[0], v[0], torch.arange(T, device="cuda"), W, S, 1 / 8, None, u, uo)["o"]
    within("paged", got, *w)
    within("window", whole, *w)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_shared_pages(rsm, dtype):
    """Two sequences with one prefix's pages in both tables."""
    c = Cache([1, 1], [80, 80], 4, 2, 64, 16, dtype, seed=6)
    c.append(rsm)
    c.table[1, :4] = c.table[0, :4]
    c.keys[1][:64], c.values[1][:64] = c.keys[0][:64], c.values[0][:64]
    c.check(rsm)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("pages,width", [(0, 0), (0, 3), (4, 0)])
def test_caches_without_pages(rsm, dtype, new, pages, width):
    """No keys anywhere: zeros, nothing written, and lengths above zero reported."""
    kc = torch.zeros(pages, 16, 2, 64, device="cuda", dtype=dtype)
    table = torch.zeros(2, width, device="cuda", dtype=torch.int32)
    cu = torch.tensor([0, new, 2 * new], device="cuda", dtype=torch.int32)
    x, k = (torch.ones(2 * new, h, 64, device="cuda", dtype=dtype) for h in (4, 2))
    for lens, status in (([0, 0], 0), ([new, 0], 7)):
        n = torch.tensor(lens, device="cuda", dtype=torch.int32)
        rsm.paged_append(k, k, kc, kc.clone(), table, cu, n)
        assert rsm.device_status() == status
        r = rsm.paged_forward(x, kc, kc, table, cu, n, new, lse=True)
        assert rsm.device_status() == status
        assert not r["o"].any() and (r["lse"] == float("-inf")).all() and not kc.any()


@pytest.mark.parametrize("page", [8, 24, 40, 16, 12])
@pytest.mark.parametrize("H,Hkv,D,new", [(4, 1, 128, 1), (8, 2, 64, 4), (6, 2, 80, 3), (4, 1, 256, 4), (5, 5, 128, 1)])
def test_few_rows_by_page_size(rsm, page, H, Hkv, D, new):
    """Tiles of 16 keys in one page, in two, and row by row; lengths around tiles, halves and pages."""
    for lens in ([5, 8, 9, 16], [17, 23, 24, 25], [40, 47, 48, 200], [1000, 39, 41, 7]):
        c = Cache([new] * 4, lens, H, Hkv, D, page, BF16, seed=page + D)
        c.check(rsm)
        c.check(rsm, W=20, S=3)


@pytest.mark.parametrize("page,slot", [(8, 2), (8, 3), (24, 1), (40, 0), (16, 1)])
def test_few_rows_with_a_page_missing(rsm, page, slot):
    """A tile of which only one half has its page."""
    c = Cache([1, 1], [130, 77], 8, 2, 128, page, BF16, seed=page + slot)
    c.append(rsm)
    c.table[0, slot] = -1
    r = rsm.paged_forward(c.q, *c.args(), 1)
    assert rsm.device_status() == 7 and rsm.device_status() == 0
    keep = [j for j in range(130) if j // page != slot]
    u, uo = roundings(BF16)
    for b, kept in ((0, keep), (1, list(range(77)))):
        w = hybrid.attend(c.q[b:b + 1], c.keys[b][kept], c.values[b][kept], torch.tensor([len(kept) - 1], device="cuda"), 0, 0,
                          1 / math.sqrt(128), None, u, uo)
        within("o", r["o"][b:b + 1], *w["o"])


def test_far_pages(rsm):
    """A cache whose last page lies past 2^31 elements and 2^32 bytes."""
    Hkv, D, page = 8, 128, 64
    pages = (1 << 31) // (page * Hkv * D) + 40
    kc = torch.empty(pages, page, Hkv, D, dtype=BF16, device="cuda")
    vc = torch.empty(pages, page, Hkv, D, dtype=BF16, device="cuda")
    small = Cache([1, 70], [130, 200], 8, Hkv, D, page, BF16, seed=7)
    n = small.k_cache.shape[0]
    kc[-n:], vc[-n:] = small.k_cache, small.v_cache
    small.table[small.table >= 0] += pages - n
    small.k_cache, small.v_cache = kc, vc
    small.check(rsm)


def test_refusals(rsm):
    c = Cache([1, 1], [20, 30], 4, 2, 64, 16, BF16)
    ok = dict(q=c.q, k_cache=c.k_cache, v_cache=c.v_cache, page_table=c.table, cu_q=c.cu_q, kv_len=c.kv_len, max_q=1)
    for kw in (dict(page_table=c.table.long()), dict(cu_q=c.cu_q[:2]), dict(kv_len=c.kv_len.cpu()), dict(q=c.q.float()),
               dict(q=c.q[:, :, :32]), dict(v_cache=c.v_cache[1:]), dict(q=c.q[None])):
        with pytest.raises(ValueError):
            rsm.paged_forward(**{**ok, **kw})
    for kw in (dict(max_q=-1), dict(window=-1), dict(scale=0.0), dict(q=c.q[:, :3].contiguous())):
        with pytest.raises(rsm.RSMError):
            rsm.paged_forward(**{**ok, **kw})
    bad = c.q.clone()
    bad[0, 0, 0] = float("nan")
    c.append(rsm)
    rsm.paged_forward(**{**ok, "q": bad}, validate=True)
    assert rsm.device_status() == 4


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new,lens", [([1, 1, 1], [4000, 70, 1]), ([40, 100], [2000, 100])])
def test_streams_and_graphs(rsm, dtype, new, lens):
    """A captured step, replayed as the lengths grow in place; two captures replayed side by side."""
    c = Cache(new, lens, 8, 2, 128, 16, dtype, seed=9)
    want = c.check(rsm)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.append(rsm)
        r = rsm.paged_forward(c.q, *c.args(), max(new))
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(r["o"], want["o"])
    graphs = []
    lens_now = c.kv_len.clone()
    c.kv_len.copy_(torch.tensor(new, dtype=torch.int32))
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cr = rsm.paged_forward(c.q, *c.args(), max(new))
        graphs.append((graph, cr))
    c.kv_len.copy_(lens_now)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for st, (graph, _) in zip(streams, graphs):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            for _ in range(3):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(cr["o"], want["o"]) for _, cr in graphs)
