"""GPU tests of rsm_window_forward and rsm_window_backward against the 64-bit form, element by element
within first-order bounds of fp32 arithmetic and the documented bf16 roundings."""
import math

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


def inputs(B, T, H, Hkv, D, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda h, s=1.0: (torch.randn(B, T, h, D, generator=g, device="cuda") * s).to(dtype)  # noqa: E731
    return r(H, 2.0), r(Hkv), r(Hkv), r(H)


# (B, T, H, Hkv, D, window, sinks): one token, one key, edges around tile sizes, groups that fill no
# tile, sinks inside, at and past the window, windows past the sequence, odd head dimensions
SHAPES = [(1, 1, 1, 1, 64, 1, 0), (2, 2, 2, 1, 8, 1, 0), (1, 5, 3, 1, 16, 2, 1), (2, 31, 4, 4, 64, 7, 0), (1, 64, 4, 2, 128, 64, 4),
          (1, 65, 6, 2, 64, 33, 5), (2, 127, 4, 1, 128, 16, 37), (1, 128, 2, 2, 128, 128, 0), (1, 129, 5, 1, 80, 128, 3),
          (1, 257, 8, 8, 128, 100, 130), (1, 300, 6, 2, 72, 1000, 0), (2, 400, 7, 1, 64, 127, 4), (1, 513, 3, 3, 96, 256, 1),
          (1, 700, 4, 2, 120, 65, 300), (1, 1025, 2, 1, 128, 511, 64), (1, 260, 2, 1, 256, 90, 2), (1, 200, 3, 3, 136, 300, 9),
          (1, 130, 64, 1, 64, 40, 2), (1, 1500, 2, 2, 128, 1, 1), (3, 333, 4, 2, 64, 200, 500),
          (1, 2048, 2, 2, 128, 512, 4), (1, 5400, 1, 1, 64, 100, 140), (1, 4200, 3, 1, 128, 300, 5), (1, 1900, 2, 2, 80, 2000, 0)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward(rsm, shape, dtype):
    B, T, H, Hkv, D, W, S = shape
    q, k, v, do = inputs(B, T, H, Hkv, D, dtype, seed=T + D)
    scale = 1 / math.sqrt(D)
    r = rsm.window_forward(q, k, v, W, S, lse=True)
    g = rsm.window_backward(q, k, v, r["o"], r["lse"], do, W, S)
    torch.cuda.synchronize()
    assert rsm.device_status() == 0
    want = hybrid.window(q, k, v, W, S, scale, do, *roundings(dtype))
    within("lse", r["lse"], *want["lse"], rms=False)
    within("o", r["o"], *want["o"])
    # over one key the gradients of q and k are zero: nothing for an rms to be measured by
    for n in ("dq", "dk", "dv"):
        within(n, g[n], *want[n], rms=W > 1 and T > 2)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scale_and_supplied_outputs(rsm, dtype):
    q, k, v, _ = inputs(1, 150, 4, 2, 64, dtype, 5)
    o, lse = torch.full_like(q, float("nan")), torch.full((1, 150, 4), float("nan"), device="cuda")
    r = rsm.window_forward(q, k, v, 50, 3, 0.31, out={"o": o, "lse": lse})
    assert r["o"] is o and r["lse"] is lse
    want = hybrid.window(q, k, v, 50, 3, 0.31, None, *roundings(dtype))
    within("o", o, *want["o"])
    within("lse", lse, *want["lse"], rms=False)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_large_scores(rsm, dtype):
    """Scores of hundreds: the running maximum keeps every exponent at or below zero."""
    q, k, v, do = inputs(1, 300, 2, 1, 128, dtype, 6)
    q = (q.float() * 20).to(dtype)
    r = rsm.window_forward(q, k, v, 200, 4, lse=True)
    want = hybrid.window(q, k, v, 200, 4, 1 / math.sqrt(128), do, *roundings(dtype))
    within("o", r["o"], *want["o"])
    g = rsm.window_backward(q, k, v, r["o"], r["lse"], do, 200, 4)
    for n in ("dq", "dk", "dv"):
        within(n, g[n], *want[n], rms=False)  # nearly one key per row: ds is a difference of like values


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_results_do_not_change(rsm, dtype):
    q, k, v, do = inputs(2, 600, 8, 2, 128, dtype, 7)
    first = None
    for _ in range(3):
        r = rsm.window_forward(q, k, v, 150, 4, lse=True)
        g = rsm.window_backward(q, k, v, r["o"], r["lse"], do, 150, 4)
        now = [r["o"], r["lse"], g["dq"], g["dk"], g["dv"]]
        if first is None:
            first = [t.clone() for t in now]
        assert all(torch.equal(a, b) for a, b in zip(first, now))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_autograd_and_skipped_gradients(rsm, dtype):
    q, k, v, do = inputs(1, 200, 4, 2, 64, dtype, 8)
    leaves = [t.clone().requires_grad_(True) for t in (q, k, v)]
    o = rsm.WindowFunction.apply(*leaves, 60, 2)
    (o.float() * do.float()).sum().backward()
    r = rsm.window_forward(q, k, v, 60, 2, lse=True, low=True)
    g = rsm.window_backward(q, k, v, r["o"], r["lse"], do, 60, 2, low=r["low"])
    assert torch.equal(o, r["o"]) and (r["low"] is None) == (dtype == F32)
    for x, n in zip(leaves, ("dq", "dk", "dv")):
        assert torch.equal(x.grad, g[n])
    for keep in range(3):
        need = [i == keep for i in range(3)]
        one = rsm.window_backward(q, k, v, r["o"], r["lse"], do, 60, 2, low=r["low"], need=need)
        for i, n in enumerate(("dq", "dk", "dv")):
            assert (one[n] is None) if not need[i] else torch.equal(one[n], g[n])
    # an expanded output gradient (a plain sum's) is not contiguous
    leaves = [t.clone().requires_grad_(True) for t in (q, k, v)]
    rsm.WindowFunction.apply(*leaves, 60, 2).sum().backward()
    ones = rsm.window_backward(q, k, v, r["o"], r["lse"], torch.ones_like(do), 60, 2, low=r["low"])
    assert all(torch.equal(x.grad, ones[n]) for x, n in zip(leaves, ("dq", "dk", "dv")))


@pytest.mark.parametrize("shape", [(2, 129, 6, 2, 64, 5, 1), (1, 300, 4, 4, 128, 9, 0), (1, 70, 2, 1, 256, 4, 2),
                                   (1, 90, 3, 3, 80, 3, 1)])
def test_what_rounding_left(rsm, shape):
    """o + low is o to 16 bits more or less, and with it the gradients of rows of few keys keep two of their three
    roundings (ds, and the result: 2^-8 / sqrt(3) rms each; the fp32 arithmetic is far below). Both are uniform in the
    worst case only; their usual size, 0.0017 each, leaves room for what the weights' rounding keeps in o."""
    B, T, H, Hkv, D, W, S = shape
    q, k, v, do = inputs(B, T, H, Hkv, D, BF16, seed=D)
    r = rsm.window_forward(q, k, v, W, S, lse=True, low=True)
    assert torch.equal(r["o"], rsm.window_forward(q, k, v, W, S)["o"])
    g = rsm.window_backward(q, k, v, r["o"], r["lse"], do, W, S, low=r["low"])
    want = hybrid.window(q, k, v, W, S, 1 / math.sqrt(D), do, *roundings(BF16))
    # the softmax weights' rounding stays in o, the result's own is gone but for half a step of the rest
    within("o + low", r["o"].double() + r["low"].double(), *want["o"], rms=False)
    off = lambda x, y: float((x - y).norm() / y.norm())  # noqa: E731
    assert off(r["o"].double() + r["low"].double(), want["o"][0]) < off(r["o"].double(), want["o"][0])
    for n in ("dq", "dk"):
        assert off(g[n].double(), want[n][0]) <= 2.0 ** -8 * (2 / 3) ** 0.5, n


def test_no_query_heads(rsm):
    """Keys and values that no query head reads: their gradients are empty sums."""
    x, k = torch.zeros(1, 5, 0, 8, device="cuda", dtype=BF16), torch.zeros(1, 5, 2, 8, device="cuda", dtype=BF16)
    r = rsm.window_forward(x, k, k, 3, lse=True)
    out = {n: torch.full_like(k, float("nan")) for n in ("dk", "dv")}
    g = rsm.window_backward(x, k, k, r["o"], r["lse"], x, 3, out=out)
    assert g["dq"].numel() == 0 and not g["dk"].any() and not g["dv"].any()
    one = rsm.window_backward(x, k, k, r["o"], r["lse"], x, 3, need=(True, False, True))
    assert one["dk"] is None and not one["dv"].any()


def test_empty_and_refused(rsm):
    for shape in ((0, 5, 2, 8), (1, 0, 2, 8), (1, 5, 0, 8)):
        x = torch.zeros(shape, device="cuda", dtype=BF16)
        r = rsm.window_forward(x, x, x, 3, lse=True)
        assert r["o"].shape == x.shape
        g = rsm.window_backward(x, x, x, r["o"], r["lse"], x, 3)
        assert g["dk"].shape == x.shape
    x = torch.zeros(1, 4, 2, 8, device="cuda", dtype=BF16)
    for bad in (dict(k=x[:, :3].contiguous()), dict(k=x.float()), dict(k=x.transpose(0, 1)), dict(k=x[0])):
        with pytest.raises(ValueError):
            rsm.window_forward(x, bad["k"], x, 3)
    for kw in (dict(window=0), dict(window=3, sinks=-1), dict(window=3, scale=-1.0)):
        with pytest.raises(rsm.RSMError):
            rsm.window_forward(x, x, x, **kw)
    with pytest.raises(ValueError):
        rsm.window_backward(x, x, x, x, torch.zeros(1, 4, 2, device="cuda"), x.float(), 3)
    y = x.float()
    with pytest.raises(rsm.RSMError):  # nothing is rounded in fp32
        rsm.window_forward(y, y, y, 3, out={"low": torch.zeros_like(y)})


def test_validate_reports_infinities(rsm):
    x = torch.zeros(1, 40, 2, 8, device="cuda", dtype=BF16)
    rsm.window_forward(x, x, x, 3, validate=True)
    assert rsm.device_status() == 0
    bad = x.clone()
    bad[0, 30, 1, 3] = float("inf")
    for a in ((bad, x, x), (x, bad, x), (x, x, bad)):
        rsm.window_forward(*a, 3, validate=True)
        assert rsm.device_status() == 4 and rsm.device_status() == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_streams_and_graphs(rsm, dtype):
    """Inputs made on one stream, calls on another; and a captured forward and backward, replayed on new
    inputs while another capture of its own workspace runs beside it."""
    q, k, v, do = inputs(1, 500, 4, 4, 128, dtype, 9)
    want = rsm.window_forward(q, k, v, 100, 4, lse=True)
    grads = rsm.window_backward(q, k, v, want["o"], want["lse"], do, 100, 4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r = rsm.window_forward(q, k, v, 100, 4, lse=True)
        g = rsm.window_backward(q, k, v, r["o"], r["lse"], do, 100, 4)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(r["o"], want["o"]) and all(torch.equal(g[n], grads[n]) for n in grads)

    static = [torch.zeros_like(t) for t in (q, k, v, do)]
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            cr = rsm.window_forward(*static[:3], 100, 4, lse=True)
            cg = rsm.window_backward(*static[:3], cr["o"], cr["lse"], static[3], 100, 4)
        graphs.append((graph, cr, cg))
    for s, t in zip(static, (q, k, v, do)):
        s.copy_(t)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for st, (graph, _, _) in zip((a, b), graphs):
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            for _ in range(3):
                graph.replay()
    torch.cuda.synchronize()
    for _, cr, cg in graphs:
        assert torch.equal(cr["o"], want["o"]) and all(torch.equal(cg[n], grads[n]) for n in grads)
