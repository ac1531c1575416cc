"""GPU tests of the block norms and their gradients against the 64-bit form, and of the operators run
together as one hybrid block."""
import math

import pytest
import torch

from oracle import hybrid
from hybrid_checks import HALF_STEP, roundings, within

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


def inputs(rows, d, ty, t, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    shape = rows if isinstance(rows, tuple) else (rows,)
    x = dict(y=(0.3 * r(*shape, d)).to(ty), gate=r(*shape, d).to(t), residual=r(*shape, d).to(t), w_post=1 + 0.2 * r(d),
             w_pre=1 + 0.2 * r(d))
    return x, r(*shape, d).to(t), r(*shape, d).to(t)


def close(name, got, want):
    """Row sums of d terms, row factors and products move a value by at most (d + 64) fp32 half steps of the
    row's largest value, and storing it by half a step of its own; a column sum by its rows' as well."""
    d = got.shape[-1]
    g, w = got.double(), want
    if g.dim() > 1:
        size = w.abs().amax(-1, keepdim=True)
    else:
        size = w.abs().amax()
    rows = 4096
    bound = (d + 64 + (rows if g.dim() == 1 else 0)) * 2.0 ** -24 * size + (HALF_STEP[got.dtype] + 2.0 ** -20) * w.abs()
    err = (g - w).abs()
    assert (err <= bound + 1e-30).all(), f"{name}: worst {float((err / (bound + 1e-30)).max()):.3g} times its bound"


SIZES = [(1, 4), (3, 8), (7, 64), (5, 100), (9, 256), (17, 260), (33, 1024), (12, 1020), (300, 2048), (6, 4096), (5, 4100),
         (40, 8192), (3, 8188), (1000, 128), (2500, 512)]


@pytest.mark.parametrize("ty,t", [(F32, F32), (BF16, BF16), (F32, BF16)])
@pytest.mark.parametrize("rows,d", SIZES)
@pytest.mark.parametrize("act", ["silu", "sigmoid"])
def test_forward_and_backward(rsm, rows, d, ty, t, act):
    x, dh, dx = inputs(rows, d, ty, t, seed=d)
    how = dict(act=act, scale=0.7, eps=1e-5)
    r = rsm.block_norm_forward(**x, **how)
    g = rsm.block_norm_backward(**x, dh=dh, dx=dx, **how)
    want = hybrid.block_norm(x["y"], x["gate"], x["residual"], x["w_post"], x["w_pre"], act, 0.7, 1e-5, dh, dx)
    for n, v in {**r, **g}.items():
        assert v.dtype == (F32 if n.startswith("dw") else ty if n == "dy" else t)
        close(n, v, want[n])


@pytest.mark.parametrize("ty,t", [(F32, F32), (BF16, BF16), (F32, BF16)])
@pytest.mark.parametrize("rows,d", [(37, 16), (1001, 12), (129, 60), (4000, 32), (130, 132), (33, 360), (700, 2500), (70, 1540),
                                    (5, 6144), (300, 6148), (9, 5000)])
def test_rows_that_share_a_warp_and_odd_widths(rsm, rows, d, ty, t):
    """Rows of 8 and 16 lanes with a last block that is not full, and widths that leave lanes and pieces idle."""
    test_forward_and_backward(rsm, rows, d, ty, t, "sigmoid")


@pytest.mark.parametrize("ty,t", [(F32, F32), (BF16, BF16), (F32, BF16)])
@pytest.mark.parametrize("rows,d", [(60000, 64), (20000, 100), (12000, 1024), (4000, 2500), (3000, 8192)])
def test_in_place_over_many_rows(rsm, rows, d, ty, t):
    """Blocks that read rows ahead of those they overwrite; and the gradients' bits do not change from call to call."""
    x, dh, dx = inputs(rows, d, ty, t, seed=2)
    want = rsm.block_norm_forward(**x)
    first = rsm.block_norm_backward(**x, dh=dh, dx=dx)
    again = rsm.block_norm_backward(**x, dh=dh, dx=dx)
    assert all(torch.equal(first[n], again[n]) for n in first)
    for name in ("residual", "y") if ty == t else ("residual",):
        y = {n: v.clone() for n, v in x.items()}
        r = rsm.block_norm_forward(**y, out={"h": y[name]})
        assert torch.equal(r["h"], want["h"]) and torch.equal(r["x"], want["x"])
    for part in (slice(0, 7), slice(rows - 7, rows)):
        few = {n: (v if n.startswith("w_") else v[part].contiguous()) for n, v in x.items()}
        w = hybrid.block_norm(few["y"], few["gate"], few["residual"], few["w_post"], few["w_pre"], "silu", 1.0, 1e-6,
                              dh[part], dx[part])
        for n in ("h", "x"):
            close(n, want[n][part], w[n])
        for n in ("dy", "dgate", "dresidual"):
            close(n, first[n][part], w[n])


@pytest.mark.parametrize("t", [BF16, F32])
def test_optional_parts(rsm, t):
    x, dh, dx = inputs((2, 5), 96, t, t, seed=3)
    for drop in ({"gate"}, {"w_pre"}, {"gate", "w_pre"}):
        y = {n: (None if n in drop else v) for n, v in x.items()}
        e = None if "w_pre" in drop else dx
        r = rsm.block_norm_forward(**y)
        g = rsm.block_norm_backward(**y, dh=dh, dx=e)
        want = hybrid.block_norm(y["y"], y["gate"], y["residual"], y["w_post"], y["w_pre"], "silu", 1.0, 1e-6, dh, e)
        for n, v in {**r, **g}.items():
            assert (v is None) == (n not in want), n
            if v is not None:
                close(n, v, want[n])
    for a, b in ((dh, None), (None, dx)):
        g = rsm.block_norm_backward(**x, dh=a, dx=b)
        want = hybrid.block_norm(x["y"], x["gate"], x["residual"], x["w_post"], x["w_pre"], "silu", 1.0, 1e-6, a, b)
        for n, v in g.items():
            close(n, v, want.get(n, torch.zeros_like(v, dtype=torch.float64)))
    g = rsm.block_norm_backward(**x)
    assert all((v == 0).all() for v in g.values())


def test_no_rows_and_in_place(rsm):
    x, dh, dx = inputs(0, 64, BF16, BF16)
    r = rsm.block_norm_forward(**x)
    g = rsm.block_norm_backward(**x, dh=dh, dx=dx)
    assert r["h"].shape == (0, 64) and (g["dw_post"] == 0).all() and (g["dw_pre"] == 0).all()
    x, _, _ = inputs(50, 512, BF16, BF16)
    want = rsm.block_norm_forward(**x)
    for name in ("residual", "y"):
        y = {n: v.clone() for n, v in x.items()}
        r = rsm.block_norm_forward(**y, out={"h": y[name]})
        assert torch.equal(r["h"], want["h"]) and torch.equal(r["x"], want["x"])


@pytest.mark.parametrize("d", [96, 1024, 8192])
def test_zero_and_extreme_rows(rsm, d):
    """A row of zeros divides by sqrt(eps), not by zero; far gates saturate."""
    x, dh, dx = inputs(4, d, F32, F32, seed=4)
    x["y"][1] = 0
    x["residual"][1] = 0
    x["gate"][2] = 200.0
    x["gate"][3] = -200.0
    r = rsm.block_norm_forward(**x, eps=1e-3)
    g = rsm.block_norm_backward(**x, dh=dh, dx=dx, eps=1e-3)
    want = hybrid.block_norm(x["y"], x["gate"], x["residual"], x["w_post"], x["w_pre"], "silu", 1.0, 1e-3, dh, dx)
    assert (r["h"][1] == 0).all() and (r["x"][1] == 0).all()
    for n, v in {**r, **g}.items():
        close(n, v, want[n])


def test_gradients_match_differences(rsm):
    """The fp32 gradients against central differences of the 64-bit form along random directions."""
    x, dh, dx = inputs(6, 64, F32, F32, seed=5)
    g = rsm.block_norm_backward(**x, dh=dh, dx=dx, scale=0.7, eps=1e-5)
    gen = torch.Generator(device="cuda").manual_seed(1)
    f = lambda z: sum((a * b.double()).sum() for a, b in zip(  # noqa: E731
        (lambda t: (t["h"], t["x"]))(hybrid.block_norm(z["y"], z["gate"], z["residual"], z["w_post"], z["w_pre"], "silu", 0.7, 1e-5)), (dh, dx)))
    for n, gn in (("y", "dy"), ("gate", "dgate"), ("residual", "dresidual"), ("w_post", "dw_post"), ("w_pre", "dw_pre")):
        way = torch.randn(x[n].shape, generator=gen, device="cuda", dtype=torch.float64)
        h = 1e-4
        up = f({**{m: v.double() for m, v in x.items()}, n: x[n].double() + h * way})
        down = f({**{m: v.double() for m, v in x.items()}, n: x[n].double() - h * way})
        slope = float((up - down) / (2 * h))
        got = float((g[n if n in g else gn].double() * way).sum())
        # the difference's own error is of order h^2; the gradient's 2^-24 a term
        assert abs(got - slope) <= 1e-4 * float((g[gn].double() * way).abs().sum()), n


@pytest.mark.parametrize("t", [BF16, F32])
def test_autograd_streams_graphs_and_repeats(rsm, t):
    x, dh, dx = inputs(700, 1024, t, t, seed=6)
    leaves = {n: v.clone().requires_grad_(True) for n, v in x.items()}
    h, xx = rsm.BlockNormFunction.apply(*leaves.values(), "sigmoid", 0.5, 1e-6)
    grads = torch.autograd.grad((h, xx), list(leaves.values()), (dh, dx))
    g = rsm.block_norm_backward(**x, dh=dh, dx=dx, act="sigmoid", scale=0.5)
    for a, n in zip(grads, ("dy", "dgate", "dresidual", "dw_post", "dw_pre")):
        assert torch.equal(a, g[n]), n
    h, xx = rsm.BlockNormFunction.apply(*leaves.values())
    h.sum().backward()  # x unused, and an expanded gradient
    one = rsm.block_norm_backward(**x, dh=torch.ones_like(dh))
    assert torch.equal(leaves["y"].grad, one["dy"]) and torch.equal(leaves["w_post"].grad, one["dw_post"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s = rsm.block_norm_backward(**x, dh=dh, dx=dx, act="sigmoid", scale=0.5)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(s[n], g[n]) for n in g)
    graph = torch.cuda.CUDAGraph()
    static = {n: torch.zeros_like(v) for n, v in x.items()}
    with torch.cuda.graph(graph):
        c = rsm.block_norm_backward(**static, dh=dh, dx=dx, act="sigmoid", scale=0.5)
        f = rsm.block_norm_forward(**static, act="sigmoid", scale=0.5)
    for n in x:
        static[n].copy_(x[n])
    for _ in range(2):
        graph.replay()
    want = rsm.block_norm_forward(**x, act="sigmoid", scale=0.5)
    assert all(torch.equal(c[n], g[n]) for n in g) and torch.equal(f["h"], want["h"]) and torch.equal(f["x"], want["x"])


def test_refusals(rsm):
    x, _, _ = inputs(4, 64, BF16, BF16)
    for kw in (dict(y=x["y"][:3]), dict(gate=x["gate"].float()), dict(w_post=x["w_post"].to(BF16)), dict(act="relu"),
               dict(residual=x["residual"].t()), dict(w_pre=x["w_pre"][:32]), dict(y=x["y"].half())):
        with pytest.raises(ValueError):
            rsm.block_norm_forward(**{**x, **kw})
    with pytest.raises(rsm.RSMError):
        rsm.block_norm_forward(**x, eps=0.0)
    y, _, _ = inputs(4, 64, BF16, F32)
    with pytest.raises(rsm.RSMError):
        rsm.block_norm_forward(**y)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_hybrid_block(rsm, dtype):
    """One mixer layer and one attention layer as a hybrid stack runs them: the mixer's fp32 output through
    its norms, then window attention over the next layer's heads and its norms; every operator against its
    64-bit form on what it was given, and the gradients back to the mixer's inputs."""
    from sparse_routed_slot_b200.workloads import make_inputs
    B, T, H, M, K, Dv = 2, 150, 4, 64, 8, 64
    m = make_inputs(B, T, H, M, Dv, dtype, "head", seed=1, device="cuda")
    x, _, _ = inputs((B, T), H * Dv, F32, dtype, seed=2)
    z, _, dx = inputs((B, T), H * Dv, dtype, dtype, seed=3)
    leaves = {n: m[n].clone().requires_grad_(True) for n in ("q", "k", "v", "logits", "f")}
    o, _ = rsm.RSMFunction.apply(leaves["q"], leaves["k"], leaves["v"], leaves["logits"], leaves["f"], K)
    h1, x1 = rsm.BlockNormFunction.apply(o.reshape(B, T, H * Dv), x["gate"], x["residual"], x["w_post"], x["w_pre"])
    heads = x1.view(B, T, H, Dv)
    kv = heads[:, :, :2].contiguous()
    a = rsm.WindowFunction.apply(heads, kv, kv, 40, 4)
    h2, x2 = rsm.BlockNormFunction.apply(a.reshape(B, T, H * Dv), z["gate"], h1, z["w_post"], z["w_pre"])
    x2.backward(dx)
    n1 = hybrid.block_norm(o.detach().view(B, T, -1), x["gate"], x["residual"], x["w_post"], x["w_pre"], "silu", 1.0, 1e-6)
    close("h1", h1, n1["h"])
    close("x1", x1, n1["x"])
    w = hybrid.window(heads.detach(), kv.detach(), kv.detach(), 40, 4, 1 / math.sqrt(Dv), None, *roundings(dtype))
    within("attention", a, *w["o"])
    n2 = hybrid.block_norm(a.detach().reshape(B, T, -1), z["gate"], h1.detach(), z["w_post"], z["w_pre"], "silu", 1.0, 1e-6)
    close("h2", h2, n2["h"])
    close("x2", x2, n2["x"])
    assert all(torch.isfinite(t.grad).all() and (t.grad != 0).any() for t in leaves.values())
