"""GPU tests of the autograd functions where autograd hands their backward a slice of a larger gradient, which is
contiguous and does not start on a 16-byte boundary."""
import pytest
import torch

from test_gpu_block_norm import inputs, rsm  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def behind_one(*outputs):
    """The outputs behind a single value in one flat tensor, and a gradient for it."""
    one = torch.ones(1, device="cuda", dtype=outputs[0].dtype)
    flat = torch.cat([one, *(o.flatten() for o in outputs)])
    g = torch.Generator(device="cuda").manual_seed(1)
    return flat, torch.randn(flat.shape, generator=g, device="cuda").to(flat.dtype)


def parts(grad, *outputs):
    sizes = [o.numel() for o in outputs]
    return [x.clone().view(o.shape) for x, o in zip(grad[1:].split(sizes), outputs)]


@pytest.mark.parametrize("t", [BF16, F32])
def test_block_norm(rsm, t):  # noqa: F811
    x, _, _ = inputs(5, 96, t, t)
    leaves = [v.clone().requires_grad_(True) for v in x.values()]
    h, xx = rsm.BlockNormFunction.apply(*leaves)
    flat, grad = behind_one(h, xx)
    got = torch.autograd.grad(flat, leaves, grad)
    dh, dx = parts(grad, h, xx)
    want = rsm.block_norm_backward(**x, dh=dh, dx=dx)
    assert all(torch.equal(a, b) for a, b in zip(got, want.values()))


def test_block_norm_of_two_parts(rsm):  # noqa: F811
    """Three rows of 100 bf16 values end on a boundary of 8 bytes."""
    (a, _, _), (b, _, _), (_, dh, _) = (inputs(n, 100, BF16, BF16, seed=n) for n in (3, 4, 7))
    b["residual"].requires_grad_(True)
    whole = torch.cat([rsm.BlockNormFunction.apply(*x.values())[0] for x in (a, b)])
    whole.backward(dh)
    want = rsm.block_norm_backward(**{n: v.detach() for n, v in b.items()}, dh=dh[3:].clone())
    assert torch.equal(b["residual"].grad, want["dresidual"])


@pytest.mark.parametrize("t", [BF16, F32])
def test_window(rsm, t):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(3)
    q, k, v = (torch.randn(1, 70, h, 64, generator=g, device="cuda").to(t).requires_grad_(True) for h in (4, 2, 2))
    o = rsm.WindowFunction.apply(q, k, v, 20, 2)
    flat, grad = behind_one(o)
    got = torch.autograd.grad(flat, (q, k, v), grad)
    r = rsm.window_forward(q.detach(), k.detach(), v.detach(), 20, 2, lse=True, low=True)
    want = rsm.window_backward(q.detach(), k.detach(), v.detach(), r["o"], r["lse"], *parts(grad, o), 20, 2, low=r["low"])
    assert all(torch.equal(a, b) for a, b in zip(got, want.values()))


def test_mixer(rsm):  # noqa: F811
    from sparse_routed_slot_b200.workloads import make_inputs
    m = make_inputs(1, 40, 2, 64, 64, F32, "head", seed=1, device="cuda")
    leaves = [m[n].clone().requires_grad_(True) for n in ("q", "k", "v", "logits", "f")]
    o, hT = rsm.RSMFunction.apply(*leaves, 8)
    flat, grad = behind_one(o, hT)
    got = torch.autograd.grad(flat, leaves, grad)
    dO, dHT = parts(grad, o, hT)
    want = rsm.backward(*(m[n] for n in ("q", "k", "v", "logits", "f")), 8, dO, dHT)
    for a, n in zip(got, ("dq", "dk", "dv", "dlogits", "df")):
        assert torch.equal(a, want[n]), n
