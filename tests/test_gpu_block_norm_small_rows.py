"""GPU tests of the block norms on rows whose mean square is next to nothing, with an eps that leaves it so: the
factors 1 / rms are large, their cubes far past fp32, and the results are not."""
import pytest
import torch

from oracle import hybrid
from test_gpu_block_norm import close, inputs, rsm  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("ty,t", [(F32, F32), (BF16, BF16), (F32, BF16)])
@pytest.mark.parametrize("d", [12, 96, 1024, 2500, 8192])
@pytest.mark.parametrize("eps", [1e-20, 1e-30])
def test_tiny_rows(rsm, d, ty, t, eps):  # noqa: F811
    """Rows 1 to 4: zeros, an output of zeros, a residual of zeros beside a small output, all values small. The
    gradients' largest are of the order of 1 / eps = 1e30."""
    x, dh, dx = inputs(6, d, ty, t, seed=d)
    x["y"][1:3] = 0
    x["residual"][1] = 0
    x["residual"][3:5] *= 0 if eps == 1e-30 else 1e-12
    x["y"][3] *= 1e-12
    x["y"][4] *= 1e-17
    x["residual"][4] = 1e-16 * dh[4]
    how = dict(act="sigmoid", scale=0.7, eps=eps)
    x["gate"][3:5] = -20  # h stays small beside a normed y
    r = rsm.block_norm_forward(**x, **how)
    g = rsm.block_norm_backward(**x, dh=dh, dx=dx, **how)
    want = hybrid.block_norm(x["y"], x["gate"], x["residual"], x["w_post"], x["w_pre"], "sigmoid", 0.7, eps, dh, dx)
    for n, v in {**r, **g}.items():
        assert torch.isfinite(v).all(), n
        close(n, v, want[n])


@pytest.mark.parametrize("t", [F32, BF16])
def test_zero_rows_at_the_smallest_eps(rsm, t):  # noqa: F811
    """Only gradients that fp32 holds: of a row of zeros those of the weights and the gate, and dresidual."""
    x, dh, dx = inputs(5, 256, t, t, seed=1)
    x["y"].zero_()
    x["residual"].zero_()
    g = rsm.block_norm_backward(**x, dh=dh, dx=dx, eps=1e-37)
    want = hybrid.block_norm(x["y"], x["gate"], x["residual"], x["w_post"], x["w_pre"], "silu", 1.0, 1e-37, dh, dx)
    for n in ("dresidual", "dgate", "dw_post", "dw_pre"):
        close(n, g[n], want[n])
    assert not g["dgate"].any() and not g["dw_post"].any() and not g["dw_pre"].any() and not torch.isnan(g["dy"]).any()
