"""What the GPU tests of the operators beside the mixer share."""
import torch

HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}  # largest relative rounding of a stored value
# Four independent roundings of at most half a bf16 step (the weight, ds, the stored o behind delta and the
# result), each uniform in the worst case: 2^-8 / sqrt(3) rms apiece. A wrong mask moves a row by about
# 1/sqrt(keys seen), far above it. In fp32 the sums' own errors stay under 2^-16.
RMS = {torch.float32: 2.0 ** -16, torch.bfloat16: 2.0 ** -8 * (4 / 3) ** 0.5}


def within(name, got, value, bound, rms=True):
    """Every element within its own bound, and the whole within the rms of its roundings."""
    g = got.detach().double()
    assert torch.isfinite(g).equal(torch.isfinite(value)), f"{name}: finite in other places"
    fine = torch.isfinite(value)
    assert torch.equal(g[~fine], value[~fine]), f"{name}: other infinities"
    err = (g - value)[fine].abs()
    over = err > bound[fine] + 1e-30
    assert not over.any(), f"{name}: {int(over.sum())} of {over.numel()} beyond their bound, worst {float((err / (bound[fine] + 1e-30)).max()):.3g} times"
    norm = value[fine].norm()
    if rms and norm > 0:
        off = float(err.norm() / norm)
        assert off <= RMS[got.dtype], f"{name}: {off:.3g} of the values' norm"


def roundings(dtype):
    """(u, uo) of oracle.hybrid.attend: bf16 inputs round the softmax weights, ds, and the results."""
    return (0.0, 0.0) if dtype == torch.float32 else (HALF_STEP[dtype], HALF_STEP[dtype])
