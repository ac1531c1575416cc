"""CPU checks of what the binding of the operators beside the mixer hands to the library: its calls on tensors
without storage, up to the C entry point, which refuses them before it reads a pointer or launches anything."""
import ctypes

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

BF16 = torch.bfloat16


@pytest.fixture()
def rsm(monkeypatch):
    import __graft_entry__
    __graft_entry__.build()
    import sparse_routed_slot_b200 as m
    from sparse_routed_slot_b200 import _lib, hybrid

    def run(fn, args, index, size_fn=None, workspace=None):
        if size_fn is not None:
            assert size_fn(ctypes.byref(args)) == hybrid._NO_SIZE
        _lib.check(fn(ctypes.byref(args), None))

    monkeypatch.setattr(hybrid, "_run", run)
    monkeypatch.setattr(hybrid, "_ptr", lambda t, *a, f=hybrid._ptr: checked(f, t, *a))
    return m


def checked(f, t, *a):
    """_ptr's checks, for a tensor whose address is None."""
    if t is not None:
        t.data_ptr = lambda: None
    return f(t, *a)


def fake(*shape, dtype=BF16):
    return torch.empty(*shape, dtype=dtype, device="cuda")


def paged(N=2, H=4, Hkv=2, D=64, pages=8, page=16, B=2, width=3):
    i32 = torch.int32
    return dict(q=fake(N, H, D), k_cache=fake(pages, page, Hkv, D), v_cache=fake(pages, page, Hkv, D),
                page_table=fake(B, width, dtype=i32), cu_q=fake(B + 1, dtype=i32), kv_len=fake(B, dtype=i32), max_q=1)


FAR = [-1, -(2**31), -(2**32), -(2**32) + 5, -(2**63)]


@pytest.mark.parametrize("x", FAR)
def test_far_negatives_are_refused(rsm, x):
    """Whatever remains of them in 32 bits: -2^32 would be zero, no window or no tokens."""
    with FakeTensorMode():
        q, k = fake(1, 9, 4, 64), fake(1, 9, 2, 64)
        for kw in (dict(window=x), dict(window=3, sinks=x)):
            with pytest.raises(rsm.RSMError, match="INVALID"):
                rsm.window_forward(q, k, k, **kw)
            with pytest.raises(rsm.RSMError, match="INVALID"):
                rsm.window_backward(q, k, k, q, fake(1, 9, 4, dtype=torch.float32), q, **kw)
        for kw in (dict(window=x), dict(window=3, sinks=x), dict(max_q=x)):
            with pytest.raises(rsm.RSMError, match="INVALID"):
                rsm.paged_forward(**{**paged(), **kw})


@pytest.mark.parametrize("n", [2**31, 2**32 + 5, 2**32 + 64])
def test_sizes_past_a_c_int_are_refused(rsm, n):
    """2^32 + 5 tokens would be taken for 5."""
    with FakeTensorMode():
        for kw in (paged(N=n, H=1, Hkv=1, D=8), paged(pages=n, page=1, Hkv=1, D=8), paged(pages=1, page=n, Hkv=1, D=8),
                   paged(B=1, width=n)):
            with pytest.raises(ValueError, match="2\\^31"):
                rsm.paged_forward(**kw)
            places = {x: kw[x] for x in ("k_cache", "v_cache", "page_table", "cu_q", "kv_len")}
            k = fake(kw["q"].shape[0], *kw["k_cache"].shape[2:])
            with pytest.raises(ValueError, match="2\\^31"):
                rsm.paged_append(k, k, **places)
        x = fake(1, n, 1, 8)
        with pytest.raises(ValueError, match="2\\^31"):
            rsm.window_forward(x, x, x, 3)
        x, w = fake(1, n), fake(n, dtype=torch.float32)
        with pytest.raises(ValueError, match="2\\^31"):
            rsm.block_norm_forward(x, None, x, w)
        with pytest.raises(ValueError, match="2\\^31"):
            rsm.block_norm_backward(x, None, x, w, dh=x)


@pytest.mark.parametrize("page", [1, 16, 64])
def test_places_close_to_2_31_are_refused(rsm, page):
    """A tile that starts below 2^31 and ends past it: its end would be negative, and all of it in sight."""
    with FakeTensorMode():
        for places in (2**31 - 64, 2**31 - 256 + page):
            kw = paged(B=1, page=page, width=places // page)
            with pytest.raises(rsm.RSMError, match="UNSUPPORTED"):
                rsm.paged_forward(**kw)
        with pytest.raises(rsm.RSMError, match="must not be NULL"):  # the next check
            rsm.paged_forward(**paged(B=1, page=page, width=(2**31 - 256) // page))
