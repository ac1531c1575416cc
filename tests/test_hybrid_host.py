"""CPU checks of the operators beside the mixer: the C structs' layouts, every refusal (nothing is
launched), and the 64-bit forms that the GPU tests compare with (gradients against central
differences, and hand-made masks)."""
import ctypes
import os
import subprocess

import pytest
import torch

from oracle import hybrid

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 1 << 20  # an aligned pointer that is never read: every call below is refused first


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    from sparse_routed_slot_b200 import _lib
    return _lib


def test_struct_layouts_match_c(lib, tmp_path):
    structs = {"rsm_window_args": lib.WindowArgs, "rsm_window_backward_args": lib.WindowBackwardArgs,
               "rsm_paged_append_args": lib.PagedAppendArgs, "rsm_paged_args": lib.PagedArgs,
               "rsm_block_norm_args": lib.BlockNormArgs, "rsm_block_norm_backward_args": lib.BlockNormBackwardArgs}
    body = ""
    for c, py in structs.items():
        body += f'printf("%zu\\n", sizeof({c}));'
        for name, _ in py._fields_:
            body += f'printf("%zu\\n", offsetof({c}, {name}));'
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "rsm.h"\nint main(void){' + body + "return 0;}\n")
    exe = tmp_path / "s"
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)])
    got = list(map(int, subprocess.check_output([str(exe)]).split()))
    want = []
    for py in structs.values():
        want += [ctypes.sizeof(py)] + [getattr(py, n).offset for n, _ in py._fields_]
    assert got == want


def _filled(a, **kw):
    for n, t in a._fields_:
        if t is ctypes.c_void_p:
            setattr(a, n, FAKE)
    for n, v in kw.items():
        setattr(a, n, v)
    return a


def _window(lib, cls, **kw):
    base = dict(B=2, T=9, H=4, Hkv=2, D=64, window=4, sinks=1, dtype=1, scale=0.125)
    return _filled(cls(), **{**base, **kw})


BAD_WINDOW = [(dict(D=12), 2), (dict(D=264), 2), (dict(D=0), 1), (dict(Hkv=3), 1), (dict(Hkv=0), 1), (dict(window=0), 1),
              (dict(window=-5), 1), (dict(sinks=-1), 1), (dict(B=-1), 1), (dict(T=-1), 1), (dict(H=-4), 1),
              (dict(dtype=5), 1), (dict(scale=0.0), 1), (dict(scale=-1.0), 1), (dict(scale=float("inf")), 1),
              (dict(scale=float("nan")), 1), (dict(q=None), 1), (dict(k=None), 1), (dict(v=FAKE + 4), 1), (dict(o=None), 1),
              (dict(lse=FAKE + 8), 1), (dict(H=130, Hkv=2), 2), (dict(T=1 << 30), 2)]


@pytest.mark.parametrize("kw,code", BAD_WINDOW)
def test_window_forward_refuses(lib, kw, code):
    a = _window(lib, lib.WindowArgs, **kw)
    assert lib.load().rsm_window_forward(ctypes.byref(a), None) == code and lib.last_error()


@pytest.mark.parametrize("kw,code", BAD_WINDOW + [(dict(dO=None), 1), (dict(lse=None), 1), (dict(dk=FAKE + 2), 1),
                                                  (dict(workspace=None), 5), (dict(workspace_bytes=3), 5),
                                                  (dict(workspace=FAKE + 16, workspace_bytes=1 << 20), 1)])
def test_window_backward_refuses(lib, kw, code):
    a = _window(lib, lib.WindowBackwardArgs, **kw)
    assert lib.load().rsm_window_backward(ctypes.byref(a), None) == code and lib.last_error()
    if code in (1, 2) and "workspace" not in kw:
        assert lib.load().rsm_window_backward_workspace_size(ctypes.byref(a)) == ctypes.c_size_t(-1).value


@pytest.mark.parametrize("kw", [dict(B=0), dict(T=0), dict(H=0, Hkv=0)])
def test_window_without_rows_does_nothing(lib, kw):
    for cls, call in ((lib.WindowArgs, "rsm_window_forward"), (lib.WindowBackwardArgs, "rsm_window_backward")):
        a = _window(lib, cls, q=None, k=None, v=None, o=None, **kw)
        assert getattr(lib.load(), call)(ctypes.byref(a), None) == 0


def _paged(lib, cls, **kw):
    base = dict(B=2, N=5, D=64, Hkv=2, num_pages=8, page_size=16, table_width=4, dtype=1)
    if cls is lib.PagedArgs:
        base.update(H=4, max_q=3, window=0, sinks=0, scale=0.125, workspace_bytes=1 << 30)
    return _filled(cls(), **{**base, **kw})


BAD_CACHE = [(dict(D=20), 2), (dict(D=0), 1), (dict(B=-1), 1), (dict(N=-1), 1), (dict(num_pages=-1), 1), (dict(page_size=0), 1),
             (dict(table_width=-1), 1), (dict(table_width=1 << 20, page_size=1 << 12), 2), (dict(k_cache=None), 1),
             (dict(v_cache=FAKE + 8), 1), (dict(page_table=None), 1), (dict(cu_q=None), 1), (dict(kv_len=None), 1),
             (dict(dtype=2), 1)]


@pytest.mark.parametrize("kw,code", BAD_CACHE + [(dict(k=None), 1), (dict(v=FAKE + 1), 1)])
def test_paged_append_refuses(lib, kw, code):
    a = _paged(lib, lib.PagedAppendArgs, **kw)
    assert lib.load().rsm_paged_append(ctypes.byref(a), None) == code and lib.last_error()


@pytest.mark.parametrize("kw,code", BAD_CACHE + [(dict(q=None), 1), (dict(o=FAKE + 8), 1), (dict(lse=FAKE + 4), 1),
                                                 (dict(Hkv=3), 1), (dict(max_q=-1), 1), (dict(window=-1), 1),
                                                 (dict(sinks=-1), 1), (dict(scale=0.0), 1), (dict(N=1 << 30, H=4), 2)])
def test_paged_forward_refuses(lib, kw, code):
    a = _paged(lib, lib.PagedArgs, **kw)
    assert lib.load().rsm_paged_forward(ctypes.byref(a), None) == code and lib.last_error()
    assert lib.load().rsm_paged_workspace_size(ctypes.byref(a)) == ctypes.c_size_t(-1).value


def test_paged_forward_asks_for_its_workspace(lib):
    a = _paged(lib, lib.PagedArgs, B=1, N=1, max_q=1, table_width=4096)
    need = lib.load().rsm_paged_workspace_size(ctypes.byref(a))
    assert 0 < need < 1 << 26
    for ws, size, code in ((None, 0, 5), (FAKE, need - 1, 5), (FAKE + 16, need, 1)):
        a.workspace, a.workspace_bytes = ws, size
        assert lib.load().rsm_paged_forward(ctypes.byref(a), None) == code and lib.last_error()


@pytest.mark.parametrize("kw", [dict(N=0), dict(B=0), dict(max_q=0)])
def test_paged_without_tokens_does_nothing(lib, kw):
    a = _paged(lib, lib.PagedArgs, **kw)
    assert lib.load().rsm_paged_forward(ctypes.byref(a), None) == 0
    assert lib.load().rsm_paged_workspace_size(ctypes.byref(a)) == 0
    if "max_q" not in kw:
        a = _paged(lib, lib.PagedAppendArgs, **kw)
        assert lib.load().rsm_paged_append(ctypes.byref(a), None) == 0


def _norm(lib, cls, **kw):
    base = dict(rows=7, d=64, y_dtype=1, dtype=1, act=0, scale=0.5, eps=1e-6)
    return _filled(cls(), **{**base, **kw})


BAD_NORM = [(dict(d=66), 2), (dict(d=8196), 2), (dict(d=0), 1), (dict(rows=-1), 1), (dict(rows=1 << 31), 2),
            (dict(y_dtype=1, dtype=0), 2), (dict(dtype=3), 1), (dict(act=2), 1), (dict(scale=float("nan")), 1),
            (dict(eps=0.0), 1), (dict(eps=float("inf")), 1), (dict(y=None), 1), (dict(residual=None), 1),
            (dict(w_post=None), 1), (dict(gate=FAKE + 8), 1)]


@pytest.mark.parametrize("kw,code", BAD_NORM + [(dict(h=None), 1), (dict(x=None), 1), (dict(w_pre=None), 1)])
def test_block_norm_refuses(lib, kw, code):
    a = _norm(lib, lib.BlockNormArgs, **kw)
    assert lib.load().rsm_block_norm_forward(ctypes.byref(a), None) == code and lib.last_error()


@pytest.mark.parametrize("kw,code", BAD_NORM + [(dict(w_pre=None), 1), (dict(gate=None), 1), (dict(dy=FAKE + 4), 1),
                                                (dict(w_pre=None, dx=None), 1), (dict(workspace=None), 5),
                                                (dict(workspace_bytes=8), 5)])
def test_block_norm_backward_refuses(lib, kw, code):
    a = _norm(lib, lib.BlockNormBackwardArgs, **kw)
    assert lib.load().rsm_block_norm_backward(ctypes.byref(a), None) == code and lib.last_error()


def test_binding_refuses_cpu_tensors(lib):
    import sparse_routed_slot_b200 as rsm
    x = torch.zeros(1, 4, 2, 8)
    with pytest.raises(ValueError, match="CUDA"):
        rsm.window_forward(x, x, x, 2)
    with pytest.raises(ValueError, match="CUDA"):
        rsm.block_norm_forward(x, None, x, torch.ones(8))
    with pytest.raises(ValueError, match="CUDA"):
        rsm.paged_append(x[0], x[0], x, x, torch.zeros(1, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                         torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="float32 or bfloat16"):
        rsm.window_forward(x.half(), x.half(), x.half(), 2)


# ------------------------------------------------------------------------------- the 64-bit forms
def _differences(f, x, h=1e-5):
    g = torch.zeros_like(x)
    for i in range(x.numel()):
        v = x.reshape(-1)[i].item()
        x.reshape(-1)[i] = v + h
        up = f().item()
        x.reshape(-1)[i] = v - h
        down = f().item()
        x.reshape(-1)[i] = v
        g.reshape(-1)[i] = (up - down) / (2 * h)
    return g


def test_window_form_sees_what_it_should():
    """One key at a time carries a marker: the row sees it exactly under the rule."""
    T, W, S = 11, 3, 2
    q = torch.zeros(1, T, 1, 8)
    v = torch.eye(T)[None, :, None, :]
    o = hybrid.attend(q[0], q[0], torch.cat([v[0], v[0]], 2), torch.arange(T), W, S, 1.0)["o"][0][:, 0, :T]
    for i in range(T):
        for j in range(T):
            seen = j <= i and (i - j < W or j < S)
            assert (o[i, j] > 0) == seen, (i, j)
    assert torch.allclose(o.sum(1), torch.ones(T, dtype=torch.float64))


def test_window_form_empty_rows():
    q = torch.randn(3, 2, 8)
    r = hybrid.attend(q, torch.randn(4, 1, 8), torch.randn(4, 1, 8), torch.tensor([-2, -1, 0]), 0, 0, 1.0)
    assert (r["o"][0][:2] == 0).all() and (r["lse"][0][:2] == float("-inf")).all() and (r["o"][0][2] != 0).any()


def test_window_form_gradients_match_differences():
    g = torch.Generator().manual_seed(1)
    q, k, v, do = (torch.randn(1, 7, h, 4, generator=g, dtype=torch.float64) for h in (4, 2, 2, 4))
    r = hybrid.window(q, k, v, 3, 1, 0.6, do)
    f = lambda: (hybrid.window(q, k, v, 3, 1, 0.6)["o"][0] * do).sum()  # noqa: E731
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        assert torch.allclose(r[name][0], _differences(f, x), rtol=1e-6, atol=1e-8), name


@pytest.mark.parametrize("act,gated", [("silu", True), ("sigmoid", True), ("silu", False)])
def test_block_norm_form_gradients_match_differences(act, gated):
    g = torch.Generator().manual_seed(2)
    y, gate, res, dh, dx = (torch.randn(3, 8, generator=g, dtype=torch.float64) for _ in range(5))
    w1, w2 = (torch.randn(8, generator=g, dtype=torch.float64) for _ in range(2))
    gate = gate if gated else None
    r = hybrid.block_norm(y, gate, res, w1, w2, act, 0.7, 1e-3, dh, dx)

    def f():
        t = hybrid.block_norm(y, gate, res, w1, w2, act, 0.7, 1e-3)
        return (t["h"] * dh).sum() + (t["x"] * dx).sum()

    for name, x in (("dy", y), ("dgate", gate), ("dresidual", res), ("dw_post", w1), ("dw_pre", w2)):
        if x is not None:
            assert torch.allclose(r[name], _differences(f, x), rtol=1e-6, atol=1e-8), name
