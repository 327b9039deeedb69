"""Host-only checks (no GPU) of the 8-bit products' and the cross entropy's
entry points: struct layout, workspace queries, and refusals, which come
before any launch."""

import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 20   # a non-null, aligned address that nothing dereferences


@pytest.fixture(scope="module")
def mir():
    import matrix_inverse_roots_amd as m
    return m


def test_xent_args_layout_matches_header(mir, tmp_path):
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "shampoo.h"', "int main(void) {",
             'printf("size %zu\\n", sizeof(shampoo_xent_args));']
    for f, _ in mir.XentArgsC._fields_:
        lines.append('printf("%s %%zu\\n", offsetof(shampoo_xent_args, %s));' % (f, f))
    lines += ["return 0;", "}"]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines))
    subprocess.run(["gcc", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I", "/opt/rocm/include",
                    str(src), "-o", str(exe)], check=True, capture_output=True)
    out = dict(l.split() for l in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    assert int(out.pop("size")) == ctypes.sizeof(mir.XentArgsC)
    for f, off in out.items():
        assert int(off) == getattr(mir.XentArgsC, f).offset, f


QUANT = dict(x=P, dt="f32", n=1, rows=4, cols=8, ld=8, stride=32, fmt="e4m3", rb=1, q=P, s=P, qt=None, st=None)


def quantize(mir, **kw):
    a = {**QUANT, **kw}
    codes = {**mir.DTYPES, "e4m3": mir.E4M3, "e5m2": mir.E5M2}
    return mir.lib.shampoo_quantize_f8(a["x"], codes.get(a["dt"], a["dt"]), a["n"], a["rows"], a["cols"], a["ld"],
                                       a["stride"], codes.get(a["fmt"], a["fmt"]), a["rb"], a["q"], a["s"], a["qt"],
                                       a["st"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), 1), (dict(rows=-1), 1), (dict(cols=-5), 1), (dict(dt="f64"), 2), (dict(dt="e4m3"), 2),
    (dict(fmt="f32"), 2), (dict(rb=2), 2), (dict(n=65536), 2), (dict(rows=1 << 23), 2), (dict(cols=1 << 23), 2),
    (dict(s=None), 1), (dict(q=None), 1), (dict(q=None, s=None), 1), (dict(qt=P), 1), (dict(x=None), 1),
    (dict(ld=7), 1), (dict(q=P + 8), 1), (dict(s=P + 2), 1), (dict(x=P + 2), 1), (dict(n=2, stride=-1), 1),
])
def test_quantize_refusals(mir, kw, status):
    assert quantize(mir, **kw) == status
    assert mir.lib.shampoo_last_error()


def test_empty_quantize_returns_at_once(mir):
    for kw in (dict(n=0), dict(rows=0), dict(cols=0)):
        assert quantize(mir, x=None, q=None, s=None, **kw) == mir.OK


PROD = dict(a=P, adt=4, sa=P, arb=1, b=P, bdt=5, sb=P, brb=128, n=1, M=4, N=8, K=128, c=P, cdt=0, ws=None, wsb=0)


def product(mir, **kw):
    a = {**PROD, **kw}
    return mir.lib.shampoo_matmul_f8(a["a"], a["adt"], a["sa"], a["arb"], a["b"], a["bdt"], a["sb"], a["brb"], a["n"],
                                     a["M"], a["N"], a["K"], a["c"], a["cdt"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(K=0), 1), (dict(K=100), 1), (dict(K=-128), 1), (dict(M=-1), 1), (dict(n=-1), 1), (dict(n=65536), 2),
    (dict(M=1 << 23), 2), (dict(adt=0), 2), (dict(bdt=2), 2), (dict(cdt=3), 2), (dict(cdt=4), 2), (dict(arb=64), 2),
    (dict(brb=0), 2), (dict(a=None), 1), (dict(sb=None), 1), (dict(c=None), 1), (dict(a=P + 8), 1), (dict(sa=P + 1), 1),
    (dict(c=P + 2), 1), (dict(M=64, N=64, K=8192), 3), (dict(M=64, N=64, K=8192, ws=P, wsb=100), 3),
    (dict(M=64, N=64, K=8192, ws=P + 64, wsb=1 << 30), 3),
])
def test_product_refusals(mir, kw, status):
    assert product(mir, **kw) == status
    assert mir.lib.shampoo_last_error()


def test_product_workspace(mir):
    assert mir.shampoo_matmul_f8_workspace(144, 1024, 1024, 1024) == 0
    assert mir.shampoo_matmul_f8_workspace(0, 5, 5, 128) == 0
    need = mir.shampoo_matmul_f8_workspace(1, 64, 64, 8192)
    assert need >= 2 * 64 * 64 * 4
    with pytest.raises(mir.ShampooError):
        mir.shampoo_matmul_f8_workspace(1, 64, 64, 100)
    assert product(mir, M=0) == mir.OK and product(mir, n=0, a=None) == mir.OK


def xent(mir, launch=False, **kw):
    a = mir.XentArgsC(hidden=P, weight=P, targets=P, loss=P, ld_hidden=64, ld_weight=64, ld_dhidden=64, ld_dweight=64,
                      N=10, V=100, d=64, ignore_index=-100, dt=mir.BF16, weight_dt=mir.BF16, dweight_dt=mir.BF16,
                      logits_dt=mir.BF16, reduction=2, scale=1.0, ws=P, ws_bytes=1 << 30)
    for k, v in kw.items():
        setattr(a, k, v)
    if launch:
        return mir.lib.shampoo_linear_xent(ctypes.byref(a), None)
    b = ctypes.c_size_t(0)
    return mir.lib.shampoo_linear_xent_workspace(ctypes.byref(a), ctypes.byref(b)), b.value


@pytest.mark.parametrize("kw,status", [
    (dict(N=-1), 1), (dict(V=0), 1), (dict(d=0), 1), (dict(dt=1), 2), (dict(dt=3), 2), (dict(weight_dt=1), 2),
    (dict(dt=0, weight_dt=2, logits_dt=0), 2), (dict(dweight=P, dweight_dt=1), 2), (dict(dt=0, weight_dt=0, logits_dt=0, dweight=P), 2),
    (dict(reduction=3), 1), (dict(reduction=-1), 1), (dict(V=1 << 21), 2), (dict(d=1 << 20), 2), (dict(panel_rows=-1), 1),
    (dict(N=1 << 30), 2), (dict(logits_dt=0), 2), (dict(logits_dt=5), 2), (dict(dt=0, weight_dt=0, logits_dt=4), 2),
    (dict(logits_dt=4, N=1 << 24), 2), (dict(ld_weight=1 << 21), 2),
])
def test_xent_refusals_of_both_calls(mir, kw, status):
    assert xent(mir, **kw)[0] == status
    assert xent(mir, True, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(hidden=None), 1), (dict(weight=None), 1), (dict(targets=None), 1), (dict(loss=None), 1), (dict(ld_hidden=63), 1),
    (dict(ld_weight=0), 1), (dict(dhidden=2 * P, ld_dhidden=32), 1), (dict(dweight=2 * P, ld_dweight=32), 1),
    (dict(hidden=P + 1), 1), (dict(targets=P + 4), 1), (dict(loss=P + 2), 1), (dict(lse=P + 1), 1), (dict(row_scale=P + 2), 1),
    (dict(dweight=2 * P + 2, dweight_dt=0), 1), (dict(weight=P + 2, weight_dt=0), 1),
    (dict(dhidden=P), 1), (dict(dweight=P), 1), (dict(dhidden=P, hidden=P, dweight=2 * P), 1),
    (dict(ws=None), 3), (dict(ws_bytes=100), 3), (dict(ws=P + 16), 3),
])
def test_xent_refusals_of_the_call(mir, kw, status):
    assert xent(mir, True, **kw) == status
    assert mir.lib.shampoo_last_error()


A, B, C, D, E, F, G, H = (k << 24 for k in range(1, 9))   # addresses 16 MiB apart


def xent_apart(mir, **kw):
    """A call whose memory lies apart but for what `kw` says (no GPU here: E_HIP once it is let through)."""
    lib = mir.lib
    status = xent(mir, True, **{**dict(hidden=A, weight=B, targets=C, loss=D, dhidden=E, dweight=F, lse=G, ws=H, ws_bytes=1 << 22), **kw})
    return status, lib.shampoo_last_error().decode()


@pytest.mark.parametrize("kw,names", [
    (dict(dhidden=A), "dhidden overlaps hidden"), (dict(dhidden=A + 128), "dhidden overlaps hidden"),
    (dict(dhidden=A - 128), "dhidden overlaps hidden"), (dict(dhidden=A + 10 * 128 - 2), "dhidden overlaps hidden"),
    (dict(dhidden=B + 256), "dhidden overlaps weight"), (dict(dweight=B + 2), "dweight overlaps weight"),
    (dict(dweight=A - 99 * 128), "dweight overlaps hidden"), (dict(dhidden=F + 640), "dhidden overlaps dweight"),
    (dict(dweight=B - 4, dweight_dt=0), "dweight overlaps weight"), (dict(loss=A), "loss overlaps hidden"),
    (dict(loss=C + 76), "loss overlaps targets"), (dict(row_scale=G + 36), "lse overlaps row_scale"),
    (dict(ws=A & ~255), "the workspace overlaps hidden"), (dict(lse=D - 36), "loss overlaps lse"),
    # views of one wider matrix: a window that meets the other's, and rows of another distance
    (dict(ld_hidden=128, ld_dhidden=128, dhidden=A + 126), "dhidden overlaps hidden"),
    (dict(ld_hidden=128, ld_dhidden=128, dhidden=A + 256 + 130), "dhidden overlaps hidden"),
    (dict(ld_hidden=128, ld_dhidden=192, dhidden=A + 128), "dhidden overlaps hidden"),
    (dict(N=1, dhidden=A + 2), "dhidden overlaps hidden"),
])
def test_xent_refuses_overlaps(mir, kw, names):
    status, message = xent_apart(mir, **kw)
    assert status == mir.E_INVALID and message == names


@pytest.mark.parametrize("kw", [
    dict(), dict(dhidden=A + 10 * 128), dict(dhidden=A - 10 * 128), dict(hidden=B), dict(weight=A),
    dict(ld_hidden=128, ld_dhidden=128, dhidden=A + 128), dict(ld_hidden=128, ld_dhidden=128, dhidden=A - 128),
    dict(ld_hidden=200, ld_dhidden=200, dhidden=A + 128 + 400), dict(N=1, ld_hidden=64, dhidden=A + 128), dict(dweight=None, dhidden=None),
    dict(ld_dhidden=128, dhidden=E, ld_dweight=128, dweight=E + 128), dict(lse=None, row_scale=G),
])
def test_xent_lets_neighbours_through(mir, kw):
    import torch
    if torch.cuda.is_available():
        pytest.skip("made-up addresses: for a machine without a GPU")
    status, message = xent_apart(mir, **kw)
    assert status == mir.E_HIP and "overlaps" not in message


@pytest.mark.parametrize("kw,names", [
    (dict(q=A + 16), "q overlaps x"), (dict(s=A), "s overlaps x"), (dict(q=B, s=B + 508), "q overlaps s"),
    (dict(q=None, s=None, qt=A - 16, st=E), "qt overlaps x"), (dict(q=B, s=C, qt=B + 256, st=E), "q overlaps qt"),
    (dict(n=3, stride=1 << 20, q=A + (2 << 22)), "q overlaps x"),
])
def test_quantize_refuses_overlaps(mir, kw, names):
    assert quantize(mir, **{**dict(x=A, q=B, s=C), **kw}) == mir.E_INVALID
    assert mir.lib.shampoo_last_error().decode() == names


@pytest.mark.parametrize("kw,names", [
    (dict(c=A), "c overlaps a"), (dict(c=B + 1020), "c overlaps b"), (dict(c=C - 124), "c overlaps a_scale"), (dict(c=D), "c overlaps b_scale"),
    (dict(M=64, N=64, K=8192, ws=A, wsb=1 << 30), "the workspace overlaps a"), (dict(M=64, N=64, K=8192, c=F, ws=F, wsb=1 << 30), "c overlaps the workspace"),
])
def test_product_refuses_overlaps(mir, kw, names):
    assert product(mir, **{**dict(a=A, b=B, sa=C, sb=D, c=E), **kw}) == mir.E_INVALID
    assert mir.lib.shampoo_last_error().decode() == names


def test_xent_workspace_is_bounded_by_the_panel(mir):
    """The exponentials of panel_rows rows, not of all; none without gradients."""
    big = dict(N=1 << 16, V=131072, d=64, dhidden=P, dweight=P)
    st, full = xent(mir, **big)
    assert st == mir.OK and full < 4 << 30
    st, small = xent(mir, panel_rows=256, **big)
    assert st == mir.OK and small < full // 4
    st, alone = xent(mir, **{**big, "dhidden": None, "dweight": None})
    assert st == mir.OK and alone < 1 << 30
    st, none = xent(mir, N=0)
    assert st == mir.OK and none < 1 << 16


@pytest.mark.parametrize("V", [65536, 100000, 131072, 131073, 262144])
def test_xent_default_panel(mir, V):
    """2 GiB of exponentials at every width: a batch that they hold is one panel, 256 rows more are two."""
    rows = (1 << 31) // (-(-V // 128) * 256) // 256 * 256
    for N, panel in ((rows, rows), (rows + 256, (rows + 256 + 511) // 512 * 256)):
        kw = dict(N=N, V=V, dhidden=P, dweight=P)
        assert xent(mir, **kw)[1] == xent(mir, panel_rows=panel, **kw)[1] > 0
        assert xent(mir, **kw)[1] != xent(mir, panel_rows=panel - 256, **kw)[1]


def test_python_checks_need_no_gpu(mir):
    import torch
    x = torch.zeros(4, 256)
    with pytest.raises(ValueError, match="device tensors"):
        mir.shampoo_quantize_f8(x)
    for kw in (dict(fmt="e3m4"), dict(block_rows=2), dict(transpose="yes")):
        with pytest.raises(ValueError):
            mir.shampoo_quantize_f8(x, **kw)
    with pytest.raises(TypeError):
        mir.shampoo_quantize_f8(x.double())
    with pytest.raises(ValueError):
        mir.shampoo_quantize_f8(x[0])
    with pytest.raises(ValueError, match="device tensors"):
        mir.shampoo_linear_xent(x, x, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        mir.shampoo_linear_xent_workspace(x, torch.zeros(5, 255), torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        mir.shampoo_linear_xent_workspace(x, x, torch.zeros(4, dtype=torch.int32))
    assert mir.shampoo_linear_xent_workspace(x, x, torch.zeros(4, dtype=torch.int64)) > 0


def test_stream_of_another_device_is_refused(mir):
    import types
    import torch
    there = types.SimpleNamespace(device=torch.device("cuda:1"), cuda_stream=0)
    here = torch.device("cuda:0")
    launched = []
    with pytest.raises(ValueError, match="stream of cuda:1"):
        mir._launch(lambda *a: launched.append(a), here, there)
    with pytest.raises(ValueError, match="stream of cuda:1"):
        mir._empty((4,), torch.float32, here, there)
    assert not launched
