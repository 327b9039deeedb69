"""Host-only checks (no GPU) of the feed-forward layers' entry points: struct
layouts, workspace queries, and refusals, which come before any launch."""

import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
P = 1 << 32   # a non-null, aligned address that nothing dereferences; buffers are P apart


@pytest.fixture(scope="module")
def mir():
    import matrix_inverse_roots_amd as m
    return m


STRUCTS = [("shampoo_linear_args", "LinearArgsC"), ("shampoo_linear_grad_args", "LinearGradArgsC"),
           ("shampoo_gated_ffn_args", "GatedArgsC"), ("shampoo_gated_ffn_grad_args", "GatedGradArgsC")]


@pytest.mark.parametrize("c,py", STRUCTS)
def test_layouts_match_header(mir, tmp_path, c, py):
    struct = getattr(mir, py)
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "shampoo.h"', "int main(void) {",
             'printf("size %%zu\\n", sizeof(%s));' % c]
    for f, _ in struct._fields_:
        lines.append('printf("%s %%zu\\n", offsetof(%s, %s));' % (f, c, f))
    lines += ["return 0;", "}"]
    src, exe = tmp_path / "layout.c", tmp_path / "layout"
    src.write_text("\n".join(lines))
    subprocess.run(["gcc", "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(ROOT, "include"), "-I", "/opt/rocm/include",
                    str(src), "-o", str(exe)], check=True, capture_output=True)
    out = dict(l.split() for l in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    assert int(out.pop("size")) == ctypes.sizeof(struct)
    for f, off in out.items():
        assert int(off) == getattr(struct, f).offset, f


def call(mir, name, struct, given, kw, launch):
    a = getattr(mir, struct)(**{**given, **kw})
    if launch:
        return getattr(mir.lib, name)(ctypes.byref(a), None)
    b = ctypes.c_size_t(0)
    return getattr(mir.lib, name + "_workspace")(ctypes.byref(a), ctypes.byref(b)), b.value


LINEAR = dict(x=P, w=2 * P, y=3 * P, ld_x=64, ld_w=64, ld_residual=96, ld_y=96, ld_keep=96, M=10, N=96, K=64, dt=2, w_dt=2,
              bias_dt=0, y_dt=2, keep_dt=2, ws=10 * P, ws_bytes=1 << 30)


def linear(mir, launch=False, **kw):
    return call(mir, "shampoo_linear", "LinearArgsC", LINEAR, kw, launch)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), 1), (dict(N=0), 1), (dict(K=0), 1), (dict(dt=1), 2), (dict(dt=3), 2), (dict(w_dt=1), 2), (dict(dt=0, y_dt=0), 2),
    (dict(y_dt=1), 2), (dict(y_dt=4), 2), (dict(activation=5), 1), (dict(activation=-1), 1), (dict(bias=P, bias_dt=1), 2),
    (dict(keep=4 * P, keep_dt=0), 2), (dict(keep=4 * P, keep_dt=5), 2), (dict(M=1 << 30), 2), (dict(N=1 << 19), 2), (dict(K=1 << 19), 2),
])
def test_linear_refusals_of_both_calls(mir, kw, status):
    assert linear(mir, **kw)[0] == status
    assert linear(mir, True, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(y=None), 1), (dict(ld_x=63), 1), (dict(ld_w=0), 1), (dict(ld_y=95), 1),
    (dict(residual=4 * P, ld_residual=95), 1), (dict(ld_x=1 << 21), 2), (dict(x=P + 1), 1), (dict(y=3 * P + 1), 1),
    (dict(w_dt=0, w=2 * P + 2), 1), (dict(bias=4 * P + 2), 1), (dict(keep=4 * P + 1), 1), (dict(keep=4 * P, ld_keep=95), 1),
    (dict(keep=4 * P, keep_dt=4), 1), (dict(keep=4 * P + 8, keep_dt=4, keep_scale=5 * P), 1),
    (dict(y=P), 1), (dict(y=2 * P), 1), (dict(y=10 * P, ld_x=65), 1), (dict(keep=3 * P), 1), (dict(residual=3 * P + 2), 1),
    (dict(residual=3 * P, ld_residual=128), 1), (dict(bias=3 * P), 1), (dict(keep=4 * P, keep_dt=4, keep_scale=3 * P), 1),
    (dict(M=40, K=8192, ld_x=8192, ld_w=8192, ws=None), 3), (dict(M=40, K=8192, ld_x=8192, ld_w=8192, ws_bytes=100), 3),
    (dict(M=40, K=8192, ld_x=8192, ld_w=8192, ws=10 * P + 16), 3),
])
def test_linear_refusals_of_the_call(mir, kw, status):
    assert linear(mir, True, **kw) == status
    assert mir.lib.shampoo_last_error()


def test_linear_workspace(mir):
    assert linear(mir) == (mir.OK, 0)                                   # ten rows: no copies, one range of k
    assert linear(mir, M=4, K=100, ld_x=101, ld_w=103)[1] == 0          # few rows take any stride
    assert linear(mir, ld_x=65)[1] >= 10 * 64 * 2                       # rows that do not start on 16 bytes
    assert linear(mir, w_dt=0)[1] >= 96 * 64 * 2                        # a float32 weight beside bfloat16
    assert linear(mir, M=40, K=8192, ld_x=8192, ld_w=8192)[1] >= 2 * 40 * 96 * 4
    assert linear(mir, M=0)[0] == mir.OK and linear(mir, True, M=0, x=None, y=None, ws=None) == mir.OK
    assert mir.lib.shampoo_linear_workspace(None, ctypes.byref(ctypes.c_size_t())) == 1
    assert mir.lib.shampoo_linear(None, None) == 1


GRAD = dict(dy=P, x=2 * P, w=3 * P, kept=4 * P, dx=5 * P, dw=6 * P, dbias=7 * P, ld_dy=96, ld_x=64, ld_w=64, ld_kept=96, ld_dx=64,
            ld_dw=64, M=10, N=96, K=64, dt=2, x_dt=2, w_dt=2, kept_dt=2, dw_dt=2, dbias_dt=0, activation=2, ws=10 * P, ws_bytes=1 << 30)


def grad(mir, launch=False, **kw):
    return call(mir, "shampoo_linear_grad", "LinearGradArgsC", GRAD, kw, launch)


@pytest.mark.parametrize("kw,status", [
    (dict(M=-1), 1), (dict(N=0), 1), (dict(K=-3), 1), (dict(dt=1), 2), (dict(w_dt=1), 2), (dict(x_dt=0), 2), (dict(x_dt=5), 2),
    (dict(kept_dt=0), 2), (dict(kept_dt=5), 2), (dict(dw_dt=1), 2), (dict(dbias_dt=1), 2), (dict(activation=9), 1), (dict(M=1 << 30), 2),
])
def test_grad_refusals_of_both_calls(mir, kw, status):
    assert grad(mir, **kw)[0] == status
    assert grad(mir, True, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dx=None, dw=None, dbias=None), 1), (dict(dy=None), 1), (dict(x=None), 1), (dict(w=None), 1), (dict(kept=None), 1),
    (dict(ld_dy=95), 1), (dict(ld_x=63), 1), (dict(ld_w=63), 1), (dict(ld_kept=95), 1), (dict(ld_dx=63), 1), (dict(ld_dw=63), 1),
    (dict(x_dt=4), 1), (dict(x_dt=4, x_scale=8 * P, x=2 * P + 8), 1), (dict(kept_dt=4), 1), (dict(kept_dt=4, kept_scale=8 * P, kept=4 * P + 8), 1),
    (dict(dy=P + 1), 1), (dict(dw=6 * P + 2, dw_dt=0), 1), (dict(dbias=7 * P + 2), 1),
    (dict(dx=P), 1), (dict(dw=3 * P), 1), (dict(dw=5 * P), 1), (dict(dbias=6 * P), 1), (dict(dx=4 * P), 1), (dict(dw=2 * P), 1),
    (dict(x_dt=4, x_scale=6 * P), 1), (dict(kept_dt=4, kept_scale=5 * P), 1),
    (dict(ws=None), 3), (dict(ws_bytes=64), 3), (dict(ws=10 * P + 128), 3),
])
def test_grad_refusals_of_the_call(mir, kw, status):
    assert grad(mir, True, **kw) == status
    assert mir.lib.shampoo_last_error()


GATED = dict(x=P, w_gate=2 * P, w_up=3 * P, w_down=4 * P, y=5 * P, ld_x=64, ld_gate=64, ld_up=64, ld_down=96, ld_residual=64, ld_y=64,
             ld_keep=96, T=10, d=64, f=96, dt=2, w_dt=2, y_dt=2, keep_dt=2, activation=4, ws=10 * P, ws_bytes=1 << 30)


def gated(mir, launch=False, **kw):
    return call(mir, "shampoo_gated_ffn", "GatedArgsC", GATED, kw, launch)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(d=0), 1), (dict(f=0), 1), (dict(dt=1), 2), (dict(w_dt=1), 2), (dict(y_dt=1), 2), (dict(activation=5), 1),
    (dict(keep_gate=6 * P), 1), (dict(keep_up=6 * P), 1), (dict(keep_gate=6 * P, keep_up=7 * P, keep_dt=1), 2), (dict(f=1 << 19), 2), (dict(T=1 << 30), 2),
])
def test_gated_refusals_of_both_calls(mir, kw, status):
    assert gated(mir, **kw)[0] == status
    assert gated(mir, True, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(w_gate=None), 1), (dict(w_up=None), 1), (dict(w_down=None), 1), (dict(y=None), 1),
    (dict(ld_x=63), 1), (dict(ld_gate=63), 1), (dict(ld_up=63), 1), (dict(ld_down=95), 1), (dict(ld_y=63), 1),
    (dict(x=P + 1), 1), (dict(residual=6 * P, ld_residual=63), 1), (dict(keep_gate=6 * P, keep_up=7 * P, ld_keep=95), 1),
    (dict(keep_gate=6 * P, keep_up=7 * P, keep_dt=4), 1), (dict(keep_gate=6 * P, keep_up=6 * P), 1),
    (dict(keep_gate=6 * P, keep_up=7 * P, keep_dt=4, keep_gate_scale=8 * P, keep_up_scale=8 * P), 1),
    (dict(y=P), 1), (dict(y=4 * P), 1), (dict(keep_gate=P, keep_up=7 * P), 1), (dict(residual=5 * P + 128), 1), (dict(ws=5 * P), 1),
    (dict(ws=None), 3), (dict(ws_bytes=100), 3), (dict(ws=10 * P + 64), 3),
])
def test_gated_refusals_of_the_call(mir, kw, status):
    assert gated(mir, True, **kw) == status
    assert mir.lib.shampoo_last_error()


GGRAD = dict(dy=P, x=2 * P, w_gate=3 * P, w_up=4 * P, w_down=5 * P, kept_gate=6 * P, kept_up=7 * P, dx=11 * P, dw_gate=12 * P, dw_up=13 * P,
             dw_down=14 * P, ld_dy=64, ld_x=64, ld_gate=64, ld_up=64, ld_down=96, ld_kept=96, ld_dx=64, ld_dw_gate=64, ld_dw_up=64,
             ld_dw_down=96, T=10, d=64, f=96, dt=2, x_dt=2, w_dt=2, kept_dt=2, dw_dt=2, activation=4, ws=20 * P, ws_bytes=1 << 30)


def ggrad(mir, launch=False, **kw):
    return call(mir, "shampoo_gated_ffn_grad", "GatedGradArgsC", GGRAD, kw, launch)


@pytest.mark.parametrize("kw,status", [
    (dict(T=-1), 1), (dict(d=0), 1), (dict(f=0), 1), (dict(dt=1), 2), (dict(w_dt=1), 2), (dict(x_dt=0), 2), (dict(kept_dt=5), 2),
    (dict(dw_dt=1), 2), (dict(activation=7), 1), (dict(d=1 << 19), 2),
])
def test_gated_grad_refusals_of_both_calls(mir, kw, status):
    assert ggrad(mir, **kw)[0] == status
    assert ggrad(mir, True, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(dx=None, dw_gate=None, dw_up=None, dw_down=None), 1), (dict(dy=None), 1), (dict(x=None), 1), (dict(w_gate=None), 1),
    (dict(w_up=None), 1), (dict(w_down=None), 1), (dict(kept_gate=None), 1), (dict(kept_up=None), 1),
    (dict(ld_dy=63), 1), (dict(ld_x=63), 1), (dict(ld_gate=63), 1), (dict(ld_down=95), 1), (dict(ld_kept=95), 1), (dict(ld_dw_up=63), 1),
    (dict(x_dt=4), 1), (dict(kept_dt=4), 1), (dict(kept_dt=4, kept_gate_scale=8 * P, kept_up_scale=9 * P, kept_up=7 * P + 4), 1),
    (dict(dx=P), 1), (dict(dw_gate=13 * P), 1), (dict(dw_down=5 * P), 1), (dict(dw_up=2 * P), 1), (dict(dx=6 * P), 1),
    (dict(x_dt=4, x_scale=12 * P), 1), (dict(kept_dt=4, kept_gate_scale=8 * P, kept_up_scale=14 * P), 1),
    (dict(ws=None), 3), (dict(ws_bytes=100), 3), (dict(ws=20 * P + 8), 3),
])
def test_gated_grad_refusals_of_the_call(mir, kw, status):
    assert ggrad(mir, True, **kw) == status
    assert mir.lib.shampoo_last_error()


def test_empty_batches(mir):
    """Workspace queries of every call, and the forward calls, which have nothing to do."""
    for big in (dict(), dict(f=5000, d=3000), dict(dt=0, w_dt=0, y_dt=0, x_dt=0, kept_dt=0, keep_dt=0, dw_dt=0)):
        lay = {{"f": "N", "d": "K"}.get(k, k): v for k, v in big.items()}
        wide = dict(ld_x=5000, ld_w=5000, ld_y=5000, ld_dy=5000, ld_gate=5000, ld_up=5000, ld_down=5000, ld_keep=5000, ld_kept=5000)

        def of(given, kw):
            return {k: v for k, v in {**wide, **kw}.items() if k in given}

        assert linear(mir, M=0, **of(LINEAR, lay))[0] == mir.OK and linear(mir, True, M=0, **of(LINEAR, lay)) == mir.OK
        assert grad(mir, M=0, **of(GRAD, lay))[0] == mir.OK
        assert gated(mir, T=0, **of(GATED, big))[0] == mir.OK and gated(mir, True, T=0, **of(GATED, big)) == mir.OK
        assert ggrad(mir, T=0, **of(GGRAD, big))[0] == mir.OK


def test_python_checks_need_no_gpu(mir):
    import torch
    x, w = torch.zeros(6, 32), torch.zeros(40, 32)
    with pytest.raises(ValueError, match="device tensors"):
        mir.shampoo_linear(x, w)
    with pytest.raises(ValueError, match="device tensors"):
        mir.shampoo_gated_ffn(x, w, w, w.t().contiguous())
    for kw in (dict(activation="tanh"), dict(bias=torch.zeros(39)), dict(bias=torch.zeros(40).double()), dict(residual=torch.zeros(6, 41)),
               dict(y=torch.zeros(6, 40, dtype=torch.float16)), dict(y=torch.zeros(6, 80)[:, ::2]), dict(keep=torch.zeros(6, 39)),
               dict(keep=torch.zeros(6, 40).bfloat16()), dict(y=torch.zeros(6, 40), residual=torch.zeros(6, 40).bfloat16()),
               dict(keep=(torch.zeros(6, 64, dtype=torch.uint8), torch.zeros(6, 2, dtype=torch.uint8))),
               dict(keep=(torch.zeros(6, 40).to(torch.float8_e4m3fn), torch.zeros(6, 2, dtype=torch.uint8))),
               dict(keep=(torch.zeros(6, 64).to(torch.float8_e4m3fn), torch.zeros(6, 3, dtype=torch.uint8)))):
        with pytest.raises(ValueError):
            mir.shampoo_linear_workspace(x, w, **kw)
    with pytest.raises(TypeError):
        mir.shampoo_linear_workspace(x.double(), w)
    with pytest.raises(ValueError):
        mir.shampoo_linear_workspace(x, torch.zeros(40, 31))
    with pytest.raises(ValueError):
        mir.shampoo_linear_workspace(x, w.bfloat16())
    assert mir.shampoo_linear_workspace(x.bfloat16(), w) >= 40 * 32 * 2
    dy = torch.zeros(6, 40)
    for kw in (dict(), dict(dx=torch.zeros(6, 31)), dict(dw=torch.zeros(40, 32).half()), dict(dbias=torch.zeros(41)),
               dict(dw=w, activation="gelu"), dict(dw=w, activation="gelu", kept=torch.zeros(6, 41))):
        with pytest.raises((ValueError, mir.ShampooError)):
            mir.shampoo_linear_grad(dy, x, w, **kw)
    with pytest.raises(ValueError, match="8 bits"):
        mir.shampoo_linear_grad_workspace(dy, (torch.zeros(6, 32).to(torch.float8_e4m3fn), torch.zeros(6, 4, dtype=torch.uint8)), w, dw=w)
    with pytest.raises(ValueError, match="one type"):
        mir.shampoo_gated_ffn_workspace(x, w, w, w.t().contiguous(), keep=(torch.zeros(6, 40), torch.zeros(6, 80)[:, :40]))
    kept = (torch.zeros(6, 40), torch.zeros(6, 40))
    with pytest.raises(ValueError, match="of one type"):
        mir.shampoo_gated_ffn_grad_workspace(x.bfloat16(), x.bfloat16(), w, w, w.t().contiguous(), tuple(k.bfloat16() for k in kept),
                                             dw_gate=w, dw_up=w.bfloat16())
    with pytest.raises(ValueError):
        mir.shampoo_kept_empty(4, 4, torch.float16, "cpu")
    q, s = mir.shampoo_kept_empty(4, 33, "e4m3", "cpu")
    assert tuple(q.shape) == (4, 64) and tuple(s.shape) == (4, 2)
