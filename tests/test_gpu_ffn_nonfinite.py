"""The feed-forward layers' gradients at kept values that are not finite: the
formulas' own results.  relu' is 1 where z > 0 and 0 elsewhere, NaN among it;
the smooth activations' derivatives are NaN at NaN and at both infinities
(z act'' is infinity times zero there); 8 bits hold an infinity as NaN."""

import pytest

import ffn_reference as ref
from test_gpu_ffn import gen_of, nans, normal

pytestmark = pytest.mark.gpu

ODD = [float("nan"), float("inf"), float("-inf")]


@pytest.fixture(scope="module")
def mir():
    import matrix_inverse_roots_amd as m
    return m


def kept_of(z, keep, dt):
    import torch
    if keep == "dtype":
        return z.to(dt)
    q, s = ref.blocks(z, 32)
    return q.to(torch.float8_e4m3fn), s.view(torch.float8_e8m0fnu)


def with_odd(gen, rows, cols):
    """Values with a NaN, an infinity and a minus infinity in rows and columns of their own."""
    import torch
    z = normal(gen, rows, cols, 1.5, torch.float32)
    for i, v in enumerate(ODD):
        z[i * (rows - 1) // 2, 5 + 17 * i] = v
    return z


@pytest.mark.parametrize("keep", ["dtype", "e4m3"])
@pytest.mark.parametrize("kind", ref.ACTS[1:])
@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
@pytest.mark.parametrize("M", [3, 150])
def test_layer(mir, M, dt, kind, keep):
    import torch
    dt = getattr(torch, dt)
    K, N = 40, 75
    gen = gen_of(M, 31)
    x, w, dy = normal(gen, M, K, 1.0, dt), normal(gen, N, K, 0.2, dt), normal(gen, M, N, 1.0, dt)
    kept = kept_of(with_odd(gen, M, N), keep, dt)
    out = dict(dx=nans(M, K, dtype=dt), dw=nans(N, K, dtype=torch.float32), dbias=nans(N, dtype=torch.float32))
    mir.shampoo_linear_grad(dy, x, w, kept=kept, activation=kind, **out)
    want = ref.linear_grad(dy, x, w, ref.widen(kept, N), kind, ref.HALF[dt] if dt != torch.float32 else 0)
    for name, got in out.items():
        v, err = want[name]
        ref.check(got, v, err + ref.HALF[got.dtype] * (v.abs() + err) + 1e-38, name)
    # a column of dz that is NaN in one row
    assert int(torch.isnan(out["dbias"]).sum()) == (0 if kind == "relu" else 3)


@pytest.mark.parametrize("keep", ["dtype", "e4m3"])
@pytest.mark.parametrize("kind", ref.ACTS[1:])
@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
@pytest.mark.parametrize("T", [3, 150])
def test_block(mir, T, dt, kind, keep):
    """The gate's values, then the up projection's."""
    import torch
    dt = getattr(torch, dt)
    d, f = 40, 75
    gen = gen_of(T, 32)
    x, dy = normal(gen, T, d, 1.0, dt), normal(gen, T, d, 1.0, dt)
    wg, wu, wd = normal(gen, f, d, 0.2, dt), normal(gen, f, d, 0.2, dt), normal(gen, d, f, 0.2, dt)
    for which in (0, 1):
        z = [normal(gen, T, f, 1.0, torch.float32) for _ in range(2)]
        z[which] = with_odd(gen, T, f)
        kept = tuple(kept_of(v, keep, dt) for v in z)
        out = dict(dx=nans(T, d, dtype=dt), dw_gate=nans(f, d, dtype=dt), dw_up=nans(f, d, dtype=dt), dw_down=nans(d, f, dtype=dt))
        mir.shampoo_gated_ffn_grad(dy, x, wg, wu, wd, kept, activation=kind, **out)
        want = ref.gated_grad(dy, x, wg, wu, wd, ref.widen(kept[0], f), ref.widen(kept[1], f), kind, ref.HALF[dt])
        for name, got in out.items():
            v, err = want[name]
            ref.check(got, v, err + ref.HALF[dt] * (v.abs() + err) + 1e-38, f"{which} {name}")


@pytest.mark.parametrize("kind", ref.ACTS[1:])
def test_large_finite_values(mir, kind):
    """Derivatives of finite values reach their limits, 1 and 0, whatever their size."""
    import torch
    z = torch.tensor([[s * v for v in (9e3, 1.1e4, 1e8, 1e13, 1.9e19, 1e32, 3.4e38) for s in (1.0, -1.0)]], device="cuda").repeat(3, 1)
    n = z.shape[1]
    dx, eye = nans(3, n, dtype=torch.float32), torch.eye(n, device="cuda")
    mir.shampoo_linear_grad(torch.ones_like(z), None, eye, kept=z, activation=kind, dx=dx)
    assert torch.equal(dx, (z > 0).float())
