"""Parity of the feed-forward layers (a product with bias, activation and
residual; the gated block; both with what the backward pass needs kept in
their type or in 8 bits) with their definitions in float64.

Tolerances count the float32 sums (K 2^-23 of the magnitudes summed), the
activations' evaluation, and half a step for each rounding to fewer bits: of
what is stored, and of h, dz, dg and du between two products."""

import pytest

import ffn_reference as ref
from helpers import log

pytestmark = pytest.mark.gpu

DTS = ["float32", "bfloat16"]


@pytest.fixture(scope="module")
def mir():
    import matrix_inverse_roots_amd as m
    return m


def normal(gen, rows, cols, size, dt, spread=0.0):
    import torch
    x = torch.randn((rows, cols), generator=gen, device="cuda") * size
    if spread:
        x *= torch.exp(spread * torch.randn((rows, 1), generator=gen, device="cuda"))
    return x.to(dt)


def gen_of(*seed):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(hash(seed) % (1 << 31))
    return g


def nans(*shape, dtype):
    import torch
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def room(mir, rows, cols, keep, dt):
    """Kept room full of NaN, or of ones' bits."""
    import torch
    if keep == "none":
        return None
    if keep == "dtype":
        return nans(rows, cols, dtype=dt)
    q, s = mir.shampoo_kept_empty(rows, cols, "e4m3", "cuda")
    q.view(torch.uint8).fill_(0x7f)
    s.view(torch.uint8).fill_(255)
    return q, s


def check_kept(kept, z, dz, dt, what):
    import torch
    if isinstance(kept, torch.Tensor):
        ref.check(kept, z, dz + ref.HALF[dt] * (z.abs() + dz), what)
        return
    q, s = kept
    rows, cols = z.shape
    wide = q.shape[1]
    assert not bool(q.float()[:, cols:].any())
    big = torch.zeros((rows, wide), dtype=torch.float64, device=z.device)
    big[:, :cols] = z.abs() + dz
    big = big.view(rows, -1, 32).amax(dim=2).repeat_interleave(32, 1)[:, :cols]
    # normal numbers: half a step of 2^-3; below 2^-6 of the scale half of 2^-9, the
    # scale at most 4 / 448 of the block's largest where a border is near
    ref.check(ref.stand(q, s, cols, 32), z, 1.001 * dz + 2.0 ** -4 * (z.abs() + dz) + 2.0 ** -10 * 4 / 448 * big + 1e-37, what)


# rows from one to many tiles, odd sizes, few outputs of a long sum (partial results), sizes below a block
SHAPES = [(1, 1, 1), (1, 1000, 300), (2, 130, 257), (3, 64, 96), (4, 2100, 40), (5, 100, 33), (33, 72, 129), (40, 4200, 136),
          (130, 256, 300), (257, 513, 700), (300, 96, 2731), (1030, 128, 520)]


@pytest.mark.parametrize("keep", ["none", "dtype", "e4m3"])
@pytest.mark.parametrize("kind", ref.ACTS)
@pytest.mark.parametrize("dt", DTS)
def test_linear(mir, dt, kind, keep):
    import torch
    dt = getattr(torch, dt)
    for k, (M, K, N) in enumerate(SHAPES):
        gen = gen_of(M, K, N)
        x, w = normal(gen, M, K, 1.0, dt, 0.5), normal(gen, N, K, 1.5 / K ** 0.5, dt)
        bias = torch.randn(N, generator=gen, device="cuda").to([torch.float32, dt][k % 2]) if k % 3 else None
        ydt = torch.float32 if k % 4 == 3 else dt
        residual = normal(gen, M, N, 1.0, ydt) if k % 2 else None
        kept = room(mir, M, N, keep, dt)
        y = mir.shampoo_linear(x, w, nans(M, N, dtype=ydt), bias=bias, activation=kind, residual=residual, keep=kept)
        z, dz, want, err = ref.linear(x, w, bias, kind, residual)
        what = f"{M} x {K} x {N}"
        ref.check(y, want, err + ref.HALF[ydt] * (want.abs() + err), what + " y")
        if kept is not None:
            check_kept(kept, z, dz, dt, what + " kept")
    log(f"linear {dt} {kind} {keep}: {len(SHAPES)} shapes")


@pytest.mark.parametrize("keep", ["dtype", "e4m3"])
@pytest.mark.parametrize("kind", ref.ACTS)
@pytest.mark.parametrize("dt", DTS)
def test_linear_grad(mir, dt, kind, keep):
    import torch
    dt = getattr(torch, dt)
    for k, (M, K, N) in enumerate(SHAPES):
        gen = gen_of(M, K, N, 1)
        x, w = normal(gen, M, K, 1.0, dt, 0.5), normal(gen, N, K, K ** -0.5, dt)
        z, dy = normal(gen, M, N, 1.5, torch.float32, 0.5), normal(gen, M, N, 1e-3, dt, 1.0)
        if keep == "e4m3":
            q, s = ref.blocks(z, 32)
            kept = q.to(torch.float8_e4m3fn), s.view(torch.float8_e8m0fnu)
            x = mir.shampoo_quantize_f8(x)
        else:
            kept = z.to(dt)
        gdt = torch.float32 if k % 3 == 0 else dt
        dx, dw, db = nans(M, K, dtype=dt), nans(N, K, dtype=gdt), nans(N, dtype=gdt)
        mir.shampoo_linear_grad(dy, x, w, kept=kept, activation=kind, dx=dx, dw=dw, dbias=db)
        want = ref.linear_grad(dy, ref.widen(x, K, 128), w, ref.widen(kept, N), kind, ref.HALF[dt] if dt != torch.float32 else 0)
        for name, got in (("dx", dx), ("dw", dw), ("dbias", db)):
            v, err = want[name]
            ref.check(got, v, err + ref.HALF[got.dtype] * (v.abs() + err) + 1e-38, f"{M} x {K} x {N} {name}")
    log(f"linear gradients {dt} {kind} {keep}: {len(SHAPES)} shapes")


GATED = [(1, 1, 1), (1, 1000, 300), (2, 130, 257), (3, 64, 96), (4, 700, 2100), (5, 100, 33), (33, 72, 129), (40, 2200, 136),
         (130, 256, 300), (257, 513, 700), (300, 96, 1371), (1030, 128, 520)]


@pytest.mark.parametrize("keep", ["none", "dtype", "e4m3"])
@pytest.mark.parametrize("kind", ref.ACTS)
@pytest.mark.parametrize("dt", DTS)
def test_gated(mir, dt, kind, keep):
    import torch
    dt = getattr(torch, dt)
    for k, (T, d, f) in enumerate(GATED):
        gen = gen_of(T, d, f)
        x = normal(gen, T, d, 1.0, dt, 0.5)
        wg, wu, wd = normal(gen, f, d, 1.5 / d ** 0.5, dt), normal(gen, f, d, d ** -0.5, dt), normal(gen, d, f, f ** -0.5, dt)
        ydt = torch.float32 if k % 4 == 3 else dt
        residual = normal(gen, T, d, 1.0, ydt) if k % 2 else None
        pair = room(mir, T, f, keep, dt), room(mir, T, f, keep, dt)
        y = mir.shampoo_gated_ffn(x, wg, wu, wd, nans(T, d, dtype=ydt), activation=kind, residual=residual,
                                  keep=None if keep == "none" else pair)
        (g, eg), (u, eu), (want, err) = ref.gated(x, wg, wu, wd, kind, residual, ref.HALF[dt])
        what = f"{T} x {d} x {f}"
        ref.check(y, want, err + ref.HALF[ydt] * (want.abs() + err), what + " y")
        if keep != "none":
            check_kept(pair[0], g, eg, dt, what + " gate")
            check_kept(pair[1], u, eu, dt, what + " up")
    log(f"gated {dt} {kind} {keep}: {len(GATED)} shapes")


@pytest.mark.parametrize("keep", ["dtype", "e4m3"])
@pytest.mark.parametrize("kind", ref.ACTS)
@pytest.mark.parametrize("dt", DTS)
def test_gated_grad(mir, dt, kind, keep):
    import torch
    dt = getattr(torch, dt)
    for k, (T, d, f) in enumerate(GATED):
        gen = gen_of(T, d, f, 1)
        x, dy = normal(gen, T, d, 1.0, dt, 0.5), normal(gen, T, d, 1e-3, dt, 1.0)
        wg, wu, wd = normal(gen, f, d, d ** -0.5, dt), normal(gen, f, d, d ** -0.5, dt), normal(gen, d, f, f ** -0.5, dt)
        kept = normal(gen, T, f, 1.5, torch.float32, 0.5), normal(gen, T, f, 1.0, torch.float32, 0.5)
        if keep == "e4m3":
            kept = tuple((q.to(torch.float8_e4m3fn), s.view(torch.float8_e8m0fnu)) for q, s in (ref.blocks(t, 32) for t in kept))
            x = mir.shampoo_quantize_f8(x)
        else:
            kept = tuple(t.to(dt) for t in kept)
        gdt = torch.float32 if k % 3 == 0 else dt
        out = dict(dx=nans(T, d, dtype=dt), dw_gate=nans(f, d, dtype=gdt), dw_up=nans(f, d, dtype=gdt), dw_down=nans(d, f, dtype=gdt))
        mir.shampoo_gated_ffn_grad(dy, x, wg, wu, wd, kept, activation=kind, **out)
        want = ref.gated_grad(dy, ref.widen(x, d, 128), wg, wu, wd, ref.widen(kept[0], f), ref.widen(kept[1], f), kind,
                              ref.HALF[dt])
        for name, got in out.items():
            v, err = want[name]
            ref.check(got, v, err + ref.HALF[got.dtype] * (v.abs() + err) + 1e-38, f"{T} x {d} x {f} {name}")
    log(f"gated gradients {dt} {kind} {keep}: {len(GATED)} shapes")
