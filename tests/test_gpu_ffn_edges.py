"""The feed-forward layers where they could go wrong: strides and alignments,
float32 weights, accumulated gradients, values that are not finite, 8-bit codes
bit by bit, graphs, streams, sizes past 32 bits; gradients against differences;
and the operators together, as a network uses them."""

import pytest

import ffn_reference as ref
from helpers import log
from test_gpu_ffn import check_kept, gen_of, nans, normal, room

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mir():
    import matrix_inverse_roots_amd as m
    return m


def view(t, off, pad):
    """t's values in rows `pad` elements longer, starting `off` elements into them; (view, whole)."""
    import torch
    whole = torch.full((t.shape[0], t.shape[1] + pad), 7.0, dtype=t.dtype, device=t.device)
    whole[:, off:off + t.shape[1]] = t
    return whole[:, off:off + t.shape[1]], whole


def untouched(whole, off, cols):
    rest = whole.clone()
    rest[:, off:off + cols] = 7.0
    return bool((rest == 7.0).all())


ODD = [(0, 8), (0, 1), (1, 3), (3, 13), (8, 16)]


@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
@pytest.mark.parametrize("M,K,N", [(3, 72, 88), (3, 71, 87), (70, 72, 88), (70, 71, 87), (40, 2112, 64)])
def test_strides_change_no_bit(mir, M, K, N, dt):
    """Views of wider rows at every alignment give the bits of contiguous tensors, and what lies around outputs stays."""
    import torch
    dt = getattr(torch, dt)
    gen = gen_of(M, K, N, 2)
    x, w, r, z = normal(gen, M, K, 1.0, dt), normal(gen, N, K, 0.1, dt), normal(gen, M, N, 1.0, dt), normal(gen, M, N, 1.0, dt)
    bias = torch.randn(N, generator=gen, device="cuda")
    keep = torch.empty_like(z)
    y = mir.shampoo_linear(x, w, bias=bias, activation="gelu", residual=r, keep=keep)
    dx, dw, db = torch.empty_like(x), torch.empty_like(w), torch.empty_like(bias)
    mir.shampoo_linear_grad(r, x, w, kept=z, activation="silu", dx=dx, dw=dw, dbias=db)
    for off, pad in ODD:
        (xv, _), (wv, _), (rv, _), (zv, _) = (view(t, off, pad) for t in (x, w, r, z))
        (yv, yw), (kv, kw), (dxv, dxw), (dwv, dww) = (view(torch.zeros_like(t), off, pad) for t in (y, keep, dx, dw))
        dbv = torch.empty(N + 4, device="cuda")[off % 4:off % 4 + N]
        mir.shampoo_linear(xv, wv, yv, bias=bias, activation="gelu", residual=rv, keep=kv)
        mir.shampoo_linear_grad(rv, xv, wv, kept=zv, activation="silu", dx=dxv, dw=dwv, dbias=dbv)
        for got, want, whole in ((yv, y, yw), (kv, keep, kw), (dxv, dx, dxw), (dwv, dw, dww)):
            assert torch.equal(got, want), (off, pad)
            assert untouched(whole, off, want.shape[1])
        assert torch.equal(dbv, db)


@pytest.mark.parametrize("T,d,f", [(70, 72, 88), (70, 71, 87), (9, 130, 45)])
def test_gated_strides_change_no_bit(mir, T, d, f):
    import torch
    dt = torch.bfloat16
    gen = gen_of(T, d, f, 3)
    x, wg, wu, wd, dy = (normal(gen, a, b, 0.3, dt) for a, b in ((T, d), (f, d), (f, d), (d, f), (T, d)))
    g, u = torch.empty((T, f), dtype=dt, device="cuda"), torch.empty((T, f), dtype=dt, device="cuda")
    y = mir.shampoo_gated_ffn(x, wg, wu, wd, keep=(g, u), residual=dy)
    out = [torch.empty_like(t) for t in (x, wg, wu, wd)]
    mir.shampoo_gated_ffn_grad(dy, x, wg, wu, wd, (g, u), *out)
    for off, pad in ODD:
        xv, wgv, wdv, dyv = (view(t, off, pad)[0] for t in (x, wg, wd, dy))
        wuv = view(wu, 0, 24)[0]                      # the two projections at different strides
        (yv, yw), (gv, gw), (uv, uw) = (view(torch.zeros_like(t), off, pad) for t in (y, g, u))
        mir.shampoo_gated_ffn(xv, wgv, wuv, wdv, yv, keep=(gv, uv), residual=dyv)
        outs = [view(torch.zeros_like(t), off, p) for t, p in zip(out, (pad, pad, pad + 5, pad))]
        mir.shampoo_gated_ffn_grad(dyv, xv, wgv, wuv, wdv, (gv, uv), *[o[0] for o in outs])
        for got, want, whole in ((yv, y, yw), (gv, g, gw), (uv, u, uw)) + tuple((o[0], t, o[1]) for o, t in zip(outs, out)):
            assert torch.equal(got, want), (off, pad)
            assert untouched(whole, off, want.shape[1])


@pytest.mark.parametrize("M", [2, 50])
def test_float32_weights_beside_bfloat16(mir, M):
    """The bits of weights rounded beforehand, forward and backward."""
    import torch
    for K, N in ((64, 96), (33, 57), (1000, 40)):
        gen = gen_of(M, K, N, 4)
        x, dy = normal(gen, M, K, 1.0, torch.bfloat16), normal(gen, M, N, 1.0, torch.bfloat16)
        w = normal(gen, N, K, 0.1, torch.float32)
        up, down = normal(gen, N, K, 0.1, torch.float32), normal(gen, K, N, 0.1, torch.float32)
        kept = dy.clone(), dy.flip(0).contiguous()
        got = []
        for turn in (lambda t: t, lambda t: t.bfloat16()):
            y = mir.shampoo_linear(x, turn(w), activation="gelu")
            dx = torch.empty_like(x)
            mir.shampoo_linear_grad(dy, x, turn(w), kept=dy, activation="relu", dx=dx)
            z = mir.shampoo_gated_ffn(x, turn(w), turn(up), turn(down))
            dx2 = torch.empty_like(x)
            mir.shampoo_gated_ffn_grad(x, x, turn(w), turn(up), turn(down), kept, dx=dx2)
            got.append((y, dx, z, dx2))
        assert all(torch.equal(a, b) for a, b in zip(*got))


@pytest.mark.parametrize("gdt", ["float32", "bfloat16"])
@pytest.mark.parametrize("T,d,f", [(64, 96, 80), (700, 40, 72), (33, 2050, 35)])
def test_accumulated_gradients(mir, T, d, f, gdt):
    """accumulate adds: old + gradient, rounded once (ranges of k and whole sums)."""
    import torch
    dt, gdt = torch.bfloat16, getattr(torch, gdt)
    gen = gen_of(T, d, f, 5)
    x, dy, w = normal(gen, T, d, 1.0, dt), normal(gen, T, f, 1.0, dt), normal(gen, f, d, 0.1, dt)
    old, oldb = normal(gen, f, d, 3.0, gdt), torch.randn(f, generator=gen, device="cuda").to(gdt)
    dw, db = old.clone(), oldb.clone()
    mir.shampoo_linear_grad(dy, x, w, kept=dy, activation="gelu", dw=dw, dbias=db, accumulate=True)
    want = ref.linear_grad(dy, x, w, dy.double(), "gelu", ref.HALF[dt])
    for name, got, before in (("dw", dw, old), ("dbias", db, oldb)):
        v, err = want[name]
        v = v + before.double()
        ref.check(got, v, err + 2 * ref.U * (v.abs() + before.double().abs()) + ref.HALF[gdt] * (v.abs() + err), name)
    h = normal(gen, T, f, 1.0, dt)
    g = dict(dw_gate=normal(gen, f, d, 3.0, gdt), dw_up=normal(gen, f, d, 3.0, gdt), dw_down=normal(gen, d, f, 3.0, gdt))
    out = {k: v.clone() for k, v in g.items()}
    wd = normal(gen, d, f, 0.1, dt)
    mir.shampoo_gated_ffn_grad(x, x, w, w, wd, (h, dy), accumulate=True, **out)
    want = ref.gated_grad(x, x, w, w, wd, h.double(), dy.double(), "silu", ref.HALF[dt])
    for name, got in out.items():
        v, err = want[name]
        v = v + g[name].double()
        ref.check(got, v, err + 2 * ref.U * (v.abs() + g[name].double().abs()) + ref.HALF[gdt] * (v.abs() + err), name)


# (rows, inner, columns): every tile in whole and ragged sizes.  bfloat16: 256 x 128
# from 257 tiles of 128 x 128 on, 256 x 256 where they fill the chip and the inner size is long or
# the epilogue a plain store; 128 x 128 two to a unit for few rows of very many columns.
# float32: 64 x 64, 128 x 128, 256 x 256.
TILES = [(2100, 40, 2100), (4090, 72, 4000), (4000, 4200, 4090), (100, 64, 70000), (2048, 136, 2048), (600, 1000, 900)]


@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
@pytest.mark.parametrize("M,K,N", TILES)
def test_every_tile(mir, M, K, N, dt):
    """Forward and backward of a layer at the sizes of each tile: all in the
    epilogue, then nothing in it."""
    import torch
    dt = getattr(torch, dt)
    half = ref.HALF[dt]
    gen = gen_of(M, K, N, 20)
    x, w, r = normal(gen, M, K, 1.0, dt, 0.3), normal(gen, N, K, K ** -0.5, dt), normal(gen, M, N, 1.0, dt)
    bias = torch.randn(N, generator=gen, device="cuda")
    kept = mir.shampoo_kept_empty(M, N, "e4m3", "cuda")
    y = mir.shampoo_linear(x, w, bias=bias, activation="gelu", residual=r, keep=kept)
    z, dz, want, err = ref.linear(x, w, bias, "gelu", r)
    ref.check(y, want, err + half * (want.abs() + err), "y")
    check_kept(kept, z, dz, dt, "kept")
    del z, dz, want, err
    y = mir.shampoo_linear(x, w)
    _, _, want, err = ref.linear(x, w, None, "none", None)
    ref.check(y, want, err + half * (want.abs() + err), "plain y")
    del y, want, err
    out = dict(dx=nans(M, K, dtype=dt), dw=nans(N, K, dtype=torch.float32), dbias=nans(N, dtype=torch.float32))
    mir.shampoo_linear_grad(r, x, w, kept=kept, activation="gelu", **out)
    want = ref.linear_grad(r, x, w, ref.widen(kept, N), "gelu", half if dt != torch.float32 else 0)
    for name, got in out.items():
        v, e = want[name]
        ref.check(got, v, e + ref.HALF[got.dtype] * (v.abs() + e), name)


@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
@pytest.mark.parametrize("keep", ["dtype", "e4m3"])
@pytest.mark.parametrize("T,d,f", [(2100, 40, 2100), (4090, 72, 4000), (4000, 4200, 2100), (100, 64, 35000), (1030, 2056, 1100)])
def test_every_tile_of_the_gated_block(mir, T, d, f, keep, dt):
    import torch
    dt = getattr(torch, dt)
    half = ref.HALF[dt]
    gen = gen_of(T, d, f, 21)
    x, dy = normal(gen, T, d, 1.0, dt, 0.3), normal(gen, T, d, 1.0, dt)
    wg, wu, wd = normal(gen, f, d, d ** -0.5, dt), normal(gen, f, d, d ** -0.5, dt), normal(gen, d, f, f ** -0.5, dt)
    pair = [room(mir, T, f, keep, dt) for _ in range(2)]
    y = mir.shampoo_gated_ffn(x, wg, wu, wd, residual=dy, keep=pair)
    (g, eg), (u, eu), (want, err) = ref.gated(x, wg, wu, wd, "silu", dy, half)
    ref.check(y, want, err + half * (want.abs() + err), "y")
    check_kept(pair[0], g, eg, dt, "gate")
    check_kept(pair[1], u, eu, dt, "up")
    del g, eg, u, eu, want, err
    both = nans(2, f, d, dtype=dt)      # the up projection's gradient below the gate's in memory
    out = dict(dx=nans(T, d, dtype=dt), dw_gate=both[1], dw_up=both[0], dw_down=nans(d, f, dtype=dt))
    mir.shampoo_gated_ffn_grad(dy, x, wg, wu, wd, pair, **out)
    want = ref.gated_grad(dy, x, wg, wu, wd, ref.widen(pair[0], f), ref.widen(pair[1], f), "silu", half)
    for name, got in out.items():
        v, e = want[name]
        ref.check(got, v, e + half * (v.abs() + e), name)


def test_each_gradient_alone_is_the_same(mir):
    import torch
    dt = torch.bfloat16
    gen = gen_of(6)
    T, d, f = 300, 136, 200
    x, dy, w = normal(gen, T, d, 1.0, dt), normal(gen, T, f, 1.0, dt), normal(gen, f, d, 0.1, dt)
    out = dict(dx=torch.empty_like(x), dw=torch.empty_like(w), dbias=torch.empty(f, device="cuda"))
    mir.shampoo_linear_grad(dy, x, w, kept=dy, activation="gelu", **out)
    for name, t in out.items():
        one = torch.empty_like(t)
        mir.shampoo_linear_grad(dy, x if name == "dw" else None, w, kept=dy, activation="gelu", **{name: one})
        assert torch.equal(one, t), name
    wd = normal(gen, d, f, 0.1, dt)
    out = dict(dx=torch.empty_like(x), dw_gate=torch.empty_like(w), dw_up=torch.empty_like(w), dw_down=torch.empty_like(wd))
    mir.shampoo_gated_ffn_grad(x, x, w, w, wd, (dy, dy), **out)
    for name, t in out.items():
        one = torch.empty_like(t)
        mir.shampoo_gated_ffn_grad(x, x, w if name == "dx" else None, w if name == "dx" else None, wd, (dy, dy), **{name: one})
        assert torch.equal(one, t), name


@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
def test_8_bit_codes_are_the_definition(mir, dt):
    """What is kept in 8 bits is the float32 sum's own code, bit for bit: with
    a float32 result and no activation both leave the same call; partial
    results, single rows, zero rows, wide and tiny scales."""
    import torch
    dt = getattr(torch, dt)
    for M, K, N in [(1, 40, 33), (4, 8, 100), (70, 130, 257), (300, 64, 520), (40, 4200, 136), (1100, 96, 1100)]:
        gen = gen_of(M, K, N, 7)
        x, w = normal(gen, M, K, 1.0, dt, 3.0), normal(gen, N, K, 1.0, dt)
        if M > 2:
            x[1] = 0
            x[2] *= 1e-36 if dt == torch.bfloat16 else 1e-37
        bias = None if M > 2 else torch.randn(N, generator=gen, device="cuda")
        q, s = mir.shampoo_kept_empty(M, N, "e4m3", "cuda")
        y = mir.shampoo_linear(x, w, torch.empty((M, N), device="cuda"), bias=bias, keep=(q, s))
        want, scale = ref.blocks(y, 32)
        assert torch.equal(s.view(torch.uint8), scale), (M, K, N)
        assert torch.equal(q.float(), want), (M, K, N)
        # the gated block's are those of what it keeps in float32
        if M > 4:
            wu, wd = normal(gen, N, K, 1.0, dt), normal(gen, K, N, 1.0, dt)
            pair = [mir.shampoo_kept_empty(M, N, "e4m3", "cuda") for _ in range(2)]
            mir.shampoo_gated_ffn(x, w, wu, wd, keep=pair)
            for (q, s), t in zip(pair, (w, wu)):
                z, dz, _, _ = ref.linear(x, t, None, "none", None)
                check_kept((q, s), z, dz, dt, f"{M} x {K} x {N}")
            if dt == torch.float32:
                wide = nans(M, N, dtype=dt), nans(M, N, dtype=dt)
                mir.shampoo_gated_ffn(x, w, wu, wd, keep=wide)
                for (q, s), t in zip(pair, wide):
                    want, scale = ref.blocks(t, 32)
                    assert torch.equal(s.view(torch.uint8), scale) and torch.equal(q.float(), want), (M, K, N)


def test_x_in_8_bits_is_widened_exactly(mir):
    """Gradients from x in 8 bits are those from the values that it stands for, bit for bit."""
    import torch
    for dt in (torch.bfloat16, torch.float32):
        for T, d, f in [(1, 1, 1), (70, 130, 96), (300, 256, 40), (65, 1000, 72)]:
            gen = gen_of(T, d, f, 8)
            x, dy, w, wd = normal(gen, T, d, 1.0, dt, 2.0), normal(gen, T, f, 1.0, dt), normal(gen, f, d, 0.1, dt), normal(gen, d, f, 0.1, dt)
            x8 = mir.shampoo_quantize_f8(x)
            wide = ref.stand(*x8, d, 128).to(dt)
            got = []
            for given in (x8, wide):
                dw, a, b = (torch.empty_like(w) for _ in range(3))
                mir.shampoo_linear_grad(dy, given, w, dw=dw)
                mir.shampoo_gated_ffn_grad(x, given, w, w, wd, (dy, dy), dw_gate=a, dw_up=b)
                got.append((dw, a, b))
            assert all(torch.equal(p, q) for p, q in zip(*got))


@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
@pytest.mark.parametrize("M", [3, 90])
def test_values_that_are_not_finite(mir, M, dt):
    """A row of x with a NaN or an infinity leaves the other rows' results as
    they are; its own are NaN (an infinity times both signs), its codes too, and its
    scale is that of the finite values."""
    import torch
    dt = getattr(torch, dt)
    gen = gen_of(M, 9)
    K, N = 40, 75
    x, w, wd = normal(gen, M, K, 1.0, dt), normal(gen, N, K, 1.0, dt), normal(gen, K, N, 0.1, dt)
    w[:, 5] = w[:, 5].abs() + 0.1
    w[::2, 5] *= -1
    bad = x.clone()
    bad[1, 7], bad[M - 1, 5] = float("nan"), float("inf")
    rows = [i for i in range(M) if i not in (1, M - 1)]
    for kind in ref.ACTS:
        y, yb = (mir.shampoo_linear(t, w, activation=kind) for t in (x, bad))
        z, zb = (mir.shampoo_gated_ffn(t, w, w, wd, activation=kind) for t in (x, bad))
        assert torch.equal(y[rows], yb[rows]) and torch.equal(z[rows], zb[rows])
        assert bool(torch.isnan(yb[1]).all()) and bool(torch.isnan(zb[1]).all())
        want = ref.act(bad[M - 1:].double() @ w.double().t(), kind)[0][0]
        if kind in ("none", "relu"):
            want = torch.where(w[:, 5] > 0, torch.full_like(want, float("inf")),
                               torch.full_like(want, float("-inf") if kind == "none" else 0.0))
            assert torch.equal(yb[M - 1].double(), want)
        else:
            assert bool((yb[M - 1][w[:, 5] > 0] == float("inf")).all()) and bool(torch.isnan(yb[M - 1][w[:, 5] < 0]).all())
    q, s = mir.shampoo_kept_empty(M, N, "e4m3", "cuda")
    mir.shampoo_linear(bad, w, keep=(q, s))
    assert bool(torch.isnan(q.float()[[1, M - 1], :N]).all()) and bool(torch.isfinite(q.float()[rows]).all())
    assert bool((s.view(torch.uint8)[[1, M - 1]] == 127).all())
    # extreme pre-activations: the limits of act and act', nothing else
    z = torch.tensor([[1e4, -1e4, 3e38, -3e38, 200.0, -200.0, 0.0, -0.0]], device="cuda").repeat(M, 1)
    dy, w8 = torch.ones((M, 8), device="cuda"), torch.eye(8, device="cuda")
    for kind in ref.ACTS[1:]:
        dx = torch.empty((M, 8), device="cuda")
        mir.shampoo_linear_grad(dy, None, w8, kept=z, activation=kind, dx=dx)
        half = 0.0 if kind == "relu" else 0.5
        assert dx[0].tolist() == [1.0, 0.0, 1.0, 0.0, 1.0, 0.0, half, half], kind
        y = mir.shampoo_linear(z, w8, activation=kind)
        assert y[0].tolist() == [z[0, 0].item(), 0.0, z[0, 2].item(), 0.0, 200.0, 0.0, 0.0, 0.0], kind


def test_empty_batches(mir):
    import torch
    x, w, wd = torch.empty((0, 24), device="cuda"), torch.ones((40, 24), device="cuda"), torch.ones((24, 40), device="cuda")
    dy = torch.empty((0, 40), device="cuda")
    assert mir.shampoo_linear(x, w, activation="gelu").shape == (0, 40)
    assert mir.shampoo_gated_ffn(x, w, w, wd).shape == (0, 24)
    for accumulate in (False, True):
        g = [torch.full(s, 3.0, device="cuda") for s in ((40, 24), (40,), (40, 24), (40, 24), (24, 40))]
        mir.shampoo_linear_grad(dy, x, w, kept=dy, activation="gelu", dx=torch.empty_like(x), dw=g[0], dbias=g[1], accumulate=accumulate)
        mir.shampoo_gated_ffn_grad(x, x, w, w, wd, (dy, dy), torch.empty_like(x), g[2], g[3], g[4], accumulate=accumulate)
        assert all(bool((t == (3.0 if accumulate else 0.0)).all()) for t in g)


@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
@pytest.mark.parametrize("M,N", [(3, 50), (40, 96), (140, 33), (300, 256)])
def test_residual_in_place(mir, M, N, dt):
    import torch
    dt = getattr(torch, dt)
    gen = gen_of(M, N, 10)
    for K in (48, 4096):
        x, w, r = normal(gen, M, K, 1.0, dt), normal(gen, N, K, 0.1, dt), normal(gen, M, N, 1.0, dt)
        want = mir.shampoo_linear(x, w, activation="relu", residual=r)
        y = r.clone()
        mir.shampoo_linear(x, w, y, activation="relu", residual=y)
        assert torch.equal(y, want)
    wg, wd = normal(gen, 64, N, 0.1, dt), normal(gen, N, 64, 0.1, dt)
    want = mir.shampoo_gated_ffn(r, wg, wg, wd, residual=r)
    y = r.clone()
    mir.shampoo_gated_ffn(r, wg, wg, wd, y, residual=y)
    assert torch.equal(y, want)


def passes(mir, s):
    """Forward and backward of both layers on tensors `s`; what they leave."""
    import torch
    k = s["keep"]
    y = mir.shampoo_linear(s["x"], s["w"], s["y"], bias=s["b"], activation="gelu", keep=k[0])
    h = mir.shampoo_gated_ffn(y, s["wg"], s["wu"], s["wd"], s["h"], residual=y, keep=(k[1], k[2]))
    mir.shampoo_gated_ffn_grad(s["dy"], y, s["wg"], s["wu"], s["wd"], (k[1], k[2]), s["dh"], s["dwg"], s["dwu"], s["dwd"])
    mir.shampoo_linear_grad(s["dh"], s["x"], s["w"], kept=k[0], activation="gelu", dx=s["dx"], dw=s["dw"], dbias=s["db"])
    return [y, h] + [s[n] for n in ("dh", "dwg", "dwu", "dwd", "dx", "dw", "db")] + [t.view(torch.uint8) for pair in k for t in pair]


def tensors(mir, seed, T=180, d=104, f=200):
    import torch
    dt = torch.bfloat16
    gen = gen_of(seed, 11)
    s = dict(x=normal(gen, T, d, 1.0, dt), w=normal(gen, d, d, 0.1, dt), b=torch.randn(d, generator=gen, device="cuda"),
             wg=normal(gen, f, d, 0.1, dt), wu=normal(gen, f, d, 0.1, dt), wd=normal(gen, d, f, 0.1, dt), dy=normal(gen, T, d, 1.0, dt))
    s["keep"] = [mir.shampoo_kept_empty(T, n, "e4m3", "cuda") for n in (d, f, f)]
    for n, like in (("y", "x"), ("h", "x"), ("dh", "x"), ("dx", "x"), ("dw", "w"), ("dwg", "wg"), ("dwu", "wu"), ("dwd", "wd")):
        s[n] = torch.empty_like(s[like])
    s["db"] = torch.empty(d, device="cuda")
    return s


@pytest.mark.parametrize("T", [3, 40, 180])
def test_captured_passes(mir, T):
    """A captured forward and backward pass, replayed on new inputs with eager
    work and allocations between, gives the eager bits every time; two graphs
    in turn."""
    import torch
    a, b, e = (tensors(mir, k, T) for k in (1, 2, 3))
    passes(mir, e)
    torch.cuda.synchronize()
    graphs = []
    for s in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = passes(mir, s)
        graphs.append((g, s, out))
    for k in range(4):
        for g, s, out in graphs:
            new = tensors(mir, 10 + k, T)
            for n in ("x", "w", "b", "wg", "wu", "wd", "dy"):
                s[n].copy_(new[n])
            junk = [torch.full((1 << 16,), float("nan"), device="cuda") for _ in range(4)]
            g.replay()
            torch.cuda.synchronize()
            del junk
            want = passes(mir, new)
            torch.cuda.synchronize()
            assert all(torch.equal(p, q) for p, q in zip(out, want)), k


def test_two_streams_at_once(mir):
    """Calls in flight on two streams, each allocating for itself, give the
    bits of one after the other, and of the same call again."""
    import torch
    want = []
    for k in range(2):
        want.append([t.clone() for t in passes(mir, tensors(mir, k, 1500, 264, 520))])
        torch.cuda.synchronize()
    for _ in range(3):
        both = [tensors(mir, k, 1500, 264, 520) for k in range(2)]
        streams = [torch.cuda.Stream() for _ in both]
        torch.cuda.synchronize()
        got = []
        for s, st in zip(both, streams):
            with torch.cuda.stream(st):
                got.append(passes(mir, s))
        junk = [torch.full((1 << 20,), float("nan"), device="cuda") for _ in range(4)]
        torch.cuda.synchronize()
        del junk
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_stream_argument(mir):
    import torch
    s, t = tensors(mir, 4), tensors(mir, 4)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    y = mir.shampoo_linear(s["x"], s["w"], activation="gelu", keep=s["keep"][0], stream=st)
    dx = torch.empty_like(s["x"])
    torch.cuda.synchronize()
    mir.shampoo_linear_grad(s["dy"], s["x"], s["w"], kept=s["keep"][0], activation="gelu", dx=dx, stream=st)
    h = mir.shampoo_gated_ffn(s["x"], s["wg"], s["wu"], s["wd"], stream=st)
    torch.cuda.synchronize()
    y2 = mir.shampoo_linear(t["x"], t["w"], activation="gelu", keep=t["keep"][0])
    dx2 = torch.empty_like(dx)
    mir.shampoo_linear_grad(t["dy"], t["x"], t["w"], kept=t["keep"][0], activation="gelu", dx=dx2)
    assert torch.equal(y, y2) and torch.equal(dx, dx2) and torch.equal(h, mir.shampoo_gated_ffn(t["x"], t["wg"], t["wu"], t["wd"]))


def test_workspace_of_the_caller(mir):
    """A given workspace, full of NaN, serves; a short one is refused."""
    import torch
    for T in (2, 70):
        s, t = tensors(mir, 5, T), tensors(mir, 5, T)
        x, r = s["x"][:, 1:], t["x"][:, 1:]
        w = s["w"][:, 1:]
        need = mir.shampoo_linear_workspace(x, w)
        y = mir.shampoo_linear(x, w)
        if need:
            ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
            assert torch.equal(mir.shampoo_linear(r, w, ws=ws), y)
            with pytest.raises(mir.ShampooError):
                mir.shampoo_linear(r, w, ws=ws[:need // 2])
        args = (s["wg"], s["wu"], s["wd"])
        need = mir.shampoo_gated_ffn_workspace(s["x"], *args)
        ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        assert torch.equal(mir.shampoo_gated_ffn(s["x"], *args, ws=ws), mir.shampoo_gated_ffn(s["x"], *args))
        with pytest.raises(mir.ShampooError):
            mir.shampoo_gated_ffn(s["x"], *args, ws=ws[:need - 256])


def test_sizes_past_32_bits(mir):
    """Rows whose elements lie more than 2^31 from the first: outputs, kept codes, the backward's operands; sampled rows."""
    import torch
    dt = torch.bfloat16
    gen = gen_of(12)
    M, K, N = 66000, 16, 33024
    x, w = normal(gen, M, K, 1.0, dt), normal(gen, N, K, 0.3, dt)
    kept = mir.shampoo_kept_empty(M, N, "e4m3", "cuda")
    y = mir.shampoo_linear(x, w, activation="silu", keep=kept)
    rows = torch.tensor([0, 1, 31000, 65023, 65024, 65100, M - 2, M - 1], device="cuda")
    some = mir.shampoo_kept_empty(8, N, "e4m3", "cuda")
    want = mir.shampoo_linear(x[rows], w, activation="silu", keep=some)
    assert torch.equal(y[rows], want)
    assert torch.equal(kept[0].view(torch.uint8)[rows], some[0].view(torch.uint8))
    assert torch.equal(kept[1].view(torch.uint8)[rows], some[1].view(torch.uint8))
    dx, db = torch.empty_like(x), torch.empty(N, device="cuda")
    mir.shampoo_linear_grad(y, x, w, kept=kept, activation="silu", dx=dx, dbias=db)
    z, v = ref.widen(some, N), y[rows]
    want, err = ref.linear_grad(v, x[rows], w, z, "silu", ref.HALF[dt])["dx"]
    ref.check(dx[rows], want, err + ref.HALF[dt] * (want.abs() + err), "dx")
    assert bool(torch.isfinite(db).all())
    del y, dx
    wd = normal(gen, K, N, 0.05, dt)
    out = mir.shampoo_gated_ffn(x, w, w, wd, keep=(kept, mir.shampoo_kept_empty(M, N, "e4m3", "cuda")))
    assert torch.equal(out[rows], mir.shampoo_gated_ffn(x[rows], w, w, wd))
    dx = torch.empty_like(x)
    mir.shampoo_gated_ffn_grad(x, x, w, w, wd, (kept, kept), dx=dx)
    z = ref.widen((kept[0][rows], kept[1][rows]), N)
    want, err = ref.gated_grad(x[rows], x[rows], w, w, wd, z, z, "silu", ref.HALF[dt])["dx"]
    ref.check(dx[rows], want, err + ref.HALF[dt] * (want.abs() + err), "gated dx")
    torch.cuda.empty_cache()


@pytest.mark.parametrize("kind", ref.ACTS)
def test_gradients_against_differences(mir, kind):
    """<gradient, v> against central differences of the layers' definition in
    float64 along random directions v."""
    import torch
    gen = gen_of(13)
    T, d, f = 21, 24, 40
    x, wg, wu, wd, r = (normal(gen, a, b, s, torch.float32) for a, b, s in ((T, d, 1.0), (f, d, 0.3), (f, d, 0.3), (d, f, 0.2), (T, d, 1.0)))
    bias, step = torch.randn(f, generator=gen, device="cuda"), 1e-5
    c, cf = normal(gen, T, d, 1.0, torch.float32), normal(gen, T, f, 1.0, torch.float32)

    def layer(x, w, b):
        return (ref.act(x @ w.t() + b, kind)[0] * cf.double()).sum()

    def block(x, wg, wu, wd):
        return (((ref.act(x @ wg.t(), kind)[0] * (x @ wu.t())) @ wd.t()) * c.double()).sum()

    z, g, u = torch.empty((T, f), device="cuda"), torch.empty((T, f), device="cuda"), torch.empty((T, f), device="cuda")
    mir.shampoo_linear(x, wg, bias=bias, activation=kind, keep=z)
    mir.shampoo_gated_ffn(x, wg, wu, wd, activation=kind, residual=r, keep=(g, u))
    one = [torch.empty_like(t) for t in (x, wg, bias)]
    mir.shampoo_linear_grad(cf, x, wg, z, kind, *one)
    two = [torch.empty_like(t) for t in (x, wg, wu, wd)]
    mir.shampoo_gated_ffn_grad(c, x, wg, wu, wd, (g, u), *two, activation=kind)
    for fn, at, grads in ((layer, (x, wg, bias), one), (block, (x, wg, wu, wd), two)):
        at = [t.double() for t in at]
        for i, grad in enumerate(grads):
            v = torch.randn(at[i].shape, generator=gen, device="cuda", dtype=torch.float64)
            hi, lo = (fn(*[t + s * step * v if j == i else t for j, t in enumerate(at)]) for s in (1, -1))
            want, got = (hi - lo) / (2 * step), (grad.double() * v).sum()
            # float32 gradients: 2 d + f terms, two roundings of the kept values; differences: step^2 of third
            # derivatives, 2^-52 / step of the sum; relu: the kinks that the step crosses (some step T f of them)
            size = float((grad.double().abs() * v.abs()).sum())
            allowed = (2 * d + 2 * f) * ref.U * size + 1e-7 * size + (20 * step * size if kind == "relu" else 0)
            assert abs(float(want - got)) <= allowed, (kind, fn.__name__, i)


def test_network_step(mir):
    """x -> gated block -> MLP (gelu, residual) -> projection loss and back,
    accumulated over two batches, then an optimizer step: float32 against
    float64, and bfloat16 with everything kept in 8 bits against that."""
    import torch
    T, d, f, V = 96, 64, 160, 300
    gen = gen_of(14)
    shapes = [(f, d), (f, d), (d, f), (f, d), (f,), (d, f), (d,), (V, d)]
    W0 = [torch.randn(s, generator=gen, device="cuda") / s[-1] ** 0.5 for s in shapes]
    data = [(torch.randn((T, d), generator=gen, device="cuda"), torch.randint(0, V, (T,), generator=gen, device="cuda")) for _ in range(2)]

    W64 = [w.double().requires_grad_() for w in W0]
    for x, t in data:
        x = x.double()
        h = x + (torch.nn.functional.silu(x @ W64[0].t()) * (x @ W64[1].t())) @ W64[2].t()
        o = h + torch.nn.functional.gelu(h @ W64[3].t() + W64[4]) @ W64[5].t() + W64[6]
        (0.5 * torch.nn.functional.cross_entropy(o @ W64[7].t(), t)).backward()
    grads64 = [w.grad for w in W64]

    def train(dt, keep):
        W = [w.clone() for w in W0]
        opt = mir.Shampoo(W, block_size=64, beta2=0.9, eps=1e-4, root=mir.RootOpts(method="cn", iters=25, eps=1e-4), graft="sgd", lr=0.1)
        G = [torch.empty_like(w) for w in W[:7]]
        for k, (x, t) in enumerate(data):
            x = x.to(dt)
            kept = [mir.shampoo_kept_empty(T, f, keep, "cuda") for _ in range(3)]
            h = mir.shampoo_gated_ffn(x, W[0], W[1], W[2], residual=x, keep=kept[:2])
            a = mir.shampoo_linear(h, W[3], bias=W[4], activation="gelu", keep=kept[2])
            o = mir.shampoo_linear(a, W[5], bias=W[6], residual=h)
            do = torch.empty_like(o)
            loss = opt.projection_loss(7, o, t, dhidden=do, scale=0.5)
            if keep == "e4m3":  # what the weights' gradients read, in 8 bits
                x, h, a = (mir.shampoo_quantize_f8(v) for v in (x, h, a))
            da, dh, dx = (torch.empty((T, n), dtype=dt, device="cuda") for n in (f, d, d))
            more = k > 0
            mir.shampoo_linear_grad(do, a, W[5], dx=da, dw=G[5], dbias=G[6], accumulate=more)
            mir.shampoo_linear_grad(da, h, W[3], kept=kept[2], activation="gelu", dx=dh, dw=G[3], dbias=G[4], accumulate=more)
            dh += do
            mir.shampoo_gated_ffn_grad(dh, x, W[0], W[1], W[2], kept[:2], dx, *G[:3], accumulate=more)
            assert bool(torch.isfinite(loss)) and bool(torch.isfinite(dx).all())
        got = [g.double() for g in G]
        opt.step(G + [None])
        assert all(bool(torch.isfinite(w).all()) and not torch.equal(w, v) for w, v in zip(W, W0))
        return got

    # nine products in a row, each off by at most (300 + 2) 2^-23 of the magnitudes it sums, which are at most
    # some 20 times its result here: 9 20 3.6e-5 as an outermost bound
    off = [float((a - b).norm() / b.norm()) for a, b in zip(train(torch.float32, torch.float32), grads64)]
    log("float32: " + " ".join("%.1e" % v for v in off))
    assert max(off) < 6.5e-3
    # 8 bits: half a step of 2^-3 at most in each of two kept factors and in the operand they meet; bfloat16's
    # roundings are 2^-8 each
    off = [float((a - b).norm() / b.norm()) for a, b in zip(train(torch.bfloat16, "e4m3"), grads64)]
    log("bfloat16, kept in 8 bits: " + " ".join("%.1e" % v for v in off))
    assert max(off) < 3 * 2.0 ** -4 + 10 * 2.0 ** -8
