"""Every tile of every product of the feed-forward layers, and few rows, bit for bit: on
whole numbers small enough that each sum is exact in float32 in any order
(the sums of magnitudes stay below 2^24), with relu, the definition in float64
has one answer, rounded where the header says.  A product that lost bits of its
operands or sums, whatever their length, would show."""

import pytest

import ffn_reference as ref
import ffn_shapes
from test_gpu_ffn import gen_of

pytestmark = pytest.mark.gpu

EXACT = 2.0 ** 24
CASES = [(dt, s) for dt in ("bfloat16", "float32") for s in ffn_shapes.FEW + ffn_shapes.LINEAR[dt]]
GATED = [(dt, s) for dt in ("bfloat16", "float32") for s in ffn_shapes.FEW + ffn_shapes.GATED[dt]]


@pytest.fixture(scope="module")
def mir():
    import matrix_inverse_roots_amd as m
    return m


def whole(gen, rows, cols, high, dt):
    """Whole numbers from -high to high."""
    import torch
    return torch.randint(-high, high + 1, (rows, cols) if cols else (rows,), generator=gen, device="cuda").to(dt)


def largest(dt, length):
    """Operands that meet others of at most 2 in a sum of this length: 11 bits, which bfloat16 does not hold, in float32."""
    import torch
    return max(1, min(2047 if dt == torch.float32 else 127, 2 ** 22 // length))


def exact(want, *sums):
    """want, given that the sums of magnitudes behind it are exact."""
    assert all(float(s.max()) < EXACT for s in sums)
    return want


def same(got, want, what):
    import torch
    if isinstance(got, torch.Tensor):
        assert torch.equal(got, want.to(got.dtype)), what
        return
    q, s = ref.blocks(want.float(), 32)
    assert torch.equal(got[1].view(torch.uint8), s), what + ": scales"
    assert torch.equal(got[0].float(), q), what + ": codes"


def room(mir, rows, cols, keep, dt):
    return mir.shampoo_kept_empty(rows, cols, dt if keep == "dtype" else "e4m3", "cuda")


def kept_of(z, keep, dt):
    import torch
    if keep == "dtype":
        return z.to(dt)
    q, s = ref.blocks(z.float(), 32)
    return q.to(torch.float8_e4m3fn), s.view(torch.float8_e8m0fnu)


@pytest.mark.parametrize("keep", ["dtype", "e4m3"])
@pytest.mark.parametrize("dt,size", CASES)
def test_layer(mir, dt, size, keep):
    import torch
    dt = getattr(torch, dt)
    M, K, N = size
    gen = gen_of(M, K, N, 41)
    x, w = whole(gen, M, K, largest(dt, K), dt), whole(gen, N, K, 2, dt)
    bias, residual = whole(gen, N, 0, 1000, torch.float32), whole(gen, M, N, 100, dt)
    kept = room(mir, M, N, keep, dt)
    y = mir.shampoo_linear(x, w, bias=bias, activation="relu", residual=residual, keep=kept)
    z = exact(x.double() @ w.double().t(), x.double().abs() @ w.double().abs().t() + 1100)
    same(mir.shampoo_linear(x, w, torch.empty((M, N), device="cuda")), z, "z")
    z = z + bias.double()
    same(y, z.clamp(min=0) + residual.double(), "y")
    same(kept, z, "kept")
    del y, z, kept, residual

    x = whole(gen, M, K, 2, dt)
    dy = whole(gen, M, N, largest(dt, max(M, N)), dt)
    kept = kept_of(whole(gen, M, N, 3, torch.float64), keep, dt)
    dz = dy.double() * (ref.widen(kept, N) > 0)
    old, oldb = whole(gen, N, K, 1000, torch.float32), whole(gen, N, 0, 1000, torch.float32)
    more = keep == "dtype"   # float32 gradients, added to; else gradients of the operands' type, from x in 8 bits
    out = dict(dx=torch.empty((M, K), dtype=dt, device="cuda"), dw=old.clone() if more else torch.empty((N, K), dtype=dt, device="cuda"),
               dbias=oldb.clone() if more else torch.empty(N, device="cuda"))
    mir.shampoo_linear_grad(dy, x if more else mir.shampoo_quantize_f8(x), w, kept=kept, activation="relu", accumulate=more, **out)
    same(out["dx"], exact(dz @ w.double(), dz.abs() @ w.double().abs()), "dx")
    dw = exact(dz.t() @ x.double(), dz.abs().t() @ x.double().abs() + 1000)
    same(out["dw"], dw + old.double() if more else dw, "dw")
    same(out["dbias"], dz.sum(dim=0) + (oldb.double() if more else 0), "dbias")


@pytest.mark.parametrize("keep", ["dtype", "e4m3"])
@pytest.mark.parametrize("dt,size", GATED)
def test_block(mir, dt, size, keep):
    import torch
    dt = getattr(torch, dt)
    T, d, f = size
    gen = gen_of(T, d, f, 42)

    def rounded(t):
        return t.to(dt).double()

    x, wg, wu, wd = whole(gen, T, d, 1, dt), whole(gen, f, d, 1, dt), whole(gen, f, d, 1, dt), whole(gen, d, f, 1, dt)
    residual = whole(gen, T, d, 100, dt)
    pair = [room(mir, T, f, keep, dt) for _ in range(2)]
    y = mir.shampoo_gated_ffn(x, wg, wu, wd, activation="relu", residual=residual, keep=pair)
    g, u = x.double() @ wg.double().t(), x.double() @ wu.double().t()
    h = g.clamp(min=0) * u
    if T > 4 or keep == "e4m3":
        h = rounded(h)   # of few rows it stays float32
    same(pair[0], g, "gate")
    same(pair[1], u, "up")
    same(y, exact(h @ wd.double().t(), h.abs() @ wd.double().abs().t() + 100) + residual.double(), "y")
    del y, pair, g, u, h

    dy = residual.clamp(-1, 1)
    kept = [kept_of(whole(gen, T, f, 3, torch.float64), keep, dt) for _ in range(2)]
    g, u = (ref.widen(t, f) for t in kept)
    dh = dy.double() @ wd.double()
    du, dg, h = rounded(dh * g.clamp(min=0)), rounded(dh * u * (g > 0)), rounded(g.clamp(min=0) * u)
    more = keep == "dtype"
    gdt = torch.float32 if more else dt
    old = dict(dw_gate=whole(gen, f, d, 1000, gdt), dw_up=whole(gen, f, d, 1000, gdt), dw_down=whole(gen, d, f, 1000, gdt))
    out = {k: v.clone() for k, v in old.items()}
    dx = torch.empty((T, d), dtype=dt, device="cuda")
    x8 = x if more else mir.shampoo_quantize_f8(x)
    mir.shampoo_gated_ffn_grad(dy, x8, wg, wu, wd, kept, dx, activation="relu", accumulate=more, **out)
    same(dx, exact(dg @ wg.double() + du @ wu.double(), dg.abs() @ wg.double().abs() + du.abs() @ wu.double().abs()), "dx")
    for name, a, b in (("dw_gate", dg, x), ("dw_up", du, x), ("dw_down", dy.double(), h)):
        want = exact(a.t() @ b.double(), a.abs().t() @ b.double().abs() + 1000)
        same(out[name], want + old[name].double() if more else want, name)
    one = torch.empty((f, d), dtype=dt, device="cuda")   # a projection's gradient alone
    mir.shampoo_gated_ffn_grad(dy, x8, None, None, wd, kept, dw_up=one, activation="relu")
    same(one, du.t() @ x.double(), "dw_up alone")


def test_rows_past_32_bits(mir):
    """Rows of which the last lie more than 2^31 elements from the first: all
    of what the calls write, sums over the rows and over the long inner size among it."""
    import torch
    dt, M, K, N, step = torch.bfloat16, 66001, 17, 33024, 6000
    gen = gen_of(43)
    x, w, wd = whole(gen, M, K, 2, dt), whole(gen, N, K, 2, dt), whole(gen, K, N, 1, dt)
    pair = [mir.shampoo_kept_empty(M, N, "e4m3", "cuda") for _ in range(2)]
    y = mir.shampoo_linear(x, w, activation="relu", keep=pair[0])
    for r in range(0, M, step):
        z = x[r:r + step].double() @ w.double().t()
        same(y[r:r + step], z.clamp(min=0), "y")
        same(tuple(t[r:r + step] for t in pair[0]), z, "kept")
    out = dict(dx=torch.empty_like(x), dw=torch.empty((N, K), device="cuda"), dbias=torch.empty(N, device="cuda"))
    mir.shampoo_linear_grad(y, x, w, kept=pair[0], activation="relu", **out)
    dw, db = torch.zeros((N, K), dtype=torch.float64, device="cuda"), torch.zeros(N, dtype=torch.float64, device="cuda")
    for r in range(0, M, step):
        dz = y[r:r + step].double() * (ref.widen(tuple(t[r:r + step] for t in pair[0]), N) > 0)
        same(out["dx"][r:r + step], exact(dz @ w.double(), dz @ w.double().abs()), "dx")
        dw += dz.t() @ x[r:r + step].double()
        db += dz.sum(dim=0)
    same(out["dbias"], exact(db, db), "dbias")
    same(out["dw"], exact(dw, 2 * db), "dw")
    del out, y, dz, z

    out = mir.shampoo_gated_ffn(x, w, w, wd, activation="relu", keep=pair)
    dx, dwd = torch.empty_like(x), torch.empty((K, N), dtype=dt, device="cuda")
    dy = x.clamp(-1, 1)
    mir.shampoo_gated_ffn_grad(dy, x, w, w, wd, pair, dx, dw_down=dwd, activation="relu")
    want, size = (torch.zeros((K, N), dtype=torch.float64, device="cuda") for _ in range(2))
    for r in range(0, M, step):
        z = x[r:r + step].double() @ w.double().t()
        h = (z.clamp(min=0) * z).to(dt).double()
        same(out[r:r + step], exact(h @ wd.double().t(), h @ wd.double().abs().t()), "gated y")
        for t in pair:
            same(tuple(v[r:r + step] for v in t), z, "gated kept")
        z = ref.widen(tuple(t[r:r + step] for t in pair[0]), N)
        d = dy[r:r + step].double()
        dh = d @ wd.double()
        dg, h = (dh * z.clamp(min=0)).to(dt).double(), (z.clamp(min=0) * z).to(dt).double()   # dg is du: the projections are equal
        same(dx[r:r + step], exact(2 * dg @ w.double(), 2 * dg.abs() @ w.double().abs()), "gated dx")
        want += d.t() @ h
        size += d.abs().t() @ h
    same(dwd, exact(want, size), "gated dw_down")
    torch.cuda.empty_cache()
