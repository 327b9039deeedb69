"""Parity of the 8-bit quantisation and block-scaled product with their
definitions in float64.

Quantisation is exact up to its one rounding, so every byte has to be the
definition's.  The product's operands are exact numbers; its sum of K terms
runs in float32 (each addition off by at most 2^-23 of the running magnitude
whichever way the matrix core rounds) and is rounded once to the result's
type: |error| <= K 2^-23 (|A| |B|^T) + eps/2 |C| per element.
"""

import numpy as np
import pytest

import f8_reference as ref
from helpers import log

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mir():
    import matrix_inverse_roots_amd as m
    return m


def values_of(q, fmt):
    import torch
    return ref.code_values(fmt)[q.view(torch.uint8).cpu().numpy()]


def bytes_of(s):
    import torch
    return s.view(torch.uint8).cpu().numpy()


def inputs(rows, cols, dtype, seed, n=1):
    """Rows of very different sizes, zero blocks, blocks at the edges of the
    format's range and the smallest numbers of the type."""
    import torch
    g = np.random.default_rng(seed)
    x = g.standard_normal((n, rows, cols)) * np.exp(2.0 * g.standard_normal((n, rows, 1)))
    x[:, ::5] = 0.0
    if rows > 2:
        x[:, 1] = 448.0 * g.choice([-1.0, 0.5, 1.0], size=(n, cols))
        x[:, 2] *= 1e-30 if dtype != torch.float16 else 1e-6
    if rows > 3:
        x[:, 3] *= 1e-40 if dtype != torch.float16 else 1e-7
    return torch.from_numpy(x).to(torch.float32).to(dtype).cuda()


SHAPES = [(1, 1), (1, 128), (3, 130), (129, 257), (128, 128), (5, 1000), (300, 64), (260, 1025)]


@pytest.mark.parametrize("transpose", [False, True, "both"])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
@pytest.mark.parametrize("dt", ["float32", "float16", "bfloat16"])
def test_quantize_is_the_definition(mir, dt, fmt, block_rows, transpose):
    import torch
    for k, (rows, cols) in enumerate(SHAPES):
        x = inputs(rows, cols, getattr(torch, dt), k, n=2)
        got = mir.shampoo_quantize_f8(x, fmt=fmt, block_rows=block_rows, transpose=transpose)
        pairs = [(got[0], False), (got[1], True)] if transpose == "both" else [(got, bool(transpose))]
        for (q, s), t in pairs:
            v, b = values_of(q, fmt), bytes_of(s)
            for i in range(2):
                qr, sr = ref.quantize(x[i].double().cpu().numpy(), fmt, block_rows, t)
                np.testing.assert_array_equal(b[i], sr, err_msg=f"scales {rows}x{cols} {t}")
                np.testing.assert_array_equal(v[i], qr, err_msg=f"values {rows}x{cols} {t}")
    log(f"{dt} {fmt} {block_rows} {transpose}: {len(SHAPES)} shapes equal")


@pytest.mark.parametrize("fmt", ["e4m3", "e5m2"])
def test_quantize_values_that_are_not_finite(mir, fmt):
    """They keep out of the block's scale; NaN stays NaN, an infinity stays
    one where the format has it."""
    import torch
    x = np.random.default_rng(3).standard_normal((130, 200)).astype(np.float32)
    x[0, 5], x[1, 7], x[2, 0] = np.nan, np.inf, -np.inf
    x[3, :128] = np.nan
    for block_rows in (1, 128):
        got = mir.shampoo_quantize_f8(torch.from_numpy(x).cuda(), fmt=fmt, block_rows=block_rows, transpose="both")
        for (q, s), t in zip(got, (False, True)):
            qr, sr = ref.quantize(x, fmt, block_rows, t)
            np.testing.assert_array_equal(bytes_of(s), sr)
            np.testing.assert_array_equal(values_of(q, fmt), qr)


def test_quantize_strided_and_misaligned_rows(mir):
    """Rows of a wider matrix, from an odd column on; matrices that are apart."""
    import torch
    big = inputs(70, 411, torch.bfloat16, 11, n=3)
    for x in (big[:, 3:40, 5:206], big[1, :, 1:], big[:, :1, 8:136], big[::2]):
        (q, s), (qt, st) = mir.shampoo_quantize_f8(x, transpose="both")
        y = x if x.dim() == 3 else x[None]
        for i in range(y.shape[0]):
            for (v, b), t in (((q, s), False), ((qt, st), True)):
                qr, sr = ref.quantize(y[i].double().cpu().numpy(), "e4m3", 1, t)
                v, b = (v, b) if x.dim() == 2 else (v[i], b[i])
                np.testing.assert_array_equal(values_of(v, "e4m3"), qr)
                np.testing.assert_array_equal(bytes_of(b), sr)


def product_case(mir, n, M, N, K, fa, fb, rba, rbb, out, seed=0):
    import torch
    g = np.random.default_rng(seed)
    a = g.standard_normal((n, M, K)) * np.exp(g.standard_normal((n, M, 1)))
    b = g.standard_normal((n, N, K)) * np.exp(g.standard_normal((n, N, 1)))
    a[:, :, K // 3] = 0.0
    a, b = (torch.from_numpy(t).float().cuda() for t in (a, b))
    qa, sa = mir.shampoo_quantize_f8(a, fmt=fa, block_rows=rba)
    qb, sb = mir.shampoo_quantize_f8(b, fmt=fb, block_rows=rbb)
    c = torch.full((n, M, N), float("nan"), dtype=getattr(torch, out), device="cuda")
    assert mir.shampoo_matmul_f8(qa, sa, qb, sb, c) is c
    got = c.double().cpu().numpy()
    eps = torch.finfo(c.dtype).eps
    tiny = torch.finfo(c.dtype).smallest_normal * eps
    worst = 0.0
    for i in range(n):
        A = ref.stand_for(values_of(qa, fa)[i], bytes_of(sa)[i], rba)
        B = ref.stand_for(values_of(qb, fb)[i], bytes_of(sb)[i], rbb)
        want = A @ B.T
        bound = K * 2.0 ** -23 * (np.abs(A) @ np.abs(B).T) + eps / 2 * np.abs(want) + tiny
        err = np.abs(got[i] - want)
        assert (err <= bound).all(), (M, N, K, float(np.nanmax(err / np.maximum(bound, 1e-300))))
        worst = max(worst, float(np.linalg.norm(got[i] - want) / max(np.linalg.norm(want), 1e-300)))
    log(f"{n} x {M} x {N} x {K} {fa} {fb} {rba} {rbb} {out}: {worst:.2e}")


@pytest.mark.parametrize("out", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (1, 4096, 1024), (33, 65, 128), (127, 129, 130), (257, 300, 384),
                                   (64, 64, 8192), (2, 1000, 5000), (300, 17, 640)])
def test_product_matches_float64(mir, M, N, K, out):
    product_case(mir, 1, M, N, K, "e4m3", "e4m3", 1, 128, out)


@pytest.mark.parametrize("M", [1, 2, 3, 4, 5, 8])
@pytest.mark.parametrize("N,K,rbb", [(1, 128, 1), (13, 700, 1), (4096, 1024, 128), (301, 3000, 128)])
def test_product_of_few_rows(mir, M, N, K, rbb):
    """One to four rows take the kernel for few rows, more the tiles; every
    pair of formats, two matrices, scales of A by row and by 128 rows."""
    for k, (fa, fb) in enumerate((("e4m3", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2"))):
        product_case(mir, 2, M, N, K, fa, fb, 128 if k % 2 else 1, rbb, ("float32", "bfloat16", "float16", "float32")[k], seed=M)


@pytest.mark.parametrize("fa,fb", [("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("rba,rbb", [(1, 1), (128, 1), (128, 128)])
def test_product_formats_and_blocks(mir, fa, fb, rba, rbb):
    product_case(mir, 2, 150, 270, 700, fa, fb, rba, rbb, "float32", seed=5)


def test_product_large_tiles_and_stacks(mir):
    """Shapes that take the 256-tiles: many tiles, several a workgroup, ragged edges."""
    product_case(mir, 17, 1024, 1000, 256, "e4m3", "e4m3", 1, 1, "float32", seed=2)
    product_case(mir, 1, 4111, 4100, 640, "e4m3", "e4m3", 1, 128, "bfloat16", seed=3)


def test_product_two_dimensional_operands_streams_and_empty(mir):
    import torch
    a = torch.randn(40, 256, device="cuda")
    b = torch.randn(50, 256, device="cuda")
    qa, qb = mir.shampoo_quantize_f8(a), mir.shampoo_quantize_f8(b, block_rows=128)
    first = mir.shampoo_matmul_f8(*qa, *qb, torch.empty(40, 50, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    second = torch.empty(40, 50, device="cuda")
    mir.shampoo_matmul_f8(*qa, *qb, second, stream=side)
    side.synchronize()
    assert torch.equal(first, second)
    none = mir.shampoo_quantize_f8(torch.empty(0, 256, device="cuda"))
    assert none[0].shape == (0, 256) and none[1].shape == (0, 4)
    out = mir.shampoo_matmul_f8(*none, *qb, torch.empty(0, 50, device="cuda"))
    assert out.shape == (0, 50)


def test_linear_layer_gradients(mir):
    """y = x W^T and its gradients as three products, against the formulas on
    the quantised operands, and the directional derivative of sum(y dy)
    against a difference quotient of the definition in float64."""
    import torch
    g = np.random.default_rng(8)
    T, K, N = 200, 320, 450
    x, w, dy = g.standard_normal((T, K)), g.standard_normal((N, K)) / 18.0, g.standard_normal((T, N))
    xd, wd, dyd = (torch.from_numpy(t).float().cuda() for t in (x, w, dy))
    xq, xt = mir.shampoo_quantize_f8(xd, transpose="both")
    wq, wt = mir.shampoo_quantize_f8(wd, block_rows=128, transpose="both")
    dq, dt = mir.shampoo_quantize_f8(dyd, fmt="e5m2", transpose="both")
    y = mir.shampoo_matmul_f8(*xq, *wq, torch.empty(T, N, device="cuda")).double().cpu().numpy()
    dx = mir.shampoo_matmul_f8(*dq, *wt, torch.empty(T, K, device="cuda")).double().cpu().numpy()
    dw = mir.shampoo_matmul_f8(*dt, *xt, torch.empty(N, K, device="cuda")).double().cpu().numpy()
    # each operand is off by at most half a step: e4m3 2^-4, e5m2 2^-3 of the
    # value (more only below the smallest normal number, 2^-15 of the block's
    # largest and far less than that here)
    e4, e5, low = 2.0 ** -4, 2.0 ** -3, 2.0 ** -9
    X, W, D = np.abs(x), np.abs(w), np.abs(dy)

    def bound(A, ea, B, eb):
        A_, B_ = A + low * A.max(), B + low * B.max()
        return (1 + ea) * A_ @ ((1 + eb) * B_) - A_ @ B_ + (A_ @ B_ - A @ B)

    assert (np.abs(y - x @ w.T) <= bound(X, e4, W.T, e4)).all()
    assert (np.abs(dx - dy @ w) <= bound(D, e5, W, e4)).all()
    assert (np.abs(dw - dy.T @ x) <= bound(D.T, e5, X, e4)).all()
    # sum(y dy) along a direction u of x: its derivative is <dx, u>
    u = g.standard_normal((T, K))
    f = lambda s: float(np.sum(((x + s * u) @ w.T) * dy))  # noqa: E731
    slope = (f(1e-3) - f(-1e-3)) / 2e-3
    assert abs(float(np.sum(dx * u)) - slope) <= float(np.sum(bound(D, e5, W, e4) * np.abs(u)))
    rel = [np.linalg.norm(a - b) / np.linalg.norm(b) for a, b in ((y, x @ w.T), (dx, dy @ w), (dw, dy.T @ x))]
    log("linear layer in 8 bits, relative: y %.3f dx %.3f dw %.3f" % tuple(rel))


def held(mir, g, n, rows, K, fmt, scales):
    """Random finite 8-bit values, the largest and smallest among them, and these scale bytes."""
    import torch
    ok = np.flatnonzero(np.isfinite(ref.code_values(fmt)))
    q = g.choice(ok, size=(n, rows, K)).astype(np.uint8)
    q[:, :, ::7] = ok[np.argmax(ref.code_values(fmt)[ok])]
    q[:, :, 3::11] = 1   # the smallest subnormal number
    s = np.full((n, scales.shape[1], ref.up(K // 128, 4)), 127, dtype=np.uint8)
    s[:, :, :K // 128] = scales
    kind = torch.float8_e4m3fn if fmt == "e4m3" else torch.float8_e5m2
    return torch.from_numpy(q).cuda().view(kind), torch.from_numpy(s).cuda().view(torch.float8_e8m0fnu), q, s


@pytest.mark.parametrize("out", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("fa,fb", [("e4m3", "e4m3"), ("e4m3", "e5m2"), ("e5m2", "e4m3"), ("e5m2", "e5m2")])
@pytest.mark.parametrize("M,N", [(4, 70), (5, 70), (300, 257)])
def test_scales_over_their_whole_range(mir, M, N, fa, fb, out):
    """Scales of 2^-127 to 2^127 on one side against the opposite on the other,
    all blocks alike, block by block, and row by row (where a huge row meets a
    huge one the result overflows in any arithmetic; those are not compared).
    16-bit results: the instructions drop what lies 2^-13 below the largest."""
    import torch
    g = np.random.default_rng(M)
    K = 640
    for kind in ("same", "blocks", "rows"):
        ends = np.array([0, 1, 7, 16, 17, 120, 127, 239, 240, 247, 254])
        if kind == "same":
            e = np.broadcast_to(ends[:, None, None], (len(ends), 1, K // 128))
            a_e, b_e = np.repeat(e, M, 1), np.repeat(254 - e, N, 1)
        elif kind == "blocks":
            e = g.choice(ends, size=(3, 1, K // 128))
            a_e, b_e = np.repeat(e, M, 1), np.repeat(254 - e, N, 1)
        else:
            a_e = np.repeat(g.choice(ends, size=(3, M, 1)), K // 128, 2)
            b_e = np.repeat(g.choice(ends, size=(3, N, 1)), K // 128, 2)
        n = len(a_e)
        a, sa, qa, ha = held(mir, g, n, M, K, fa, a_e)
        b, sb, qb, hb = held(mir, g, n, N, K, fb, b_e)
        c = torch.full((n, M, N), float("nan"), dtype=getattr(torch, out), device="cuda")
        got = mir.shampoo_matmul_f8(a, sa, b, sb, c).double().cpu().numpy()
        lim = torch.finfo(c.dtype)
        for i in range(n):
            A, B = ref.stand_for(ref.code_values(fa)[qa[i]], ha[i], 1), ref.stand_for(ref.code_values(fb)[qb[i]], hb[i], 1)
            want, size = A @ B.T, np.abs(A) @ np.abs(B).T
            # no partial sum overflows; below the smallest normal numbers the
            # result's and the sums' absolute steps count
            safe = size < lim.max
            assert kind == "rows" or out == "float16" or safe.all()
            bound = (K * 2.0 ** -23 + (2.0 ** -13 if out != "float32" else 0.0)) * size + lim.eps / 2 * np.abs(want)
            bound += lim.smallest_normal * lim.eps + K * 2.0 ** -126
            err = np.abs(got[i] - want)
            assert (err <= bound)[safe].all(), (kind, i, float(np.nanmax((err / bound)[safe])), int(np.isnan(got[i][safe]).sum()))


def test_quantised_values_near_the_largest_float32(mir):
    """Entries just below 2^128 round up to it; their products with small numbers are ordinary."""
    import torch
    x = torch.full((40, 256), 3.4e38, device="cuda")
    x[::2] *= -0.99
    w = torch.full((70, 256), 2.0 ** -100, device="cuda")
    a, b = mir.shampoo_quantize_f8(x), mir.shampoo_quantize_f8(w)
    A = ref.stand_for(values_of(a[0], "e4m3"), bytes_of(a[1]), 1)
    B = ref.stand_for(values_of(b[0], "e4m3"), bytes_of(b[1]), 1)
    assert np.abs(A).max() == 2.0 ** 128
    for rows in (4, 5, 40):
        for out in (torch.float32, torch.bfloat16):
            c = mir.shampoo_matmul_f8(a[0][:rows], a[1][:rows], *b, torch.empty((rows, 70), dtype=out, device="cuda"))
            want = A[:rows] @ B.T
            assert (np.abs(c.double().cpu().numpy() - want) <= 2.0 ** (-8 if out == torch.bfloat16 else -14) * np.abs(want)).all()


def test_extreme_blocks_of_many_tiles_and_split_k(mir):
    """A few extreme blocks among ordinary ones: tiles of every shape, several
    a workgroup, and a k that is split; the other results keep their bits."""
    import torch
    g = np.random.default_rng(1)
    for n, M, N, K in ((3, 150, 260, 512), (9, 1500, 1030, 256), (1, 64, 64, 8192)):
        a = torch.from_numpy(g.standard_normal((n, M, K))).float().cuda()
        b = torch.from_numpy(g.standard_normal((n, N, K))).float().cuda()
        (qa, sa), (qb, sb) = mir.shampoo_quantize_f8(a), mir.shampoo_quantize_f8(b)
        plain = mir.shampoo_matmul_f8(qa, sa, qb, sb, torch.empty((n, M, N), device="cuda"))
        ha, hb = sa.view(torch.uint8), sb.view(torch.uint8)
        # block 1 of a few rows of A at 2^120, and of every row of B of those matrices at 2^-120
        rows = g.integers(0, M, 5)
        ha[0, torch.from_numpy(rows).cuda(), 1] = 247
        hb[0, :, 1] = 7
        c = mir.shampoo_matmul_f8(qa, sa, qb, sb, torch.full((n, M, N), float("nan"), device="cuda"))
        assert torch.equal(c[1:], plain[1:])
        A, B = (ref.stand_for(values_of(q, "e4m3")[0], bytes_of(s)[0], 1) for q, s in ((qa, sa), (qb, sb)))
        want, size = A @ B.T, np.abs(A) @ np.abs(B).T
        err = np.abs(c[0].double().cpu().numpy() - want)
        assert (err <= K * 2.0 ** -23 * size + 2.0 ** -24 * np.abs(want)).all()
