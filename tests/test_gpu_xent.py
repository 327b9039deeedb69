"""Parity of the projection's softmax cross entropy and its gradients with
the formulas in float64.

Tolerances.  A logit is a float32 sum of d products (exact for bfloat16,
rounded for float32): off by at most dz = (d + 1) 2^-23 |x| |w|.  The row's
lse then is off by at most max dz and the rounding of itself; exp and log
add a few units of 2^-23 (t below).  A softmax entry is off by the relative
2 max dz + t, and in the bfloat16 form by two roundings of 2^-8 more.  The
gradients' sums add K 2^-23 of their magnitudes, and their own rounding eps/2.
"""

import numpy as np
import pytest

from helpers import log

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


@pytest.fixture(scope="module")
def mir():
    import matrix_inverse_roots_amd as m
    return m


def make(N, d, V, dt, seed, size=1.5, skip=0.2):
    import torch
    g = np.random.default_rng(seed)
    dtype = getattr(torch, dt)
    w = torch.from_numpy(g.standard_normal((V, d)) * size / np.sqrt(d)).float().to(dtype)
    t = g.integers(0, V, N)
    h = g.standard_normal((N, d)) + w.double().numpy()[t] * g.uniform(0, 8, (N, 1))
    t = np.where(g.uniform(size=N) < skip, -100, t)
    if N:
        t[0] = V - 1
    h = torch.from_numpy(h).float().to(dtype)
    return h.cuda(), w.cuda(), torch.from_numpy(t).cuda()


def definition(h, w, t, reduction, row_scale=None, scale=1.0):
    """(losses or loss, dh, dw, lse) in float64, and bounds of the first three's errors."""
    x, W = h.double().cpu().numpy(), w.double().cpu().numpy()
    t = t.cpu().numpy()
    N, d = x.shape
    z = x @ W.T
    dz = (d + 1) * U * (np.abs(x) @ np.abs(W).T)
    m = z.max(axis=1, keepdims=True)
    lse = np.log(np.exp(z - m).sum(axis=1)) + m[:, 0]
    kept = t != -100
    at = np.where(kept, t, 0)
    rows = np.arange(N)
    s = np.full(N, scale) if row_scale is None else scale * row_scale.double().cpu().numpy()
    wide = dz.max(axis=1)
    # exp2 of (z - m) log2 e: the product's rounding is 2^-24 of an exponent of at most 130
    few = 160 * U
    own = np.ones(N) if reduction == "none" else s   # "none" gives the rows' losses as they are
    loss = np.where(kept, own * (lse - z[rows, at]), 0.0)
    loss_err = np.where(kept, np.abs(own) * (2 * wide + few + 2 * U * (np.abs(lse) + np.abs(z[rows, at]))), 0.0) + 2 * U * np.abs(loss)
    g = np.where(kept, s, 0.0)
    if reduction == "mean":
        g = g / max(int(kept.sum()), 1)
        loss, loss_err = loss.sum() / max(int(kept.sum()), 1), loss_err.sum() / max(int(kept.sum()), 1) + U * abs(loss.sum())
    elif reduction == "sum":
        loss, loss_err = loss.sum(), loss_err.sum() + U * np.abs(loss).sum()
    P = np.exp(z - lse[:, None])
    half = 2.0 ** -8 if "bfloat16" in str(h.dtype) else U
    rel = (2 * wide + few + 2 * U * np.abs(lse))[:, None] + 2.1 * half
    dP = P * rel
    P = P.copy()
    # the target's own entry comes from its float32 logit and is rounded once
    p_t = P[rows, at].copy()
    P[rows, at] -= 1.0
    dP[rows, at] = p_t * rel[:, 0] + half * np.abs(P[rows, at])
    P, dP = P * g[:, None], dP * np.abs(g)[:, None]
    import torch
    eps = torch.finfo(h.dtype).eps
    aP = np.abs(P) + dP
    dh, dw = P @ W, P.T @ x
    dh_err = dP @ np.abs(W) + (w.shape[0] + 8) * U * (aP @ np.abs(W)) + eps / 2 * np.abs(dh)
    dw_err = dP.T @ np.abs(x) + (N + 8) * U * (aP.T @ np.abs(x)) + eps / 2 * np.abs(dw)
    return loss, dh, dw, lse, loss_err, dh_err * 1.01 + 1e-37, dw_err * 1.01 + 1e-37


def check(got, want, bound, what):
    got = got.double().cpu().numpy()
    err = np.abs(got - want)
    assert np.isfinite(got).all(), what
    assert (err <= bound).all(), (what, float(np.max(err / np.maximum(bound, 1e-300))))
    n = np.linalg.norm(want)
    return float(np.linalg.norm(got - want) / n) if n > 0 else float(np.linalg.norm(got))


def run(mir, N, d, V, dt, reduction="mean", seed=0, row_scale=False, scale=1.0, grads=True, dw_f32=False, **kw):
    import torch
    h, w, t = make(N, d, V, dt, seed)
    rs = torch.from_numpy(np.random.default_rng(seed + 1).uniform(-1, 2, N)).float().cuda() if row_scale else None
    nan = float("nan")
    dh = torch.full_like(h, nan) if grads else None
    dw = torch.full_like(w, nan, dtype=torch.float32 if dw_f32 else w.dtype) if grads else None
    lse = torch.full((N,), nan, device="cuda")
    loss = mir.shampoo_linear_xent(h, w, t, reduction=reduction, row_scale=rs, scale=scale, dhidden=dh, dweight=dw,
                                   lse=lse, **kw)
    L, DH, DW, LSE, eL, eDH, eDW = definition(h, w, t, reduction, rs, scale)
    far = [check(loss, L, eL, "loss")]
    wide = (d + 1) * U * np.max(np.abs(h.double().cpu().numpy()) @ np.abs(w.double().cpu().numpy()).T, axis=1, initial=0.0)
    check(lse, LSE, wide + 160 * U + 2 * U * np.abs(LSE), "lse")
    if grads:
        far += [check(dh, DH, eDH, "dhidden"), check(dw, DW, eDW, "dweight")]
    log(f"N {N} d {d} V {V} {dt} {reduction}: " + " ".join("%.1e" % f for f in far))


SIZES = [(1, 1, 1), (1, 64, 1000), (3, 100, 129), (2, 8, 2), (130, 96, 257), (64, 1000, 128), (257, 33, 700), (300, 200, 5001)]


@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
@pytest.mark.parametrize("N,d,V", SIZES)
def test_loss_and_gradients(mir, N, d, V, dt, reduction):
    run(mir, N, d, V, dt, reduction)


@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
def test_loss_alone_row_scales_and_scale(mir, dt):
    run(mir, 200, 128, 3000, dt, "none", grads=False)
    run(mir, 200, 128, 3000, dt, "none", row_scale=True, scale=0.25)
    run(mir, 200, 128, 3000, dt, "mean", row_scale=True, scale=3.0)


@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
@pytest.mark.parametrize("panel", [1, 100, 256])
def test_rows_taken_in_panels(mir, dt, panel):
    """Several panels, the last one shorter; the weight's gradient sums over them."""
    run(mir, 600 if panel > 1 else 5, 72, 900, dt, "mean", panel_rows=panel)


def test_weight_gradient_in_float32_and_accumulated(mir):
    """Two micro-batches into one float32 gradient, in one and in several panels."""
    import torch
    for panel in (0, 64):
        h1, w, t1 = make(150, 64, 777, "bfloat16", 1)
        h2, _, t2 = make(90, 64, 777, "bfloat16", 2)
        dw = torch.zeros(777, 64, device="cuda")
        want, bound = 0.0, 0.0
        for h, t in ((h1, t1), (h2, t2)):
            mir.shampoo_linear_xent(h, w, t, dweight=dw, accumulate=True, scale=0.5, panel_rows=panel)
            r = definition(h, w, t, "mean", scale=0.5)
            want, bound = want + r[2], bound + r[6]
        check(dw, want, bound + U * np.abs(want), "accumulated")
        run(mir, 150, 64, 777, "bfloat16", dw_f32=True, panel_rows=panel)
        # and onto a bfloat16 gradient: one more rounding
        db = torch.ones(777, 64, device="cuda", dtype=torch.bfloat16)
        mir.shampoo_linear_xent(h1, w, t1, dweight=db, accumulate=True, panel_rows=panel)
        r = definition(h1, w, t1, "mean")
        check(db, r[2] + 1.0, r[6] + 2.0 ** -8 * np.abs(r[2] + 1.0), "onto bfloat16")


@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
def test_no_row_kept_and_no_rows(mir, dt):
    import torch
    h, w, t = make(40, 64, 300, dt, 3)
    t.fill_(-100)
    dh, dw = torch.full_like(h, float("nan")), torch.full_like(w, float("nan"))
    for red in ("mean", "sum"):
        assert mir.shampoo_linear_xent(h, w, t, dhidden=dh, dweight=dw, reduction=red).item() == 0.0
        assert not dh.any() and not dw.any()
    assert not mir.shampoo_linear_xent(h, w, t, reduction="none").any()
    e = h[:0]
    dw.fill_(float("nan"))
    assert mir.shampoo_linear_xent(e, w, t[:0], dhidden=dh[:0], dweight=dw).item() == 0.0
    assert not dw.any()
    dw.fill_(2.0)
    mir.shampoo_linear_xent(e, w, t[:0], dweight=dw, accumulate=True)
    assert (dw == 2.0).all()


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
@pytest.mark.parametrize("with_dweight", [False, True])
def test_no_rows_with_a_pointer_to_targets(mir, with_dweight, reduction):
    """The C call with N = 0 and every pointer valid (an empty tensor's is
    null, so the binding does not come this way): loss 0, dweight 0 or, accumulated, as it was."""
    import ctypes
    import torch
    w = torch.ones(70, 64, device="cuda")
    h, dw = torch.ones(3, 64, device="cuda"), torch.full_like(w, 3.0)
    t, loss = torch.zeros(3, dtype=torch.int64, device="cuda"), torch.full((), 9.0, device="cuda")
    a = mir.XentArgsC(hidden=h.data_ptr(), weight=w.data_ptr(), targets=t.data_ptr(), loss=loss.data_ptr(), ld_hidden=64,
                      ld_weight=64, ld_dhidden=64, ld_dweight=64, N=0, V=70, d=64, ignore_index=-100, dt=mir.F32,
                      weight_dt=mir.F32, dweight_dt=mir.F32, logits_dt=mir.F32, reduction=mir.REDUCTIONS[reduction], scale=1.0,
                      dweight=dw.data_ptr() if with_dweight else None)
    need = ctypes.c_size_t(0)
    assert mir.lib.shampoo_linear_xent_workspace(ctypes.byref(a), ctypes.byref(need)) == mir.OK
    ws = torch.empty(need.value, dtype=torch.uint8, device="cuda")
    a.ws, a.ws_bytes = ws.data_ptr(), need.value
    stream = torch.cuda.current_stream().cuda_stream
    for accumulate in (1, 0):
        a.accumulate = accumulate
        assert mir.lib.shampoo_linear_xent(ctypes.byref(a), stream) == mir.OK
        torch.cuda.synchronize()
        assert loss.item() == (9.0 if reduction == "none" else 0.0)
        assert (dw == (3.0 if accumulate or not with_dweight else 0.0)).all()


@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
def test_targets_outside_the_vocabulary(mir, dt):
    """Loud, and only where they are: NaN in that row's loss and gradient."""
    import torch
    for bad in (300, -1, 1 << 40):
        h, w, t = make(40, 64, 300, dt, 4)
        t[7] = bad
        dh = torch.empty_like(h)
        loss = mir.shampoo_linear_xent(h, w, t, dhidden=dh, reduction="none")
        nan = torch.isnan(loss).cpu().numpy()
        assert nan[7] and nan.sum() == 1
        rows = torch.isnan(dh).all(dim=1).cpu().numpy()
        assert rows[7] and torch.isnan(dh).any(dim=1).sum().item() == 1


@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
def test_extreme_logits(mir, dt):
    """Logits of +-10^4 neither overflow nor lose the row; a column of -inf
    logits has probability zero; an infinite row is NaN and stays alone."""
    import torch
    h, w, t = make(70, 64, 500, dt, 5, size=1.0)
    h, w = h.clone(), w.clone()
    h[3] *= 3000.0
    h[4] = 0.0
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    loss = mir.shampoo_linear_xent(h, w, t, dhidden=dh, dweight=dw, reduction="none")
    r = definition(h, w, t, "none")
    check(loss, r[0], r[4], "loss")
    check(dh, r[1], r[5], "dhidden")
    check(dw, r[2], r[6], "dweight")
    h[:] = h.abs() + 0.1
    w[17] = -float("inf")
    t[:] = 3
    z = h.double() @ w.double().t()
    loss = mir.shampoo_linear_xent(h, w, t, reduction="none").double()
    want = torch.logsumexp(z, 1) - z[:, 3]
    assert torch.allclose(loss, want, rtol=1e-4, atol=1e-3)
    h[9] = float("nan")
    loss = mir.shampoo_linear_xent(h, w, t, reduction="none")
    assert torch.isnan(loss).nonzero().flatten().tolist() == [9]


@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
def test_strided_and_misaligned_rows(mir, dt):
    """Views of wider matrices, inputs and gradients; what lies between the rows stays as it was."""
    import torch
    h0, w0, t = make(90, 100, 333, dt, 6)
    H = torch.zeros(90, 131, dtype=h0.dtype, device="cuda")
    W = torch.zeros(333, 117, dtype=h0.dtype, device="cuda")
    H[:, 3:103], W[:, 1:101] = h0, w0
    DH, DW = torch.full_like(H, 5.0), torch.full_like(W, 5.0)
    loss = mir.shampoo_linear_xent(H[:, 3:103], W[:, 1:101], t, dhidden=DH[:, 3:103], dweight=DW[:, 1:101])
    r = definition(h0, w0, t, "mean")
    check(loss, r[0], r[4], "loss")
    check(DH[:, 3:103], r[1], r[5], "dhidden")
    check(DW[:, 1:101], r[2], r[6], "dweight")
    for D, a, b in ((DH, 3, 103), (DW, 1, 101)):
        assert (D[:, :a] == 5.0).all() and (D[:, b:] == 5.0).all()


def test_gradient_against_differences(mir):
    """The hidden gradient along a direction, against a central difference of
    the definition (float64)."""
    import torch
    h, w, t = make(20, 48, 400, "float32", 7)
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    mir.shampoo_linear_xent(h, w, t, dhidden=dh, dweight=dw)
    g = np.random.default_rng(9)
    for M, D in ((h, dh), (w, dw)):
        u = torch.from_numpy(g.standard_normal(tuple(M.shape))).cuda()

        def f(s):
            a = (h.double() + s * u) if M is h else h.double()
            b = (w.double() + s * u) if M is w else w.double()
            keep = t != -100
            return torch.nn.functional.cross_entropy((a @ b.t())[keep], t[keep]).item()

        slope = (f(1e-4) - f(-1e-4)) / 2e-4
        # third derivatives are of the size of the logits' spread cubed: 1e-8
        # times a few hundred at most; float32 gradients 1e-5 of their size
        assert abs((D.double() * u).sum().item() - slope) <= 1e-5 * (D.double().abs() * u.abs()).sum().item() + 1e-5


def test_same_bits_every_time_on_every_stream(mir):
    import torch
    h, w, t = make(500, 256, 4001, "bfloat16", 10)
    got = []
    side = torch.cuda.Stream()
    for stream in (None, None, side):
        dh, dw = torch.empty_like(h), torch.empty_like(w)
        torch.cuda.synchronize()
        loss = torch.empty((), device="cuda")
        ws = torch.full((mir.shampoo_linear_xent_workspace(h, w, t, dh, dw),), 0xFF, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        mir.shampoo_linear_xent(h, w, t, loss=loss, dhidden=dh, dweight=dw, ws=ws, stream=stream)
        torch.cuda.synchronize()
        got.append((loss, dh, dw))
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))


def test_captured_and_replayed(mir):
    """A graph of the loss with its gradients and an 8-bit product, replayed on
    refilled buffers with eager work between, gives the eager call's bits."""
    import torch
    h, w, t = make(300, 128, 2500, "bfloat16", 12)
    dh, dw, loss = torch.empty_like(h), torch.empty_like(w), torch.empty((), device="cuda")
    c = torch.empty(300, 2500, device="cuda")
    ws = torch.empty(mir.shampoo_linear_xent_workspace(h, w, t, dh, dw), dtype=torch.uint8, device="cuda")

    def work():
        mir.shampoo_linear_xent(h, w, t, loss=loss, dhidden=dh, dweight=dw, ws=ws)
        a, b = mir.shampoo_quantize_f8(h), mir.shampoo_quantize_f8(w, block_rows=128)
        mir.shampoo_matmul_f8(*a, *b, c)

    work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        work()
    for seed in range(5):
        h2, _, t2 = make(300, 128, 2500, "bfloat16", 20 + seed)
        h.copy_(h2)
        t.copy_(t2)
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (loss, dh, dw, c)]
        for x in (loss, dh, dw, c):
            x.fill_(float("nan"))
        work()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, (loss, dh, dw, c)))


def test_default_panels_of_a_long_batch(mir):
    """More rows than one default panel holds (float32, a wide vocabulary):
    equal panels, against float64 within the bounds of `definition`, which are
    formed on the device here.  (A sum of 131072 float32 terms may be off by
    131072 2^-23 of the sum of their magnitudes; the results of panels of 0,
    700 and 5200 rows differ among themselves by 1e-5 of their size, as
    a plain float32 product does from float64.)"""
    import torch
    N, d, V = 5200, 16, 131072
    h, w, t = make(N, d, V, "float32", 13)
    x, W = h.double(), w.double()
    keep = t != -100
    n = int(keep.sum())
    dw, dw_err, loss, loss_err = torch.zeros_like(W), torch.zeros_like(W), 0.0, 0.0
    dh, dh_err = torch.zeros_like(x), torch.zeros_like(x)
    for r in range(0, N, 650):
        X, k = x[r:r + 650], keep[r:r + 650].double()
        at = t[r:r + 650].clamp(min=0)
        rows = torch.arange(len(at), device="cuda")
        z = X @ W.t()
        wide = (d + 1) * U * (X.abs() @ W.abs().t()).amax(dim=1)
        lse = torch.logsumexp(z, dim=1)
        zt = z[rows, at]
        loss += float(((lse - zt) * k).sum()) / n
        loss_err += float(((2 * wide + 160 * U + 4 * U * (lse.abs() + zt.abs())) * k).sum()) / n
        P = torch.softmax(z, dim=1)
        dP = P * (2 * wide + 160 * U + 2 * U * lse.abs() + 2.1 * U)[:, None]
        P[rows, at] -= 1.0
        dP[rows, at] += U * P[rows, at].abs()
        P, dP = P * (k / n)[:, None], dP * (k / n)[:, None]
        A = P.abs() + dP
        dh[r:r + 650], dh_err[r:r + 650] = P @ W, dP @ W.abs() + (V + 8) * U * (A @ W.abs())
        dw += P.t() @ X
        dw_err += dP.t() @ X.abs() + (N + 8) * U * (A.t() @ X.abs())
    for panel in (0, 700):
        gh, gw = torch.empty_like(h), torch.empty_like(w)
        got = mir.shampoo_linear_xent(h, w, t, dhidden=gh, dweight=gw, panel_rows=panel)
        assert abs(got.item() - loss) <= loss_err + U * abs(loss)
        assert ((gh.double() - dh).abs() <= 1.01 * dh_err + U * dh.abs()).all()
        assert ((gw.double() - dw).abs() <= 1.01 * dw_err + U * dw.abs()).all()


@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
@pytest.mark.parametrize("N,d,V,panel", [(90, 64, 300, 0), (90, 64, 300, 32), (300, 33, 700, 0), (300, 33, 700, 100), (70, 2200, 257, 0)])
def test_ignored_rows_may_hold_anything(mir, dt, N, d, V, panel):
    """NaN and infinities in ignored rows (padding) reach no gradient and no
    loss: bit for bit what zeros there give.  The rows themselves stay as
    they were, and dhidden's are zero."""
    import torch
    h, w, t = make(N, d, V, dt, 14)
    t[5] = -100
    skip = t == -100
    got = []
    for fill in (0.0, float("nan"), float("inf"), -float("inf")):
        x = h.clone()
        x[skip] = fill
        before = x.clone()
        rs = torch.ones(N, device="cuda")
        rs[skip] = fill
        for kind in ((None, torch.float8_e4m3fn) if dt == "bfloat16" else (None,)):
            dh, dw = torch.full_like(h, 7.0), torch.full_like(w, 7.0)
            loss = mir.shampoo_linear_xent(x, w, t, dhidden=dh, dweight=dw, row_scale=rs, panel_rows=panel, logits_dtype=kind)
            assert torch.equal(x.view(torch.uint8), before.view(torch.uint8))
            assert not dh[skip].any()
            got.append((kind, loss, dh, dw))
    for kind, *r in got:
        first = next(g for g in got if g[0] == kind)[1:]
        assert all(torch.isfinite(a).all() and torch.equal(a, b) for a, b in zip(r, first))
