"""The projection's loss where a row's target has a probability near one.

The loss is log(1 + sum over v != t of exp(z_v - z_t)).  If every logit that
enters it carries an error of at most dz, the same error wherever that logit
is used, then its slope with respect to a logit is that column's probability
and the loss is off by at most (1 - p_t) 2 dz e^(4 dz): next to nothing for a
confident row, however large its logits.  To that come the sum's and the
logarithm's own roundings (`own` below).  A target's logit summed a second
time, in another order, would add 2 dz as it is.
"""

import numpy as np
import pytest

import f8_reference as ref
from helpers import log

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


@pytest.fixture(scope="module")
def mir():
    import matrix_inverse_roots_amd as m
    return m


def make(N, d, V, dt, seed, level=1000.0):
    """Logits around `level` (a part that all columns share), the target ahead by 10 to 20."""
    import torch
    g = np.random.default_rng(seed)
    h = d // 2
    w = np.empty((V, d))
    w[:, :h] = g.uniform(1.0, 2.0, h)
    w[:, h:] = g.standard_normal((V, d - h)) * 0.5
    t = g.integers(0, V, N)
    x = np.empty((N, d))
    x[:, :h] = g.uniform(0.5, 1.5, (N, h)) * level / (1.5 * h)
    own = w[t, h:]
    x[:, h:] = own * (g.uniform(10.0, 20.0, (N, 1)) / (own * own).sum(axis=1, keepdims=True))
    dtype = getattr(torch, dt)
    return (torch.from_numpy(x).float().to(dtype).cuda(), torch.from_numpy(w).float().to(dtype).cuda(),
            torch.from_numpy(t).cuda())


def definition(X, W, t, drop=0.0):
    """(loss, its bound, probabilities, what their own logarithms may be off by) in float64."""
    N, d = X.shape
    z = X @ W.T
    dz = ((drop + (d + 1) * U) * (np.abs(X) @ np.abs(W).T)).max(axis=1)
    rows = np.arange(N)
    apart = np.exp(z - z[rows, t][:, None])
    apart[rows, t] = 0.0
    others = apart.sum(axis=1)
    loss = np.log1p(others)
    away = others / (1.0 + others)
    # a sum of 64 terms by a lane and of 13 by steps of the tree, each addition
    # off by half a step of a sum that may reach twice 1 + others; exp and log
    # off by a few units
    few = 160 * U
    own = few * others + 80 * U * (1.0 + others) / 2 + 4 * U * loss
    return loss, 2 * dz * away * np.exp(4 * dz) + own, apart / (1.0 + others)[:, None], 2 * dz + few


CASES = [(1, 64, 300), (40, 64, 2000), (300, 128, 129), (5, 1000, 20001)]


@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
@pytest.mark.parametrize("N,d,V", CASES)
def test_loss_of_confident_rows(mir, N, d, V, dt):
    import torch
    h, w, t = make(N, d, V, dt, N + d)
    loss = mir.shampoo_linear_xent(h, w, t, reduction="none")
    want, bound, _, _ = definition(h.double().cpu().numpy(), w.double().cpu().numpy(), t.cpu().numpy())
    got = loss.double().cpu().numpy()
    log(f"N {N} d {d} V {V} {dt}: losses {want.min():.1e} to {want.max():.1e}, off by {np.abs(got - want).max():.1e}")
    assert (got >= 0).all()
    assert (np.abs(got - want) <= bound).all(), float((np.abs(got - want) / bound).max())
    dh, dw = torch.empty_like(h), torch.empty_like(w)
    assert torch.equal(mir.shampoo_linear_xent(h, w, t, reduction="none", dhidden=dh, dweight=dw), loss)


@pytest.mark.parametrize("wdt", ["float32", "bfloat16"])
@pytest.mark.parametrize("N,d,V", CASES)
def test_loss_of_confident_rows_with_8_bit_logits(mir, N, d, V, wdt):
    """The logits' error is the matrix instructions': 2^-13 of |x| |w| on the
    quantised operands, the target's logit included in it."""
    import torch
    h, w, t = make(N, d, V, "bfloat16", N + d, level=100.0)
    w = w.float() * 1.001 if wdt == "float32" else w
    values = []
    for m in (h, w):
        q, s = mir.shampoo_quantize_f8(m)
        values.append(ref.stand_for(ref.code_values("e4m3")[q.view(torch.uint8).cpu().numpy()], s.view(torch.uint8).cpu().numpy(), 1))
    # one operand's roundings may cost the target its lead: confident rows only
    want, bound, _, _ = definition(*values, t.cpu().numpy(), drop=2.0 ** -13)
    sure = want < 0.1
    assert sure.any()
    got = mir.shampoo_linear_xent(h, w, t, reduction="none", logits_dtype=torch.float8_e4m3fn).double().cpu().numpy()
    assert (got >= 0).all()
    assert (np.abs(got - want) <= bound)[sure].all(), float((np.abs(got - want) / bound)[sure].max())


@pytest.mark.parametrize("kind", ["float32", "bfloat16", "8-bit"])
@pytest.mark.parametrize("N,V", [(1280, 13312), (2048, 32768)])
def test_every_target_is_found_over_many_tiles(mir, N, V, kind):
    """Several tiles for each workgroup, small and large ones, of one to two
    stages of k each: every row's own target, a few of them in each tile."""
    import torch
    d = 64
    h, w, t = make(N, d, V, "float32" if kind == "float32" else "bfloat16", N, level=100.0)
    X, W = h.double().cpu().numpy(), w.double().cpu().numpy()
    if kind == "8-bit":
        X, W = (ref.stand_for(ref.code_values("e4m3")[q.view(torch.uint8).cpu().numpy()], s.view(torch.uint8).cpu().numpy(), 1)
                for q, s in (mir.shampoo_quantize_f8(m) for m in (h, w)))
    got = mir.shampoo_linear_xent(h, w, t, reduction="none", logits_dtype=torch.float8_e4m3fn if kind == "8-bit" else None)
    want, bound, _, _ = definition(X, W, t.cpu().numpy(), drop=2.0 ** -13 if kind == "8-bit" else 0.0)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (got >= 0).all() and (err <= bound).all(), float((err / bound).max())


@pytest.mark.parametrize("logits", ["own", "8-bit"])
@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
def test_a_vocabulary_of_one(mir, dt, logits):
    """Its only column has probability one: no loss and no gradient, exactly."""
    import torch
    if logits == "8-bit" and dt == "float32":
        return
    g = np.random.default_rng(3)
    h, w = (torch.from_numpy(g.standard_normal((n, 333)) * 7).float().to(getattr(torch, dt)).cuda() for n in (150, 1))
    t = torch.zeros(150, dtype=torch.int64, device="cuda")
    dh, dw = torch.full_like(h, 5.0), torch.full_like(w, 5.0)
    loss = mir.shampoo_linear_xent(h, w, t, reduction="none", dhidden=dh, dweight=dw,
                                   logits_dtype=torch.float8_e4m3fn if logits == "8-bit" else None)
    assert not loss.any() and not dh.any() and not dw.any()


@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
def test_gradient_of_confident_rows(mir, dt):
    """dhidden, whose shared part cancels in the definition: each probability
    off by 2 dz and a few units relative to itself (bfloat16: and two roundings),
    the target's by as much relative to what the others sum to, and by its
    loss's own error, which is what it is made from."""
    import torch
    N, d, V = 60, 64, 1500
    h, w, t = make(N, d, V, dt, 11)
    dh = torch.empty_like(h)
    mir.shampoo_linear_xent(h, w, t, reduction="none", dhidden=dh)
    X, W, T = h.double().cpu().numpy(), w.double().cpu().numpy(), t.cpu().numpy()
    loss, bound, P, rel = definition(X, W, T)
    half = 2.0 ** -8 if dt == "bfloat16" else U
    dP = P * (rel * np.exp(2 * rel) + 2.1 * half)[:, None]
    rows = np.arange(N)
    P[rows, T] = -P.sum(axis=1)
    dP[rows, T] = bound + (half + 4 * U) * np.abs(P[rows, T])
    want = P @ W
    err = dP @ np.abs(W) + (V + 8) * U * ((np.abs(P) + dP) @ np.abs(W)) + torch.finfo(h.dtype).eps / 2 * np.abs(want)
    got = dh.double().cpu().numpy()
    log(f"{dt}: gradient off by {np.linalg.norm(got - want) / np.linalg.norm(want):.1e}")
    assert (np.abs(got - want) <= 1.01 * err).all(), float((np.abs(got - want) / err).max())


@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
def test_large_logits_lose_nothing_in_the_softmax(mir, dt):
    """Logits 4096 + k / 4 are exact in every order of summation, so the
    gradient is off by the softmax's own roundings alone (exp of differences
    up to 130 and a few units: 160 U) and those of the products and results."""
    import torch
    N, V = 50, 700
    g = np.random.default_rng(2)
    x = np.stack([np.full(N, 4096.0), np.ones(N)], axis=1)
    w = np.stack([np.ones(V), g.integers(0, 32, V) / 4.0], axis=1)
    t = g.integers(0, V, N)
    dtype = getattr(torch, dt)
    h, W = (torch.from_numpy(a).float().to(dtype).cuda() for a in (x, w))
    dh = torch.empty_like(h)
    loss = mir.shampoo_linear_xent(h, W, torch.from_numpy(t).cuda(), reduction="none", dhidden=dh)
    z = x @ w.T
    p = np.exp(z - z.max(axis=1, keepdims=True))
    p /= p.sum(axis=1, keepdims=True)
    want = -np.log(p[np.arange(N), t])
    assert (np.abs(loss.double().cpu().numpy() - want) <= 160 * U + 4 * U * want).all()
    half = 2.0 ** -8 if dt == "bfloat16" else U
    dP = p * (160 * U + 2.1 * half)
    p[np.arange(N), t] -= 1.0
    dP[np.arange(N), t] = (160 * U + half) * np.abs(p[np.arange(N), t])
    # the second column of dhidden: the first sums to zero
    want = p @ w[:, 1]
    err = dP @ w[:, 1] + (V + 8) * U * ((np.abs(p) + dP) @ w[:, 1]) + torch.finfo(dtype).eps / 2 * np.abs(want)
    assert (np.abs(dh.double().cpu().numpy()[:, 1] - want) <= 1.01 * err).all()
