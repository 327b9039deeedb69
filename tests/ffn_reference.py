"""The feed-forward layers' definitions in float64 (torch, no code of the
package), and bounds on what float32 evaluation may be off by."""

import math

import torch

U = 2.0 ** -23                       # a float32 addition, whichever way it is rounded
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float8_e4m3fn: 2.0 ** -4}
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
STEEPEST = 1.13                      # |act'| of the steepest of them


def cdf(z):
    """Phi(z) through the scaled complementary error function: a device's ndtr
    loses its lower tail's digits (2e-2 at z = -8)."""
    low = 0.5 * torch.special.erfcx(z.abs() * math.sqrt(0.5)) * torch.exp(-z * z / 2)
    return torch.where(z < 0, low, 1 - low)


def act(z, kind):
    """(act(z), act'(z))."""
    if kind in (None, "none"):
        return z, torch.ones_like(z)
    if kind == "relu":
        return z.clamp(min=0), (z > 0).double()
    if kind == "gelu":
        p = cdf(z)
        return z * p, p + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    k = 2 * math.sqrt(2 / math.pi)
    p, dp = (k * (z + 0.044715 * z ** 3), k * (1 + 3 * 0.044715 * z * z)) if kind == "gelu_tanh" else (z, torch.ones_like(z))
    s = torch.sigmoid(p)
    return z * s, s + z * s * torch.sigmoid(-p) * dp


def act_off(z, kind):
    """How far float32 evaluation of act(z) and act'(z) may be off: the
    exponentials' arguments, z^2 / 2 or p(z), are rounded a few times (each
    2^-24 relative), the fitted polynomial is 3.6e-7 off, the rest is a dozen
    roundings.  act' also loses what 1 - sigma does where sigma is near one."""
    if kind in (None, "none", "relu"):
        return torch.zeros_like(z), torch.zeros_like(z)
    rel = (8 + z * z + (0.0714 * z.abs() ** 3 if kind == "gelu_tanh" else 0) + 2 * z.abs()) * 2.0 ** -22
    a, d = act(z, kind)
    if kind == "gelu":
        p = cdf(z)
        spread = p + z.abs() * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    else:
        k = 2 * math.sqrt(2 / math.pi)
        p, dp = (k * (z + 0.044715 * z ** 3), k * (1 + 3 * 0.044715 * z * z)) if kind == "gelu_tanh" else (z, torch.ones_like(z))
        s = torch.sigmoid(p)
        spread = s + z.abs() * s * dp * (torch.sigmoid(-p) + 2.0 ** -22)
    return rel * a.abs() + 1e-36, rel * spread + 1e-36


def two(e):
    """2^e (float64) for whole e, from its bits: a device's pow may be off in the last one."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def blocks(x, block):
    """x [rows, cols] in float32 -> (e4m3 values as float32, scale bytes) per ``block`` columns of a row, exactly."""
    rows, cols = x.shape
    wide = -(-cols // block) * block
    p = torch.zeros((rows, wide), dtype=torch.float64, device=x.device)
    p[:, :cols] = x.double()
    p = p.view(rows, -1, block)
    size = torch.where(torch.isfinite(p), p.abs(), torch.zeros_like(p)).amax(dim=2)
    e = torch.zeros_like(size)
    on = size > 0
    e[on] = torch.ceil(torch.log2(size[on] / 448.0))
    e = torch.where(on & (size <= 448.0 * two(e - 1)), e - 1, e)
    e = torch.where(on & (size > 448.0 * two(e)), e + 1, e).clamp(-127, 127)
    v = p / two(e)[:, :, None]
    a = v.abs()
    low = torch.floor(torch.log2(torch.where(a > 0, a, torch.ones_like(a)))).clamp(min=-6)
    step = two(low - 3)
    q = torch.where(torch.isfinite(v), torch.round(v / step) * step, torch.full_like(v, float("nan")))
    return q.reshape(rows, wide).float(), (e + 127).to(torch.uint8)


def stand(q, s, cols, block):
    """What 8-bit values and scales stand for, float64 [rows, cols]."""
    rows, wide = q.shape
    e = s.view(torch.uint8).double()[:, :wide // block] - 127
    return (q.double().view(rows, -1, block) * two(e)[:, :, None]).view(rows, wide)[:, :cols]


def widen(kept, cols, block=32):
    return kept.double() if isinstance(kept, torch.Tensor) else stand(kept[0], kept[1], cols, block)


def check(got, want, err, what):
    """|got - want| <= err, element by element; NaN and infinities in the same places."""
    got, want = got.double(), want.double()
    odd = ~torch.isfinite(want)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what + ": NaN in other places"
    if bool(odd.any()):
        assert torch.equal(torch.nan_to_num(got[odd], nan=0.0), torch.nan_to_num(want[odd], nan=0.0)), what
    far = torch.where(odd, torch.zeros_like(want), (got - want).abs() - err)
    if far.numel() and float(far.max()) > 0:
        at = int(far.reshape(-1).argmax())
        raise AssertionError("%s: %.9g for %.9g, allowed %.3g, at %d of %s" % (
            what, got.reshape(-1)[at], want.reshape(-1)[at], err.reshape(-1)[at] if err.numel() > 1 else float(err), at, tuple(want.shape)))


def linear(x, w, bias, kind, residual):
    """(z, y, and how far float32 sums may be off in each), float64; x, w as the products read them."""
    x, w = x.double(), w.double()
    z, size = x @ w.t(), x.abs() @ w.abs().t()
    if bias is not None:
        z, size = z + bias.double(), size + bias.double().abs()
    dz = (x.shape[1] + 2) * U * size
    y = act(z, kind)[0]
    dy = STEEPEST * dz + act_off(z, kind)[0]
    if residual is not None:
        y = y + residual.double()
        dy = dy + U * (y.abs() + residual.double().abs())
    return z, dz, y, dy


def linear_grad(dy, x, w, z, kind, half):
    """{name: (gradient, allowed)}; ``half``: the rounding of dz between its products (0: none), and of what is stored."""
    dy, x, w = dy.double(), x.double(), w.double()
    if kind in (None, "none"):
        dz, off = dy, torch.zeros_like(dy)
    else:
        dz = dy * act(z, kind)[1]
        off = dy.abs() * act_off(z, kind)[1] + 2 * U * dz.abs()
    rounded = off + (0 if kind in (None, "none") else half) * (dz.abs() + off)
    M, N = dy.shape

    def product(a, da, b):
        return a @ b, 1.01 * da @ b.abs() + (a.shape[1] + 2) * U * ((a.abs() + da) @ b.abs())

    return {"dx": product(dz, rounded, w), "dw": product(dz.t(), rounded.t(), x),
            "dbias": (dz.sum(dim=0), (off + (M + 2) * U * dz.abs()).sum(dim=0))}


def gated(x, wg, wu, wd, kind, residual, half):
    """((g, dg), (u, du), (y, dy)): values and how far each may be off; ``half``: the rounding of h."""
    x, wg, wu, wd = (t.double() for t in (x, wg, wu, wd))
    g, u = x @ wg.t(), x @ wu.t()
    dg, du = ((x.shape[1] + 2) * U * (x.abs() @ t.abs().t()) for t in (wg, wu))
    a = act(g, kind)[0]
    da = STEEPEST * dg + act_off(g, kind)[0]
    h = a * u
    dh = da * u.abs() + (a.abs() + da) * du + U * h.abs()
    dh = dh + half * (h.abs() + dh)
    y = h @ wd.t()
    dy = 1.01 * dh @ wd.abs().t() + (wd.shape[1] + 2) * U * ((h.abs() + dh) @ wd.abs().t())
    if residual is not None:
        y = y + residual.double()
        dy = dy + U * (y.abs() + residual.double().abs())
    return (g, dg), (u, du), (y, dy)


def gated_grad(dy, x, wg, wu, wd, g, u, kind, half):
    """{name: (gradient, allowed)}; ``half``: the rounding of h, dg and du between the products."""
    dy, x, wg, wu, wd = (t.double() for t in (dy, x, wg, wu, wd))
    a, s = act(g, kind)
    da, ds = act_off(g, kind)
    dh = dy @ wd
    e = (dy.shape[1] + 2) * U * (dy.abs() @ wd.abs())
    h, dg, du = a * u, dh * u * s, dh * a
    oh = da * u.abs() + U * h.abs()
    og = e * (u * s).abs() + (dh.abs() + e) * u.abs() * ds + 3 * U * dg.abs()
    ou = e * a.abs() + (dh.abs() + e) * da + 2 * U * du.abs()
    oh, og, ou = (o + half * (v.abs() + o) for o, v in ((oh, h), (og, dg), (ou, du)))

    def product(p, dp, b):
        return p @ b, 1.01 * dp @ b.abs() + (p.shape[1] + 2) * U * ((p.abs() + dp) @ b.abs())

    both, off = torch.cat((dg, du), 1), torch.cat((og, ou), 1)
    d = {"dx": product(both, off, torch.cat((wg, wu))), "dw_gate": product(dg.t(), og.t(), x), "dw_up": product(du.t(), ou.t(), x)}
    want, err = product(h.t(), oh.t(), dy)
    d["dw_down"] = want.t(), err.t()
    return d
