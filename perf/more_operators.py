"""Measured cases of the feed-forward layers' operators.

Three operators, each through the package's entry points where ``own`` is true
and as elementary torch operations where it is not:

* ``linear``: y = act(x W^T + bias) + residual and its gradients
  (``shampoo_linear``, ``shampoo_linear_grad``);
* ``gated``: y = (act(x Wg^T) * (x Wu^T)) Wd^T + residual and its gradients
  (``shampoo_gated_ffn``, ``shampoo_gated_ffn_grad``);
* activation checkpoints in 8 bits (``keep="e4m3"`` in either): what the
  forward pass keeps for the backward one (the pre-activations, and x for a
  weight's gradient) is held in 8 bits with power-of-two scales.

The gradients' cases take what the forward pass kept as their input, in the
type in which it was kept, as a training step's backward pass does.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
ACTIVATIONS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # serving: one token through the 1024-wide decoder's MLP-up layer
        dict(name="linear one token", op="linear", grad=False, M=1, K=1024, N=4096, dtype="bf16", act="gelu",
             bias=True, residual=False, keep="none"),
        # a small float32 layer, odd sizes, everything in the epilogue, the pre-activation kept
        dict(name="linear ragged f32", op="linear", grad=False, M=777, K=1000, N=2731, dtype="f32", act="gelu_tanh",
             bias=True, residual=True, keep="dtype"),
        # a training step's MLP-down layer of that decoder, its residual stream added
        dict(name="linear with residual", op="linear", grad=False, M=8192, K=4096, N=1024, dtype="bf16", act="none",
             bias=True, residual=True, keep="none"),
        # the MLP-up layer's gradients
        dict(name="linear gradients", op="linear", grad=True, M=8192, K=1024, N=4096, dtype="bf16", act="gelu",
             bias=True, residual=False, keep="dtype"),
        # a packed batch of odd length through the MLP-up layer, its pre-activation kept in 8 bits
        dict(name="linear kept in 8 bits", op="linear", grad=False, M=8191, K=1024, N=4096, dtype="bf16", act="gelu",
             bias=True, residual=False, keep="e4m3"),
        # its gradients from that and from an input kept in 8 bits
        dict(name="linear gradients from 8 bits", op="linear", grad=True, M=8191, K=1024, N=4096, dtype="bf16",
             act="gelu", bias=True, residual=False, keep="e4m3"),
        # serving: one token through a gated block of the same widths
        dict(name="gated one token", op="gated", grad=False, T=1, d=1024, f=4096, dtype="bf16", act="silu",
             residual=True, keep="none"),
        # a small batch of requests, odd widths
        dict(name="gated ragged", op="gated", grad=False, T=77, d=1000, f=2731, dtype="bf16", act="gelu_tanh",
             residual=True, keep="none"),
        # a float32 training step of a small block, odd sizes
        dict(name="gated gradients f32", op="gated", grad=True, T=999, d=1000, f=1371, dtype="f32", act="gelu",
             residual=False, keep="dtype"),
        # a training step's forward pass, both projections kept in 8 bits
        dict(name="gated kept in 8 bits", op="gated", grad=False, T=8192, d=1024, f=4096, dtype="bf16", act="silu",
             residual=True, keep="e4m3"),
        # a wide block's forward pass, both projections kept as they are
        dict(name="gated large", op="gated", grad=False, T=8192, d=4096, f=10240, dtype="bf16", act="silu",
             residual=True, keep="dtype"),
        # its gradients, from 8 bits
        dict(name="gated gradients large 8 bits", op="gated", grad=True, T=8192, d=4096, f=10240, dtype="bf16",
             act="silu", residual=False, keep="e4m3"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    grad = rng.random() < 0.5
    # a backward pass belongs to training: batches of tokens
    rows = _log(rng, 64, 16384) if grad else _log(rng, 1, 16384)
    dtype = rng.choice(["f32", "bf16", "bf16"])
    keep = rng.choice(["dtype", "e4m3"] if grad else ["none", "dtype", "e4m3"])
    if rng.random() < 0.5:
        return dict(op="linear", grad=grad, M=rows, K=_log(rng, 64, 4096), N=_log(rng, 64, 4096), dtype=dtype,
                    act=rng.choice(ACTIVATIONS), bias=rng.random() < 0.7, residual=not grad and rng.random() < 0.5,
                    keep=keep)
    return dict(op="gated", grad=grad, T=rows, d=_log(rng, 64, 2048), f=_log(rng, 64, 4096), dtype=dtype,
                act=rng.choice(ACTIVATIONS[1:]), residual=not grad and rng.random() < 0.5, keep=keep)


def _up(x, m):
    return -(-x // m) * m


def work(case):
    c = case
    size = 4 if c["dtype"] == "f32" else 2

    def held(rows, cols, block=32):
        if c["keep"] == "none":
            return 0
        return rows * cols * size if c["keep"] == "dtype" else rows * (_up(cols, block) + _up(cols, block) // block)

    if c["op"] == "linear":
        M, K, N = c["M"], c["K"], c["N"]
        bias = 4 * N if c["bias"] else 0
        if not c["grad"]:
            return {"bytes": (M * K + N * K + M * N * (2 if c["residual"] else 1)) * size + bias + held(M, N),
                    "flops": 2 * M * K * N}
        x = held(M, K, 128)
        z = held(M, N) if c["act"] != "none" else 0
        return {"bytes": (M * N + 2 * N * K + M * K) * size + x + z + bias, "flops": 4 * M * K * N}
    T, d, f = c["T"], c["d"], c["f"]
    if not c["grad"]:
        return {"bytes": (T * d * (3 if c["residual"] else 2) + 3 * d * f) * size + 2 * held(T, f), "flops": 6 * T * d * f}
    return {"bytes": (2 * T * d + 6 * d * f) * size + held(T, d, 128) + 2 * held(T, f), "flops": 12 * T * d * f}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _values(gen, shape, spread):
    """Normal values whose rows differ in size, with a few large entries, as activations have."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= torch.exp(spread * torch.randn(shape[:-1] + (1,), generator=gen, device="cuda"))
    x *= 1.0 + 7.0 * (torch.rand(shape, generator=gen, device="cuda") < 1e-3)
    return x


def _blocks(x, block):
    """x [rows, cols] float32 -> (e4m3 values, power-of-two scales) for each ``block`` columns of a row."""
    rows, cols = x.shape
    p = torch.zeros((rows, _up(cols, block)), device=x.device)
    p[:, :cols] = x
    p = p.view(rows, -1, block)
    size = p.abs()
    amax = torch.where(torch.isfinite(size), size, torch.zeros_like(size)).amax(dim=2)
    frac, e = torch.frexp(amax)
    e = e - 9 + (frac > 0.875).to(e.dtype)  # the least e with amax <= 448 * 2^e
    e = torch.where(amax > 0, e.clamp(-127, 127), torch.zeros_like(e))
    inverse = ((127 - e) << 23).to(torch.int32).view(torch.float32)  # 2^-e from its exponent's bits
    q = (p * inverse[:, :, None]).to(torch.float8_e4m3fn).view(rows, -1)
    return q, (e + 127).to(torch.uint8)


def _held(x, keep, dt, block=32):
    """x as the forward pass keeps it."""
    if keep == "dtype":
        return x.to(dt)
    q, s = _blocks(x, block)
    if block == 128:  # the rows' scales in fours
        full = torch.full((s.shape[0], _up(s.shape[1], 4)), 127, dtype=torch.uint8, device=x.device)
        full[:, :s.shape[1]] = s
        s = full
    return q, s.view(torch.float8_e8m0fnu)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    dt = DTYPES[c["dtype"]]

    def normal(rows, cols, size):
        return (torch.randn((rows, cols), generator=gen, device="cuda") * size).to(dt)

    if c["op"] == "linear":
        M, K, N = c["M"], c["K"], c["N"]
        s = {"case": c, "w": normal(N, K, 1.2 / math.sqrt(K)),
             "bias": 0.3 * torch.randn(N, generator=gen, device="cuda") if c["bias"] else None}
        x = _values(gen, (M, K), 0.3)
        if not c["grad"]:
            s["x"] = x.to(dt)
            s["residual"] = _values(gen, (M, N), 0.3).to(dt) if c["residual"] else None
            s["y"] = torch.empty((M, N), dtype=dt, device="cuda")
            s["keep"] = _room(M, N, c["keep"], dt)
            return s
        s["x"] = _held(x, c["keep"], dt, 128)
        s["kept"] = _held(_values(gen, (M, N), 0.3), c["keep"], dt) if c["act"] != "none" else None
        s["dy"] = (_values(gen, (M, N), 1.0) * 1e-3).to(dt)
        s["dx"], s["dw"] = torch.empty((M, K), dtype=dt, device="cuda"), torch.empty((N, K), dtype=dt, device="cuda")
        s["dbias"] = torch.empty(N, device="cuda") if c["bias"] else None
        return s
    T, d, f = c["T"], c["d"], c["f"]
    s = {"case": c, "wg": normal(f, d, 1.2 / math.sqrt(d)), "wu": normal(f, d, 1.0 / math.sqrt(d)),
         "wd": normal(d, f, 1.0 / math.sqrt(f))}
    x = _values(gen, (T, d), 0.3)
    if not c["grad"]:
        s["x"] = x.to(dt)
        s["residual"] = _values(gen, (T, d), 0.3).to(dt) if c["residual"] else None
        s["y"] = torch.empty((T, d), dtype=dt, device="cuda")
        s["keep"] = None if c["keep"] == "none" else (_room(T, f, c["keep"], dt), _room(T, f, c["keep"], dt))
        return s
    s["x"] = _held(x, c["keep"], dt, 128)
    s["kept"] = (_held(1.2 * _values(gen, (T, f), 0.3), c["keep"], dt), _held(_values(gen, (T, f), 0.3), c["keep"], dt))
    s["dy"] = (_values(gen, (T, d), 1.0) * 1e-3).to(dt)
    s["dx"] = torch.empty((T, d), dtype=dt, device="cuda")
    for name, like in (("dwg", "wg"), ("dwu", "wu"), ("dwd", "wd")):
        s[name] = torch.empty_like(s[like])
    return s


def _room(rows, cols, keep, dt):
    """Tensors that receive what a forward pass keeps."""
    if keep == "none":
        return None
    if keep == "dtype":
        return torch.empty((rows, cols), dtype=dt, device="cuda")
    wide = _up(cols, 32)
    return (torch.empty((rows, wide), dtype=torch.float8_e4m3fn, device="cuda"),
            torch.empty((rows, wide // 32), dtype=torch.float8_e8m0fnu, device="cuda"))


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------
def _wide(t, cols, block=32):
    """The values that a kept matrix stands for, float32."""
    if isinstance(t, torch.Tensor):
        return t.float()
    q, s = t
    rows, held = q.shape
    return (q.float().view(rows, held // block, block) * s.float()[:, :held // block, None]).view(rows, held)[:, :cols]


def plain_act(z, act, derivative=False):
    """act(z), or (act(z), act'(z))."""
    one = torch.ones_like(z)
    if act == "none":
        return (z, one) if derivative else z
    if act == "relu":
        on = torch.where(z > 0, one, torch.zeros_like(z))
        return (z * on, on) if derivative else z * on
    if act == "gelu":
        # Phi(z) from erfc, which keeps its digits in the lower tail
        p = 0.5 * torch.special.erfc(z * -math.sqrt(0.5))
        if not derivative:
            return z * p
        return z * p, p + z * torch.exp(-0.5 * z * z) * (1.0 / math.sqrt(2.0 * math.pi))
    if act == "gelu_tanh":
        k = 2.0 * math.sqrt(2.0 / math.pi)
        s = 1.0 / (1.0 + torch.exp(-k * (z + 0.044715 * z * z * z)))
        if not derivative:
            return z * s
        return z * s, s + z * s * (1.0 - s) * (k * (1.0 + 3 * 0.044715 * z * z))
    s = 1.0 / (1.0 + torch.exp(-z))
    return (z * s, s + z * s * (1.0 - s)) if derivative else z * s


def plain_linear(x, w, bias, act, residual, keep, dt):
    z = x.float() @ w.float().t()
    if bias is not None:
        z = z + bias.float()
    y = plain_act(z, act)
    if residual is not None:
        y = y + residual.float()
    return (y.to(dt),) if keep == "none" else (y.to(dt), _held(z, keep, dt))


def plain_linear_grad(dy, x, w, kept, act, want_bias, dt):
    dz = dy.float()
    if act != "none":
        dz = dz * plain_act(_wide(kept, dy.shape[1]), act, True)[1]
    dx = dz @ w.float()
    dw = dz.t() @ _wide(x, w.shape[1], 128)
    return (dx.to(dt), dw.to(dt)) + ((dz.sum(dim=0),) if want_bias else ())


def plain_gated(x, wg, wu, wd, act, residual, keep, dt):
    x = x.float()
    g, u = x @ wg.float().t(), x @ wu.float().t()
    y = (plain_act(g, act) * u) @ wd.float().t()
    if residual is not None:
        y = y + residual.float()
    return (y.to(dt),) if keep == "none" else (y.to(dt), (_held(g, keep, dt), _held(u, keep, dt)))


def plain_gated_grad(dy, x, wg, wu, wd, kept, act, dt):
    T, f = dy.shape[0], wg.shape[0]
    g, u = _wide(kept[0], f), _wide(kept[1], f)
    a, da = plain_act(g, act, True)
    dy, x = dy.float(), _wide(x, wg.shape[1], 128)
    dh = dy @ wd.float()
    dg, du = dh * u * da, dh * a
    del dh, da
    dx = dg @ wg.float() + du @ wu.float()
    return dx.to(dt), (dg.t() @ x).to(dt), (du.t() @ x).to(dt), (dy.t() @ (a * u)).to(dt)


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(state):
    s, c = state, state["case"]
    if own:
        import matrix_inverse_roots_amd as mir
    dt, act = s["w" if c["op"] == "linear" else "wg"].dtype, c["act"]
    if c["op"] == "linear" and not c["grad"]:
        if not own:
            return plain_linear(s["x"], s["w"], s["bias"], act, s["residual"], c["keep"], dt)
        y = mir.shampoo_linear(s["x"], s["w"], s["y"], bias=s["bias"], activation=act, residual=s["residual"], keep=s["keep"])
        return (y,) if s["keep"] is None else (y, s["keep"])
    if c["op"] == "linear":
        if not own:
            return plain_linear_grad(s["dy"], s["x"], s["w"], s["kept"], act, s["dbias"] is not None, dt)
        mir.shampoo_linear_grad(s["dy"], s["x"], s["w"], kept=s["kept"], activation=act, dx=s["dx"], dw=s["dw"], dbias=s["dbias"])
        return (s["dx"], s["dw"]) + ((s["dbias"],) if s["dbias"] is not None else ())
    if not c["grad"]:
        if not own:
            return plain_gated(s["x"], s["wg"], s["wu"], s["wd"], act, s["residual"], c["keep"], dt)
        y = mir.shampoo_gated_ffn(s["x"], s["wg"], s["wu"], s["wd"], s["y"], activation=act, residual=s["residual"], keep=s["keep"])
        return (y,) if s["keep"] is None else (y, s["keep"])
    if not own:
        return plain_gated_grad(s["dy"], s["x"], s["wg"], s["wu"], s["wd"], s["kept"], act, dt)
    mir.shampoo_gated_ffn_grad(s["dy"], s["x"], s["wg"], s["wu"], s["wd"], s["kept"], activation=act, dx=s["dx"],
                               dw_gate=s["dwg"], dw_up=s["dwu"], dw_down=s["dwd"])
    return s["dx"], s["dwg"], s["dwu"], s["dwd"]


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------
def _kept64(z, keep):
    """z where it is kept as it is.  Codes of 8 bits have no value of their own
    here: on which side of a rounding border (for a scale: of a power of two)
    one lands is decided by the last bit of the sum before it."""
    return z if keep == "dtype" else None


def _stand64(t, cols, block=32):
    if torch.is_tensor(t):
        return t.double()
    values, scales = t[0].double(), t[1].double()
    return (values * scales.repeat_interleave(block, 1)[:, :values.shape[1]])[:, :cols]


def _act64(z, act):
    """(act(z), act'(z)) in float64."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp(min=0), (z > 0).double()
    if act == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        r = math.sqrt(2 / math.pi)
        t = torch.tanh(r * (z + 0.044715 * z ** 3))
        # 1 + t through the logistic function, which keeps its digits where t is near -1
        half = torch.sigmoid(2 * r * (z + 0.044715 * z ** 3))
        return z * half, half + 0.5 * z * (1 - t * t) * r * (1 + 3 * 0.044715 * z * z)
    half = torch.sigmoid(z)
    return z * half, half * (1 + z * (1 - half))


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "linear":
        w = s["w"].double()
        if c["grad"]:
            dz = s["dy"].double()
            if c["act"] != "none":
                dz = dz * _act64(_stand64(s["kept"], c["N"]), c["act"])[1]
            got = dz @ w, dz.t() @ _stand64(s["x"], c["K"], 128)
            return got + ((dz.sum(dim=0),) if c["bias"] else ())
        z = torch.matmul(s["x"].double(), w.t())
        if c["bias"]:
            z = z + s["bias"].double()
        y = _act64(z, c["act"])[0]
        if c["residual"]:
            y = y + s["residual"].double()
        return (y,) if c["keep"] == "none" else (y, _kept64(z, c["keep"]))
    wg, wu, wd = s["wg"].double(), s["wu"].double(), s["wd"].double()
    if not c["grad"]:
        x = s["x"].double()
        g, u = torch.matmul(x, wg.t()), torch.matmul(x, wu.t())
        y = torch.matmul(_act64(g, c["act"])[0] * u, wd.t())
        if c["residual"]:
            y = y + s["residual"].double()
        return (y,) if c["keep"] == "none" else (y, (_kept64(g, c["keep"]), _kept64(u, c["keep"])))
    x, dy = _stand64(s["x"], c["d"], 128), s["dy"].double()
    g, u = (_stand64(t, c["f"]) for t in s["kept"])
    a, slope = _act64(g, c["act"])
    dwd = dy.t() @ (a * u)
    dh = dy @ wd
    du = dh * a
    dg = dh.mul_(u).mul_(slope)
    return torch.matmul(torch.cat((dg, du), dim=1), torch.cat((wg, wu))), dg.t() @ x, du.t() @ x, dwd
