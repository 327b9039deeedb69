"""Measured cases of the 8-bit block-scaled product and of the projection loss.

Four operators, each through the package's entry points where ``own`` is true
and as elementary torch operations where it is not:

* ``quantize``: a matrix (or its transpose, or both in one call) to 8-bit
  floating point with a power-of-two scale for each block of 128
  (``shampoo_quantize_f8``);
* ``product``: C = A B^T of two such matrices (``shampoo_matmul_f8``);
* ``linear``: a linear layer's forward and both gradients on those two;
* ``xent``: softmax cross entropy of hidden @ weight^T against target rows,
  the loss alone or with the gradients of both (``shampoo_linear_xent``).
"""

import math

import torch

own = False

FORMATS = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}


# ----------------------------------------------------------------------------
# cases
# ----------------------------------------------------------------------------
def listed():
    return [
        # one token's activations on their way into a product: launch latency
        dict(name="quantize one token", op="quantize", n=1, rows=1, cols=1024, dtype="bf16", fmt="e4m3",
             block_rows=1, transpose=False),
        # a training batch's activations, a scale for each row and 128 columns
        dict(name="quantize activations", op="quantize", n=1, rows=8192, cols=4096, dtype="bf16", fmt="e4m3",
             block_rows=1, transpose=False),
        # a projection's float32 master weight with an odd vocabulary, 128 x 128 blocks
        dict(name="quantize weight blocks", op="quantize", n=1, rows=50001, cols=1024, dtype="f32", fmt="e4m3",
             block_rows=128, transpose=False),
        # output gradients for the weight's gradient: blocks along the tokens, transposed, the wide-range format
        dict(name="quantize gradients transposed", op="quantize", n=1, rows=8191, cols=4096, dtype="bf16", fmt="e5m2",
             block_rows=1, transpose=True),
        # serving: one token through a layer of the 1024-wide decoder
        dict(name="product one token", op="product", n=1, M=1, N=4096, K=1024, a_fmt="e4m3", b_fmt="e4m3",
             b_rows=128, out="bf16"),
        # a ragged batch against odd sizes
        dict(name="product ragged", op="product", n=1, M=777, N=1000, K=4200, a_fmt="e4m3", b_fmt="e4m3",
             b_rows=1, out="f16"),
        # the preconditioning product of a stack of 1024-blocks
        dict(name="product stack", op="product", n=144, M=1024, N=1024, K=1024, a_fmt="e4m3", b_fmt="e4m3",
             b_rows=1, out="f32"),
        # a wide layer over a long batch
        dict(name="product large", op="product", n=1, M=16384, N=8192, K=8192, a_fmt="e4m3", b_fmt="e4m3",
             b_rows=128, out="bf16"),
        # a training step of the decoder's MLP-up layer: three products and the quantisations they need
        dict(name="linear training", op="linear", tokens=8192, K=1024, N=4096, dtype="bf16"),
        # the loss of one token (scoring while serving), the whole vocabulary
        dict(name="loss one token", op="xent", N=1, d=1024, V=32768, dtype="bf16", grads=False, reduction="none"),
        # a float32 training step of a small projection with odd sizes, rows without a target among them
        dict(name="loss and gradients f32", op="xent", N=999, d=1024, V=10007, dtype="f32", grads=True,
             reduction="mean"),
        # a training step of a large projection
        dict(name="loss and gradients large", op="xent", N=8192, d=4096, V=131072, dtype="bf16", grads=True,
             reduction="mean"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "linear", "xent", "xent"])
    if op == "quantize":
        return dict(op=op, n=rng.choice([1, 1, 3]), rows=_log(rng, 1, 16384), cols=_log(rng, 64, 8192),
                    dtype=rng.choice(["f32", "bf16", "f16"]), fmt=rng.choice(["e4m3", "e5m2"]),
                    block_rows=rng.choice([1, 128]), transpose=rng.random() < 0.5)
    if op == "product":
        n = rng.choice([1, 1, 1, 5])
        return dict(op=op, n=n, M=_log(rng, 1, 8192), N=_log(rng, 64, 8192), K=_log(rng, 64, 8192),
                    a_fmt=rng.choice(["e4m3", "e4m3", "e5m2"]), b_fmt=rng.choice(["e4m3", "e4m3", "e5m2"]),
                    b_rows=rng.choice([1, 128]), out=rng.choice(["f32", "bf16", "f16"]))
    if op == "linear":
        return dict(op=op, tokens=_log(rng, 64, 16384), K=_log(rng, 128, 4096), N=_log(rng, 128, 4096), dtype="bf16")
    dtype = rng.choice(["f32", "bf16", "bf16"])
    return dict(op=op, N=_log(rng, 1, 4096), d=_log(rng, 64, 2048), V=_log(rng, 500, 65536 if dtype == "f32" else 131072),
                dtype=dtype, grads=rng.random() < 0.6, reduction=rng.choice(["mean", "sum", "none"]))


def _up(x, m):
    return -(-x // m) * m


def work(case):
    c = case
    size = {"f32": 4, "bf16": 2, "f16": 2}
    if c["op"] == "quantize":
        r, k = (c["cols"], c["rows"]) if c["transpose"] else (c["rows"], c["cols"])
        scales = _up(r, c["block_rows"]) // c["block_rows"] * _up(_up(k, 128) // 128, 4)
        return {"bytes": c["n"] * (c["rows"] * c["cols"] * size[c["dtype"]] + r * _up(k, 128) + scales),
                "flops": 3 * c["n"] * c["rows"] * c["cols"]}
    if c["op"] == "product":
        K = c["K"]
        return {"bytes": c["n"] * ((c["M"] + c["N"]) * (K + K // 128) + c["M"] * c["N"] * size[c["out"]]),
                "flops": 2 * c["n"] * c["M"] * c["N"] * K}
    if c["op"] == "linear":
        T, K, N = c["tokens"], c["K"], c["N"]
        return {"bytes": 2 * (T * K + N * K + T * N) * 2, "flops": 6 * T * K * N}
    N, d, V = c["N"], c["d"], c["V"]
    once = (N * d + V * d) * size[c["dtype"]]
    return {"bytes": (2 if c["grads"] else 1) * once + 8 * N, "flops": (6 if c["grads"] else 2) * N * d * V}


# ----------------------------------------------------------------------------
# inputs
# ----------------------------------------------------------------------------
def _values(gen, shape, dtype, spread):
    """Normal values whose rows differ in size, with a few large entries, as activations have."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= torch.exp(spread * torch.randn(shape[:-1] + (1,), generator=gen, device="cuda"))
    x *= 1.0 + 15.0 * (torch.rand(shape, generator=gen, device="cuda") < 1e-3)
    return x.to(dtype)


def _operand(gen, n, rows, cols, fmt, block_rows):
    """A matrix as it is held: 8-bit values [n, rows, K] and scales, K the padded width."""
    K = _up(cols, 128)
    x = torch.randn((n, rows, K), generator=gen, device="cuda") * (LARGEST[fmt] / 5)
    x.clamp_(-LARGEST[fmt], LARGEST[fmt])
    x[..., cols:] = 0
    q = x.to(FORMATS[fmt])
    held = torch.full((n, -(-rows // block_rows), _up(K // 128, 4)), 127, dtype=torch.uint8, device="cuda")
    least = 108 if fmt == "e4m3" else 101
    held[..., :K // 128] = torch.randint(least, least + 14, (n, held.shape[1], K // 128), generator=gen, device="cuda").to(torch.uint8)
    return q, held.view(torch.float8_e8m0fnu)


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    if c["op"] == "quantize":
        return {"case": c, "x": _values(gen, (c["n"], c["rows"], c["cols"]), DTYPES[c["dtype"]], 1.0)}
    if c["op"] == "product":
        a, a_scale = _operand(gen, c["n"], c["M"], c["K"], c["a_fmt"], 1)
        b, b_scale = _operand(gen, c["n"], c["N"], c["K"], c["b_fmt"], c["b_rows"])
        out = torch.empty((c["n"], c["M"], c["N"]), dtype=DTYPES[c["out"]], device="cuda")
        return {"case": c, "a": a, "a_scale": a_scale, "b": b, "b_scale": b_scale, "c": out}
    if c["op"] == "linear":
        dt = DTYPES[c["dtype"]]
        x = _values(gen, (c["tokens"], c["K"]), dt, 0.3)
        w = (torch.randn((c["N"], c["K"]), generator=gen, device="cuda") / math.sqrt(c["K"])).to(dt)
        dy = _values(gen, (c["tokens"], c["N"]), dt, 1.0) * 1e-3
        return {"case": c, "x": x, "w": w, "dy": dy, "y": torch.empty_like(dy), "dx": torch.empty_like(x),
                "dw": torch.empty_like(w)}
    dt = DTYPES[c["dtype"]]
    N, d, V = c["N"], c["d"], c["V"]
    weight = (torch.randn((V, d), generator=gen, device="cuda") * (1.5 / math.sqrt(d))).to(dt)
    targets = torch.randint(0, V, (N,), generator=gen, device="cuda")
    hidden = torch.randn((N, d), generator=gen, device="cuda")
    # some rows already point at their target, as far as a trained model's do
    hidden += weight[targets].float() * (6.0 * torch.rand((N, 1), generator=gen, device="cuda"))
    # a packed batch's padding and prompts have no target; the first row always has one
    skip = torch.rand(N, generator=gen, device="cuda") < 0.1
    skip[0] = False
    targets = torch.where(skip, torch.full_like(targets, -100), targets)
    state = {"case": c, "hidden": hidden.to(dt), "weight": weight, "targets": targets}
    if c["grads"]:
        state["dhidden"] = torch.empty((N, d), dtype=dt, device="cuda")
        state["dweight"] = torch.empty((V, d), dtype=dt, device="cuda")
        if c["reduction"] == "none":  # the gradient that arrives at each row's loss
            state["row_scale"] = torch.rand(N, generator=gen, device="cuda") / N
    return state


# ----------------------------------------------------------------------------
# plain forms
# ----------------------------------------------------------------------------
def plain_quantize(x, fmt, block_rows, transpose):
    """(values, scales): 2^e the least power of two that keeps a block's largest finite entry in range."""
    x = x.float()
    if x.dim() == 2:
        return tuple(t[0] for t in plain_quantize(x[None], fmt, block_rows, transpose))
    if transpose:
        x = x.transpose(1, 2)
    n, rows, cols = x.shape
    K, R = _up(cols, 128), _up(rows, block_rows)
    p = torch.zeros((n, R, K), device=x.device)
    p[:, :rows, :cols] = x
    blocks = p.view(n, R // block_rows, block_rows, K // 128, 128)
    size = blocks.abs()
    amax = torch.where(torch.isfinite(size), size, torch.zeros_like(size)).amax(dim=(2, 4))
    frac, e = torch.frexp(amax)
    e = e - (9 if fmt == "e4m3" else 16) + (frac > 0.875).to(e.dtype)
    e = torch.where(amax > 0, e.clamp(-127, 127), torch.zeros_like(e))
    inverse = ((127 - e) << 23).to(torch.int32).view(torch.float32)  # 2^-e from its exponent's bits
    q = (blocks * inverse[:, :, None, :, None]).to(FORMATS[fmt]).view(n, R, K)[:, :rows].contiguous()
    held = torch.full((n, R // block_rows, _up(K // 128, 4)), 127, dtype=torch.uint8, device=x.device)
    held[..., :K // 128] = (e + 127).to(torch.uint8)
    return q, held.view(torch.float8_e8m0fnu)


def _widen(q, scale, dtype=torch.float32):
    """The values that 8-bit blocks stand for."""
    n, rows, K = q.shape
    block_rows = 1 if scale.shape[1] == rows else 128
    s = scale[..., :K // 128].to(dtype).repeat_interleave(block_rows, 1)[:, :rows]
    return (q.to(dtype).view(n, rows, K // 128, 128) * s[..., None]).view(n, rows, K)


def plain_product(a, a_scale, b, b_scale, dtype):
    if a.dim() == 2:
        return plain_product(a[None], a_scale[None], b[None], b_scale[None], dtype)[0]
    return torch.matmul(_widen(a, a_scale), _widen(b, b_scale).transpose(1, 2).contiguous()).to(dtype)


def plain_xent(hidden, weight, targets, reduction, row_scale, grads):
    x, w = hidden.float(), weight.float()
    z = x @ w.t()
    top = z.amax(dim=1, keepdim=True)
    e = torch.exp(z - top)
    total = e.sum(dim=1, keepdim=True)
    lse = (torch.log(total) + top)[:, 0]
    kept = targets != -100
    at = torch.where(kept, targets, torch.zeros_like(targets))
    loss = torch.where(kept, lse - z.gather(1, at[:, None])[:, 0], torch.zeros_like(lse))
    count = kept.sum().clamp(min=1).float()
    out = loss.sum() / count if reduction == "mean" else loss.sum() if reduction == "sum" else loss
    if not grads:
        return out, None, None
    g = kept.float()
    if reduction == "mean":
        g = g / count
    if row_scale is not None:
        g = g * row_scale
    del z
    p = e.div_(total)
    p.scatter_add_(1, at[:, None], torch.full_like(at, -1, dtype=torch.float32)[:, None])
    p *= g[:, None]
    return out, (p @ w).to(hidden.dtype), (p.t() @ x).to(weight.dtype)


# ----------------------------------------------------------------------------
# one pass
# ----------------------------------------------------------------------------
def run(state):
    c = state["case"]
    if own:
        import matrix_inverse_roots_amd as mir
    if c["op"] == "quantize":
        if own:
            return mir.shampoo_quantize_f8(state["x"], fmt=c["fmt"], block_rows=c["block_rows"], transpose=c["transpose"])
        return plain_quantize(state["x"], c["fmt"], c["block_rows"], c["transpose"])
    if c["op"] == "product":
        a, sa, b, sb = state["a"], state["a_scale"], state["b"], state["b_scale"]
        if own:
            return mir.shampoo_matmul_f8(a, sa, b, sb, state["c"])
        return plain_product(a, sa, b, sb, state["c"].dtype)
    if c["op"] == "linear":
        x, w, dy = state["x"], state["w"], state["dy"]
        if own:
            xq, xt = mir.shampoo_quantize_f8(x, fmt="e4m3", block_rows=1, transpose="both")
            wq, wt = mir.shampoo_quantize_f8(w, fmt="e4m3", block_rows=128, transpose="both")
            dyq, dyt = mir.shampoo_quantize_f8(dy, fmt="e5m2", block_rows=1, transpose="both")
            return (mir.shampoo_matmul_f8(*xq, *wq, state["y"]), mir.shampoo_matmul_f8(*dyq, *wt, state["dx"]),
                    mir.shampoo_matmul_f8(*dyt, *xt, state["dw"]))
        quantize = plain_quantize
        xq, wq, dyq = quantize(x, "e4m3", 1, False), quantize(w, "e4m3", 128, False), quantize(dy, "e5m2", 1, False)
        xt, wt, dyt = quantize(x, "e4m3", 1, True), quantize(w, "e4m3", 128, True), quantize(dy, "e5m2", 1, True)
        return (plain_product(*xq, *wq, x.dtype), plain_product(*dyq, *wt, x.dtype), plain_product(*dyt, *xt, w.dtype))
    if own:
        loss = mir.shampoo_linear_xent(state["hidden"], state["weight"], state["targets"], reduction=c["reduction"],
                                       row_scale=state.get("row_scale"), dhidden=state.get("dhidden"),
                                       dweight=state.get("dweight"))
        return (loss, state["dhidden"], state["dweight"]) if c["grads"] else loss
    got = plain_xent(state["hidden"], state["weight"], state["targets"], c["reduction"], state.get("row_scale"), c["grads"])
    return got if c["grads"] else got[0]


# ----------------------------------------------------------------------------
# the definition in 64 bits
# ----------------------------------------------------------------------------
def _two(e):
    """2^e (float64) for whole e, from its bits."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _grid(v, fmt):
    """v (float64, in range) on the 8-bit format's grid, ties to even."""
    mant, low = (3, -6) if fmt == "e4m3" else (2, -14)
    e = torch.frexp(v).exponent.double() - 1
    step = _two(torch.clamp(e, min=low) - mant)
    return torch.round(v / step) * step


def _blocks64(x, fmt, block_rows):
    """[rows, cols] float64 -> (8-bit values, scales as numbers), block by block."""
    rows, cols = x.shape
    K, R = _up(cols, 128), _up(rows, block_rows)
    x = torch.nn.functional.pad(x, (0, K - cols, 0, R - rows))
    tiles = x.reshape(R // block_rows, block_rows, K // 128, 128)
    big = tiles.abs().amax(dim=3).amax(dim=1)
    e = torch.ceil(torch.log2(torch.where(big > 0, big, torch.full_like(big, LARGEST[fmt])) / LARGEST[fmt]))
    # the logarithm's own rounding: one step down where that still holds the block, one up where it does not
    e = torch.where(big <= LARGEST[fmt] * _two(e - 1), torch.where(big > 0, e - 1, e), e)
    e = torch.where(big > LARGEST[fmt] * _two(e), e + 1, e).clamp(-127, 127)
    s = _two(e)
    q = _grid(tiles / s[:, None, :, None], fmt).reshape(R, K)[:rows]
    scale = torch.ones((R // block_rows, _up(K // 128, 4)), dtype=torch.float64, device=x.device)
    scale[:, :K // 128] = s
    return q, scale


def _stand64(q, scale, block_rows):
    rows, K = q.shape
    s = scale[:, :K // 128].repeat_interleave(128, 1).repeat_interleave(block_rows, 0)[:rows]
    return q * s


def exact(case, seed):
    c, s = case, prepare(case, seed)
    if c["op"] == "quantize":
        got = [_blocks64((m.double().t() if c["transpose"] else m.double()), c["fmt"], c["block_rows"]) for m in s["x"]]
        return torch.stack([q for q, _ in got]), torch.stack([t for _, t in got])
    if c["op"] == "product":
        a_e, b_e = s["a_scale"].double(), s["b_scale"].double()
        one = lambda q, t, rb: _stand64(q.double(), t, rb)  # noqa: E731
        return torch.stack([one(s["a"][i], a_e[i], 1) @ one(s["b"][i], b_e[i], c["b_rows"]).t() for i in range(c["n"])])
    if c["op"] == "linear":
        both = lambda m, fmt, rb: _stand64(*_blocks64(m.double(), fmt, rb), rb)  # noqa: E731
        x, w, dy = s["x"], s["w"], s["dy"]
        T, K, N = c["tokens"], c["K"], c["N"]
        y = both(x, "e4m3", 1) @ both(w, "e4m3", 128).t()
        dx = both(dy, "e5m2", 1)[:, :N] @ both(w.t(), "e4m3", 128)[:, :N].t()
        dw = both(dy.t(), "e5m2", 1)[:, :T] @ both(x.t(), "e4m3", 1)[:, :T].t()
        return y, dx, dw
    x, w, t = s["hidden"].double(), s["weight"].double(), s["targets"]
    kept = t >= 0
    logits = x @ w.t()
    lse = torch.logsumexp(logits, dim=1)
    rows = torch.arange(len(t), device=t.device)
    at = t.clamp(min=0)
    loss = (lse - logits[rows, at]) * kept
    count = max(int(kept.sum()), 1)
    out = {"mean": loss.sum() / count, "sum": loss.sum(), "none": loss}[c["reduction"]]
    if not c["grads"]:
        return out
    g = kept.double() / (count if c["reduction"] == "mean" else 1)
    if "row_scale" in s:
        g = g * s["row_scale"].double()
    logits.sub_(lse[:, None]).exp_()
    # the target's own entry from the sum of all others, which keeps it where its probability is near one
    logits[rows, at] = 0
    logits[rows, at] = -logits.sum(dim=1)
    logits *= g[:, None]
    return out, logits @ w, logits.t() @ x
