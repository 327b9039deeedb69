"""The paths over the 8-bit products and the projection's loss together: the
loss with 8-bit logits, projection_loss feeding an optimizer step, and a whole
training step of a small network on these operators."""

import numpy as np
import pytest

import f8_reference as ref
from helpers import log
from test_gpu_xent import definition, make, check

pytestmark = pytest.mark.gpu

U = 2.0 ** -23


@pytest.fixture(scope="module")
def mir():
    import matrix_inverse_roots_amd as m
    return m


def code(q, s, rb, fmt):
    """What quantised blocks stand for, in float64."""
    import torch
    return ref.stand_for(ref.code_values(fmt)[q.view(torch.uint8).cpu().numpy()], s.view(torch.uint8).cpu().numpy(), rb)


@pytest.mark.parametrize("wdt", ["float32", "bfloat16"])
@pytest.mark.parametrize("reduction", ["mean", "none"])
@pytest.mark.parametrize("N,d,V", [(1, 1, 2), (3, 100, 129), (130, 96, 257), (300, 200, 5001), (257, 640, 700)])
def test_loss_with_8_bit_logits(mir, N, d, V, reduction, wdt):
    """The softmax, its loss and its gradient are those of the 8-bit logits;
    the gradients' products use the bfloat16 operands.  The 8-bit products drop
    what lies 2^-13 below the largest of an instruction's: dz = (2^-13 + d 2^-23)
    |x| |w| on the quantised operands."""
    import torch
    h, w, t = make(N, d, V, "bfloat16", N + d)
    w = w.float() * 1.001 if wdt == "float32" else w
    dh, dw = torch.full_like(h, float("nan")), torch.full((V, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    loss = mir.shampoo_linear_xent(h, w, t, reduction=reduction, dhidden=dh, dweight=dw, logits_dtype=torch.float8_e4m3fn)
    alone = mir.shampoo_linear_xent(h, w, t, reduction=reduction, logits_dtype=torch.float8_e4m3fn)
    assert torch.equal(loss, alone)
    X, W = code(*mir.shampoo_quantize_f8(h), 1, "e4m3"), code(*mir.shampoo_quantize_f8(w), 1, "e4m3")
    z = X @ W.T
    dz = ((2.0 ** -13 + (d + 1) * U) * (np.abs(X) @ np.abs(W).T)).max(axis=1)
    tt = t.cpu().numpy()
    kept, at, rows = tt != -100, np.where(tt != -100, tt, 0), np.arange(N)
    m = z.max(axis=1, keepdims=True)
    lse = np.log(np.exp(z - m).sum(axis=1)) + m[:, 0]
    count = max(int(kept.sum()), 1)
    each = np.where(kept, lse - z[rows, at], 0.0)
    few = 2 * dz + 160 * U + 4 * U * (np.abs(lse) + np.abs(z[rows, at]))
    if reduction == "mean":
        check(loss, each.sum() / count, (few * kept).sum() / count + U * abs(each.sum()), "loss")
    else:
        check(loss, each, few * kept + 2 * U * np.abs(each), "loss")
    g = kept / (count if reduction == "mean" else 1)
    P = np.exp(z - lse[:, None])
    rel = few[:, None] + 2.1 * 2.0 ** -8
    dP = P * rel
    p_t = P[rows, at].copy()
    P[rows, at] -= 1.0
    dP[rows, at] = p_t * rel[:, 0] + 2.0 ** -8 * np.abs(P[rows, at])
    P, dP = P * g[:, None], dP * g[:, None]
    x, y = h.double().cpu().numpy(), w.bfloat16().double().cpu().numpy()
    for got, want, err in ((dh, P @ y, dP @ np.abs(y) + V * U * ((np.abs(P) + dP) @ np.abs(y))),
                           (dw, P.T @ x, dP.T @ np.abs(x) + N * U * ((np.abs(P) + dP).T @ np.abs(x)))):
        check(got, want, 1.01 * (err + 2.0 ** -8 * np.abs(want)) + 1e-37, "gradient")
    # and the loss stays near the bfloat16 one: logits off by the operands' roundings
    b = definition(h, w.bfloat16(), t, reduction)[0]
    log(f"N {N} d {d} V {V} {wdt}: loss {np.mean(loss.cpu().numpy()):.4f}, with bfloat16 logits {np.mean(b):.4f}")


def test_8_bit_logits_refusals(mir):
    import torch
    h, w, t = make(10, 64, 200, "float32", 1)
    with pytest.raises(ValueError, match="bfloat16 hidden"):
        mir.shampoo_linear_xent(h, w, t, logits_dtype=torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        mir.shampoo_linear_xent(h.bfloat16(), w, t, logits_dtype=torch.float8_e5m2)


def optimizer(mir, V, d, gdt, **kw):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    W = [torch.randn((96, 64), generator=g, device="cuda"), torch.randn((V, d), generator=g, device="cuda") / d ** 0.5]
    hp = dict(block_size=128, beta2=0.9, eps=1e-4, root=mir.RootOpts(method="cn", iters=25, eps=1e-4), graft="sgd", lr=0.05,
              grad_dtype=gdt)
    return mir.Shampoo(W, **{**hp, **kw})


@pytest.mark.parametrize("hdt,gdt", [("float32", "float32"), ("bfloat16", "float32"), ("bfloat16", "bfloat16")])
def test_projection_loss_feeds_the_step(mir, hdt, gdt):
    """Two micro-batches through projection_loss, then a step with None, give
    the bits of the same step on the gradient computed by hand; the loss and
    hidden's gradient match float64."""
    import torch
    V, d = 500, 64
    hd, gd = getattr(torch, hdt), getattr(torch, gdt)
    a, b = optimizer(mir, V, d, gd), optimizer(mir, V, d, gd)
    for step in range(2):
        g0 = torch.randn(96, 64, device="cuda").to(gd)
        dw = torch.empty((V, d), dtype=gd, device="cuda")
        for k in range(2):
            h, _, t = make(70 + k, d, V, hdt, 10 * step + k)
            dh = torch.empty_like(h)
            loss = a.projection_loss(1, h, t, dhidden=dh, scale=0.5)
            w = b.params[1]
            wr = w if hd == torch.float32 else w.to(hd)
            r = definition(h, wr, t, "mean", scale=0.5)
            check(loss, r[0], r[4], "loss")
            check(dh, r[1], r[5], "dhidden")
            mir.shampoo_linear_xent(h, w, t, dweight=dw, scale=0.5, accumulate=k > 0)
        a.step([g0, None])
        b.step([g0, dw])
        for x, y in zip(a.params, b.params):
            assert torch.equal(x, y)
    with pytest.raises(ValueError, match="projection_loss"):
        a.step([g0, None])
    a.step([g0, dw])


def test_projection_loss_refusals(mir):
    import torch
    opt = optimizer(mir, 200, 64, torch.bfloat16)
    h, _, t = make(10, 64, 200, "float32", 1)
    with pytest.raises(ValueError, match="float32 gradients"):
        opt.projection_loss(1, h, t)
    with pytest.raises(ValueError):
        opt.projection_loss(1, h.bfloat16()[:, :32], t)
    with pytest.raises(IndexError):
        opt.projection_loss(2, h.bfloat16(), t)
    opt = mir.Shampoo([torch.zeros((4, 8, 8), device="cuda")], block_size=64)
    with pytest.raises(ValueError, match="dimensions"):
        opt.projection_loss(0, h, t)


def test_captured_step_on_the_kept_gradient(mir):
    """capture() with None replays on the buffer that projection_loss fills."""
    import torch
    V, d = 300, 64
    a, b = (optimizer(mir, V, d, torch.float32) for _ in range(2))
    g0 = torch.randn(96, 64, device="cuda")

    def loss(o, k):
        h, _, t = make(60, d, V, "bfloat16", k)
        return o.projection_loss(1, h, t)

    for o in (a, b):
        loss(o, 0)
        o.step([g0, None])
    loss(a, 1)
    replay = a.capture([g0, None])
    for k in range(1, 5):
        la = loss(a, k) if k > 1 else None
        lb = loss(b, k)
        torch.cuda.synchronize()
        replay()
        torch.cuda.synchronize()
        b.step([g0, None])
        assert la is None or torch.equal(la, lb)
        for x, y in zip(a.params, b.params):
            assert torch.equal(x, y)


def test_float32_weight_beside_bfloat16_hidden(mir):
    """The same bits as with the weight rounded beforehand, at every alignment."""
    import torch
    for d in (64, 33, 100):
        h, w, t = make(50, d, 333, "bfloat16", d)
        w32 = torch.randn(333, d, device="cuda")
        out = []
        for weight in (w32, w32.bfloat16()):
            dh, dw = torch.empty_like(h), torch.empty(333, d, device="cuda")
            out.append((mir.shampoo_linear_xent(h, weight, t, dhidden=dh, dweight=dw), dh, dw))
        assert all(torch.equal(x, y) for x, y in zip(*out))


def test_network_step_in_8_bits(mir):
    """x -> x W0^T in 8 bits -> projection loss -> 8-bit gradients of the layer
    with 8-bit logits -> 8-bit gradients of the layer -> a step: the layer's
    products against float64 on the same operands, the rest finite and moving."""
    import torch
    T, K, d, V = 160, 96, 192, 700
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    W = [torch.randn((d, K), generator=g, device="cuda") / K ** 0.5, torch.randn((V, d), generator=g, device="cuda") / d ** 0.5]
    opt = mir.Shampoo(W, block_size=128, beta2=0.9, eps=1e-4, root=mir.RootOpts(method="cn", iters=25, eps=1e-4), graft="sgd",
                      lr=0.5, grad_dtype=torch.bfloat16, precondition_dtype=torch.bfloat16)
    x = torch.randn((T, K), generator=g, device="cuda").bfloat16()
    t = torch.randint(0, V, (T,), generator=g, device="cuda")
    for step in range(3):
        (xq, xt) = mir.shampoo_quantize_f8(x, transpose="both")
        wq = mir.shampoo_quantize_f8(W[0], block_rows=128)
        h = mir.shampoo_matmul_f8(*xq, *wq, torch.empty((T, d), dtype=torch.bfloat16, device="cuda"))
        X, W0 = code(*xq, 1, "e4m3"), code(*wq, 128, "e4m3")
        want = X @ W0.T
        bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -13 * (np.abs(X) @ np.abs(W0).T)
        assert (np.abs(h.double().cpu().numpy() - want) <= bound).all()
        dh = torch.empty_like(h)
        loss = opt.projection_loss(1, h, t, dhidden=dh, logits_dtype=torch.float8_e4m3fn)
        again = mir.shampoo_linear_xent(h, W[1], t, logits_dtype=torch.float8_e4m3fn)
        assert torch.equal(loss, again) and torch.isfinite(loss) and torch.isfinite(dh).all()
        dt = mir.shampoo_quantize_f8(dh, fmt="e5m2", transpose=True)
        dw = mir.shampoo_matmul_f8(*dt, *xt, torch.empty((d, K), dtype=torch.bfloat16, device="cuda"))
        D, Xt = code(*dt, 1, "e5m2"), code(*xt, 1, "e4m3")
        want = D @ Xt.T
        bound = 2.0 ** -8 * np.abs(want) + 2.0 ** -13 * (np.abs(D) @ np.abs(Xt).T)
        assert (np.abs(dw.double().cpu().numpy() - want) <= bound).all()
        before = [w.clone() for w in W]
        opt.step([dw, None])
        assert all(torch.isfinite(w).all() and not torch.equal(w, b) for w, b in zip(W, before))
        log(f"step {step}: loss {loss.item():.4f}")


def test_workspaces_belong_to_the_stream_that_uses_them(mir):
    """Calls on a side stream that allocate for themselves, with allocations of
    the same sizes filled on the current stream right behind them."""
    import torch
    h, w, t = make(1500, 512, 20001, "bfloat16", 3)
    a = mir.shampoo_quantize_f8(h[:64].repeat(1, 16))
    sizes = [mir.shampoo_linear_xent_workspace(h, w, t, h, w) // 4, mir.shampoo_matmul_f8_workspace(1, 64, 64, 8192) // 4]
    assert min(sizes) > 0
    want = []
    for stream in (None, torch.cuda.Stream()):
        dh, dw = torch.empty_like(h), torch.empty_like(w)
        c = torch.empty((64, 64), device="cuda")
        for k in range(3):
            torch.cuda.synchronize()
            loss = mir.shampoo_linear_xent(h, w, t, dhidden=dh, dweight=dw, stream=stream)
            mir.shampoo_matmul_f8(*a, *a, c, stream=stream)
            junk = [torch.full((n,), float("nan"), device="cuda") for n in sizes for _ in range(2)]
            torch.cuda.synchronize()
            del junk
        want.append([x.clone() for x in (loss, dh, dw, c)])
    assert all(torch.equal(x, y) for x, y in zip(*want))


def test_two_calls_at_once(mir):
    """Two streams, each with its own call in flight, give the bits of one after the other."""
    import torch
    data = [make(700, 256, 9001, "bfloat16", k) for k in range(2)]
    out = []
    for streams in ((None, None), (torch.cuda.Stream(), torch.cuda.Stream())):
        torch.cuda.synchronize()
        got = []
        for (h, w, t), s in zip(data, streams):
            dh, dw = torch.empty_like(h), torch.empty_like(w)
            torch.cuda.synchronize() if s is None else None
            got += [mir.shampoo_linear_xent(h, w, t, dhidden=dh, dweight=dw, stream=s), dh, dw]
        torch.cuda.synchronize()
        out.append(got)
    assert all(torch.equal(x, y) for x, y in zip(*out))


def test_kept_gradient_belongs_to_its_stream(mir):
    """The kept gradient's first call on a side stream, while the current
    stream still fills memory of that size that it has given back."""
    import torch
    h, w, t = make(300, 64, 5001, "bfloat16", 5)
    want = torch.empty_like(w)
    mir.shampoo_linear_xent(h, w.float(), t, dweight=want)
    side = torch.cuda.Stream()
    for k in range(3):
        opt = mir.Shampoo([w.float()], block_size=64, grad_dtype=torch.bfloat16)
        torch.cuda.synchronize()
        busy = torch.empty((64, 1 << 20), device="cuda")
        junk = torch.empty_like(w)
        for _ in range(20):
            busy.fill_(1.0)
        junk.fill_(float("nan"))
        del junk
        opt.projection_loss(0, h, t, stream=side)
        torch.cuda.synchronize()
        assert torch.equal(opt._kept[0], want)


def busy(stream, ms=10):
    """Some milliseconds of work on ``stream``, so that what follows there starts late."""
    import torch
    with torch.cuda.stream(stream):
        x = torch.empty((64, 1 << 20), device="cuda")
        for _ in range(10 * ms):
            x.fill_(1.0)


@pytest.mark.parametrize("captured", [False, True])
def test_loss_and_step_on_different_streams(mir, captured):
    """Micro-batches on two side streams, steps on the current one, each in turn
    held up, with no synchronisation by the caller: the bits of the same calls
    one after the other."""
    import torch
    V, d, steps = 500, 64, 5
    a, b = (optimizer(mir, V, d, torch.bfloat16) for _ in range(2))
    g0 = torch.randn(96, 64, device="cuda").bfloat16()
    data = [[make(70 + k, d, V, "bfloat16", 10 * s + k)[::2] for k in range(2)] for s in range(steps)]
    want, got = [], []
    for s in range(steps):
        for h, t in data[s]:
            want.append(a.projection_loss(1, h, t, scale=0.5))
            torch.cuda.synchronize()
        a.step([g0, None])
        torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    cur = torch.cuda.current_stream()
    step = lambda: b.step([g0, None])  # noqa: E731
    torch.cuda.synchronize()
    for s in range(steps):
        if s == 1 and captured:
            for h, t in data[s]:
                got.append(b.projection_loss(1, h, t, scale=0.5, stream=sides[0]))
            step = b.capture([g0, None])
        else:
            for k, (h, t) in enumerate(data[s]):
                if (s + k) % 3 == 0:
                    busy(sides[k])
                got.append(b.projection_loss(1, h, t, scale=0.5, stream=sides[k]))
        if s % 2:
            busy(cur)
        step()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    assert all(torch.equal(x, y) for x, y in zip(a.params, b.params))


def test_replay_needs_a_gradient_of_its_own(mir):
    """A replay without a projection_loss since the last step raises, as a step
    does, and changes nothing; with one it goes on."""
    import torch
    V, d = 300, 64
    opt = optimizer(mir, V, d, torch.float32)
    g0 = torch.randn(96, 64, device="cuda")
    h, _, t = make(60, d, V, "bfloat16", 1)
    opt.projection_loss(1, h, t)
    opt.step([g0, None])
    opt.projection_loss(1, h, t)
    replay = opt.capture([g0, None])
    replay()
    before, steps = [p.clone() for p in opt.params], opt.t
    for _ in range(2):
        with pytest.raises(ValueError, match="projection_loss"):
            replay()
    assert opt.t == steps and all(torch.equal(p, q) for p, q in zip(opt.params, before))
    opt.projection_loss(1, h, t)
    replay()
    assert opt.t == steps + 1 and not torch.equal(opt.params[1], before[1])


def test_loss_in_a_graph_of_the_caller(mir):
    """A capture of the loss with its step replays as the eager calls run; a
    capture of the loss alone is no gradient for a step outside, until an
    eager call has made one, to which its replays then add."""
    import torch
    V, d = 300, 64
    a, b = (optimizer(mir, V, d, torch.float32) for _ in range(2))
    g0 = torch.randn(96, 64, device="cuda")
    h, _, t = make(60, d, V, "bfloat16", 1)
    for o in (a, b):
        o.projection_loss(1, h, t)
        o.step([g0, None])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = a.projection_loss(1, h, t)
        a.step([g0, None])
    for k in range(4):
        h2, _, t2 = make(60, d, V, "bfloat16", 10 + k)
        h.copy_(h2)
        t.copy_(t2)
        graph.replay()
        torch.cuda.synchronize()
        want = b.projection_loss(1, h, t)
        b.step([g0, None])
        torch.cuda.synchronize()
        assert torch.equal(loss, want)
        assert all(torch.equal(p, q) for p, q in zip(a.params, b.params))
    alone = torch.cuda.CUDAGraph()
    with torch.cuda.graph(alone):
        a.projection_loss(1, h, t)
    with pytest.raises(ValueError, match="projection_loss"):
        a.step([g0, None])
    # two more micro-batches by replays behind an eager one
    for o in (a, b):
        o.projection_loss(1, h, t, scale=0.25)
    torch.cuda.synchronize()
    more = torch.cuda.CUDAGraph()
    with torch.cuda.graph(more):
        a.projection_loss(1, h, t, scale=0.25)
    for _ in range(2):
        more.replay()
        b.projection_loss(1, h, t, scale=0.25)
    for o in (a, b):
        o.step([g0, None])
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a.params, b.params))
    # none of these leaves the next capture anything to add to
    again = torch.cuda.CUDAGraph()
    with torch.cuda.graph(again):
        a.projection_loss(1, h, t)
        a.step([g0, None])
    again.replay()
    b.projection_loss(1, h, t)
    b.step([g0, None])
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a.params, b.params))
