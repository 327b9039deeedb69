"""Host-only: a workspace tensor whose elements do not lie in one piece (a view
that repeats or skips) is refused before anything is launched; its size would
say nothing about the memory behind its address."""

import pytest


@pytest.fixture
def mir(monkeypatch):
    import torch
    import matrix_inverse_roots_amd as m

    def never(*args):
        raise AssertionError("launched")

    monkeypatch.setattr(m, "_on_device", lambda *tensors: torch.device("cpu"))
    monkeypatch.setattr(m, "_dev", lambda t, name: None)
    monkeypatch.setattr(m, "_launch", never)
    monkeypatch.setattr(m, "_stream", never)
    return m


def calls(mir, ws):
    import torch
    x, w, wd = torch.zeros(40, 32), torch.zeros(64, 32), torch.zeros(32, 64)
    dy, kept = torch.zeros(40, 64), torch.zeros(40, 64)
    q, s = torch.zeros(8, 128).to(torch.float8_e4m3fn), torch.zeros(8, 4, dtype=torch.uint8)
    m = torch.zeros(2, 32, 32)
    return [
        lambda: mir.shampoo_linear(x, w, dy, ws=ws),
        lambda: mir.shampoo_linear_grad(dy, x, w, dw=w, ws=ws),
        lambda: mir.shampoo_gated_ffn(x, w, w, wd, torch.zeros(40, 32), ws=ws),
        lambda: mir.shampoo_gated_ffn_grad(x, x, w, w, wd, (kept, kept), dx=torch.zeros(40, 32), ws=ws),
        lambda: mir.shampoo_matmul_f8(q, s, q, s, torch.zeros(8, 8), ws=ws),
        lambda: mir.shampoo_linear_xent(x, w, torch.zeros(40, dtype=torch.int64), torch.zeros(()), ws=ws),
        lambda: mir.shampoo_inverse_root(m, m.clone(), 4, mir.RootOpts(), ws=ws),
        lambda: mir.shampoo_precondition(torch.zeros(4, 32, 32), m, m.clone(), ws=ws),
    ]


@pytest.mark.parametrize("k", range(8))
def test_views_that_repeat_or_skip(mir, k):
    import torch
    for ws in (torch.zeros(1, dtype=torch.uint8).expand(1 << 24), torch.zeros(1 << 16, dtype=torch.uint8)[::2],
               torch.zeros(256, 256, dtype=torch.uint8).t()):
        with pytest.raises(ValueError, match="contiguous"):
            calls(mir, ws)[k]()
    with pytest.raises(AssertionError, match="launched"):
        calls(mir, torch.zeros(1 << 16, dtype=torch.uint8))[k]()
