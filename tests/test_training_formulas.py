"""The gradients' formulas, as the GPU tests hold the kernels to them, against central
differences in 64 bits (no GPU)."""
import math

import pytest
import torch

D = torch.float64
C = math.sqrt(8 / math.pi)


def _ops(monkeypatch=None):
    import importlib
    import sys
    import os
    here = os.path.dirname(os.path.abspath(__file__))
    if here not in sys.path:
        sys.path.insert(0, here)
    return importlib.import_module("test_gpu_training_operators")


def _diff(f, x, eps=1e-5):
    """df/dx of a scalar function, element by element."""
    g = torch.zeros_like(x)
    flat, out = x.view(-1), g.view(-1)
    for i in range(flat.numel()):
        keep = float(flat[i])
        flat[i] = keep + eps
        a = f()
        flat[i] = keep - eps
        b = f()
        flat[i] = keep
        out[i] = (a - b) / (2 * eps)
    return g


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
def test_slopes(act):
    ops = _ops()
    z = torch.cat([torch.linspace(-6, 6, 61, dtype=D) + 0.013, torch.tensor([-20., 20.], dtype=D)])
    v = lambda t: ops.act_ref(t, act)[0]
    assert torch.allclose(ops.slope_ref(z, act), (v(z + 1e-5) - v(z - 1e-5)) / 2e-5, atol=1e-8)


def test_layer_norm_gradients():
    g = torch.Generator().manual_seed(1)
    x, w, b, dy = (torch.randn(*s, dtype=D, generator=g) for s in ((3, 8), (8,), (8,), (3, 8)))

    def value():
        c = x - x.mean(1, keepdim=True)
        return (((c / (c.square().mean(1, keepdim=True) + 1e-3).sqrt()) * w + b) * dy).sum()

    c = x - x.mean(1, keepdim=True)
    rs = 1 / (c.square().mean(1, keepdim=True) + 1e-3).sqrt()
    h, gg = c * rs, dy * w
    dx = rs * (gg - gg.mean(1, keepdim=True) - h * (gg * h).mean(1, keepdim=True))
    assert torch.allclose(dx, _diff(value, x), atol=1e-8)
    assert torch.allclose((dy * h).sum(0), _diff(value, w), atol=1e-8)
    assert torch.allclose(dy.sum(0), _diff(value, b), atol=1e-8)


@pytest.mark.parametrize("twice", [False, True])
def test_balance_gradient(twice):
    ops = _ops()
    g = torch.Generator().manual_seed(2)
    T, E, k = 5, 6, 3
    l = torch.randn(T, E, dtype=D, generator=g)
    idx = torch.randint(0, E, (T, k), generator=g) if twice else torch.rand(T, E, generator=g).topk(k, 1).indices
    keep = torch.tensor([True, True, False, True, True])
    dw = torch.randn(T, k, dtype=D, generator=g)
    coef, scale = (0.7, 0.3), 1.5

    def value():  # the counts are constants; gate weights are the softmax over the picked logits
        loss = ops.balance_ref(l, idx, keep, coef)[0]
        w = torch.softmax(l.gather(1, idx), 1)
        return scale * (coef[0] * loss[0] + coef[1] * loss[1]) + (w * dw)[keep].sum()

    w = torch.softmax(l.gather(1, idx), 1)
    d = ops.balance_ref(l, idx, keep, coef, w, dw, scale)[3]
    assert torch.allclose(d, _diff(value, l), atol=1e-8)
