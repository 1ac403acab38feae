"""The training calls as a user's torch.autograd.Function makes them: norm, projection with function and residual, and
router with its losses as one step, the gradients of every leaf against 64-bit automatic differentiation."""
import pytest
import torch

from test_gpu_operators import D, DEV, HALF, gen, randn
from test_gpu_training_operators import phi, stream_rows

pytestmark = pytest.mark.gpu
COEF = (0.5, 0.05)


def functions(lmoe):
    class Norm(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, w, b):
            out, mean, rstd = lmoe.layer_norm(x, w, b, stats=True)
            ctx.save_for_backward(x, w, mean, rstd)
            return out

        @staticmethod
        def backward(ctx, dy):
            x, w, mean, rstd = ctx.saved_tensors
            return lmoe.layer_norm_backward(dy.contiguous(), x, mean, rstd, w)

    class Linear(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, W, bias, res):
            out, pre = lmoe.linear_act_bf16(x, W, bias, "gelu", res, pre=True)
            ctx.save_for_backward(x, W, pre)
            return out

        @staticmethod
        def backward(ctx, dout):
            x, W, pre = ctx.saved_tensors
            need = ctx.needs_input_grad
            dx, dW, db = lmoe.linear_act_bf16_backward(dout.contiguous(), x, W, "gelu", pre, *need[:3])
            return dx, dW, db, dout if need[3] else None

    class Router(torch.autograd.Function):
        """(gate weights, losses' weighted sum) of a row's latent; the picks have no gradient."""

        @staticmethod
        def forward(ctx, lat, Wr, mask, k):
            logits, idx, gate = lmoe.route(lat, Wr, k)
            loss, _, _ = lmoe.balance_loss(logits, idx, mask, COEF)
            ctx.save_for_backward(lat, Wr, mask, logits, idx, gate)
            ctx.mark_non_differentiable(idx)
            return gate, COEF[0] * loss[0] + COEF[1] * loss[1], idx

        @staticmethod
        def backward(ctx, dgate, dtotal, _):
            lat, Wr, mask, logits, idx, gate = ctx.saved_tensors
            dl = lmoe.balance_loss(logits, idx, mask, COEF, True, gate, dgate.contiguous(), dtotal.reshape(1))[3]
            dlat, dWr, _ = lmoe.linear_act_bf16_backward(dl, lat, Wr.bfloat16(), want_dbias=False, dW=torch.empty_like(Wr))
            return dlat, dWr, None, None

    return Norm.apply, Linear.apply, Router.apply


def leaves(g, T, H, d, E):
    return {"stream": stream_rows(g, T, H, torch.float32), "w": 1 + 0.1 * torch.randn(H, device=DEV, generator=g),
            "b": 0.1 * torch.randn(H, device=DEV, generator=g), "W": randn(g, d, H, scale=H ** -0.5),
            "bias": 0.1 * torch.randn(d, device=DEV, generator=g), "res": randn(g, T, d, scale=0.1),
            "Wr": torch.randn(E, d, device=DEV, generator=g) * d ** -0.5}


@pytest.mark.parametrize("T", [48, 200, 4000])
def test_a_step_through_autograd_functions(cuda_lib, T):
    H, d, E, k, scale = 520, 256, 64, 8, 1.5
    g = gen(T)
    v = leaves(g, T, H, d, E)
    mask = torch.rand(T, device=DEV, generator=g) < 0.8
    dgate = torch.randn(T, k, device=DEV, generator=g) * (0.1 / T)
    norm, linear, router = functions(cuda_lib)
    p = {n: t.clone().requires_grad_() for n, t in v.items()}
    lat = linear(norm(p["stream"], p["w"], p["b"]), p["W"], p["bias"], p["res"])
    gate, total, idx = router(lat, p["Wr"], mask, k)
    (scale * total + (gate * dgate).sum()).backward()
    assert cuda_lib.last_call_status() == cuda_lib.OK
    # the same in 64 bits on the same picks
    q = {n: t.detach().to(D).requires_grad_() for n, t in v.items()}
    c = q["stream"] - q["stream"].mean(1, keepdim=True)
    n6 = c / (c.square().mean(1, keepdim=True) + 1e-5).sqrt() * q["w"] + q["b"]
    z = n6 @ q["W"].t() + q["bias"]
    l = (z * phi(z) + q["res"]) @ q["Wr"].t()
    N = int(mask.sum())
    f = torch.bincount(idx[mask].reshape(-1).long(), minlength=E).to(D) * E / (k * N)
    m = mask[:, None].to(D)
    bal = ((torch.softmax(l, 1) * m).sum(0) / N * f).sum()
    zl = (torch.logsumexp(l, 1).square() * m[:, 0]).sum() / N
    want = COEF[0] * bal + COEF[1] * zl
    (scale * want + (torch.softmax(l.gather(1, idx.long()), 1) * dgate.to(D) * m).sum()).backward()
    total, want = float(total.detach()), float(want.detach())
    assert abs(total - want) < 1e-2 * abs(want)
    # bf16 roundings on the way (n, lat, dl or Wr, dlat, dz, the result), at most HALF of the norm each, by products that
    # keep norms apart by at most a ratio of about one: 6 of them, with room for two
    for n in p:
        assert p[n].grad.dtype == p[n].dtype
        assert float((p[n].grad.to(D) - q[n].grad).norm()) < 8 * HALF * float(q[n].grad.norm()), n


def test_the_calls_themselves_are_not_recorded(cuda_lib):
    """Outputs carry no graph, whatever the inputs require: the gradients are the _backward calls'."""
    g = gen(2)
    x, W = randn(g, 8, 64).requires_grad_(), randn(g, 16, 64).requires_grad_()
    assert not cuda_lib.linear_act_bf16(x, W, act="silu").requires_grad
    assert not cuda_lib.layer_norm(x).requires_grad
    l = torch.randn(8, 16, device=DEV, generator=g).requires_grad_()
    idx = torch.zeros(8, 2, dtype=torch.int32, device=DEV)
    assert not any(t.requires_grad for t in cuda_lib.balance_loss(l, idx, grad=True))
