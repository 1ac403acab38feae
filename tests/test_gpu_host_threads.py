"""Host threads that call at once, each on a stream and with buffers of its own: a call of one size leaves alone what a
call of another size has set up for its launch."""
import ctypes
import threading

import pytest
import torch

from test_gpu_operators import DEV, gen, randn

pytestmark = pytest.mark.gpu
CALLS = 4000


def at_once(calls):
    """Each call (of the C entry point, which runs without Python's lock) many times by a thread of its own; all succeed."""
    codes = [set() for _ in calls]
    gate = threading.Barrier(len(calls))

    def work(i):
        torch.cuda.set_device(DEV)
        gate.wait()
        for _ in range(CALLS):
            codes[i].add(calls[i]())

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(calls))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert all(c == {0} for c in codes), codes


def test_layer_norm_gradients_of_other_widths(cuda_lib):
    lmoe = cuda_lib
    g = gen(1)
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    calls, outs, keep = [], [], []
    for H in (520, 1024, 6400, 7168):  # one instance of the kernel, other sizes of its ring
        x, mean, rstd = randn(g, 8, H), torch.zeros(8, device=DEV), torch.ones(8, device=DEV)
        want = lmoe.layer_norm_backward(x, x, mean, rstd)
        dx, dw, db = torch.empty_like(x), torch.empty(H, device=DEV), torch.empty(H, device=DEV)
        n = lmoe.layer_norm_backward_workspace_size(8, H)
        ws, s = torch.empty(n, dtype=torch.uint8, device=DEV), torch.cuda.Stream(DEV)
        args = (p(x), p(x), 0, p(mean), p(rstd), None, None, 8, H, p(dx), p(dw), p(db), p(ws), n, ctypes.c_void_p(s.cuda_stream))
        calls.append(lambda args=args: lmoe._layer_norm_back(*args))
        outs.append((want, (dx, dw, db)))
        keep.append((x, mean, rstd, ws, s))
    torch.cuda.synchronize()
    at_once(calls)
    assert all(torch.equal(a, b) for want, got in outs for a, b in zip(want, got))


def test_balance_losses_of_other_widths(cuda_lib):
    lmoe = cuda_lib
    g = gen(2)
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    calls, outs, keep = [], [], []
    for E in (1028, 1536, 2048):
        l = torch.randn(40, E, device=DEV, generator=g)
        idx = torch.rand(40, E, device=DEV, generator=g).topk(4, 1).indices.to(torch.int32).contiguous()
        want = lmoe.balance_loss(l, idx, coef=(0.5, 0.25), grad=True)
        loss, counts, probs = torch.empty(2, device=DEV), torch.empty(E, dtype=torch.int32, device=DEV), torch.empty(E, device=DEV)
        d, n = torch.empty_like(l), lmoe.balance_loss_workspace_size(40, E, 4)
        ws, s = torch.zeros(n, dtype=torch.uint8, device=DEV), torch.cuda.Stream(DEV)
        grad = lmoe.BalanceGrad(d.data_ptr(), 0.5, 0.25, None, None, None)
        args = (p(l), p(idx), None, 40, E, 4, p(loss), p(counts), p(probs), ctypes.byref(grad), p(ws), n,
                ctypes.c_void_p(s.cuda_stream))
        calls.append(lambda args=args: lmoe._balance(*args))
        outs.append((want, (loss, counts, probs, d)))
        keep.append((l, idx, ws, s, grad))
    torch.cuda.synchronize()
    at_once(calls)
    assert all(torch.equal(a, b) for want, got in outs for a, b in zip(want, got))


@pytest.mark.parametrize("T", [64, 2000])
def test_permutes_of_other_expert_counts(cuda_lib, T):
    lmoe = cuda_lib
    g = gen(T)
    p = lambda t: ctypes.c_void_p(t.data_ptr())
    calls, outs, keep = [], [], []
    for E in (896, 1600, 2048):
        idx = torch.rand(T, E, device=DEV, generator=g).topk(4, 1).indices.to(torch.int32).contiguous()
        want = lmoe.permute(idx, E)[:4]
        got = [torch.empty_like(t) for t in want]
        n = lmoe.permute_workspace_size(T, E, 4)
        ws, s, dims = torch.zeros(n, dtype=torch.uint8, device=DEV), torch.cuda.Stream(DEV), lmoe.dims(T, 128, E, 4, 32)
        args = (p(idx), ctypes.byref(dims), *map(p, got), p(ws), n, ctypes.c_void_p(s.cuda_stream))
        calls.append(lambda args=args: lmoe._permute(*args))
        outs.append((want, got))
        keep.append((idx, ws, s, dims))
    torch.cuda.synchronize()
    at_once(calls)
    assert all(torch.equal(a, b) for want, got in outs for a, b in zip(want, got))
