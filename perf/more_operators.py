"""Workloads of the operators that a layer's dense, trained neighbours need: the linear layer with bias, activation and
residual in one pass, layer norm, the router's balance loss, each with its gradients.

`run` computes a case in plain torch operations, or, where `own` is true, by the library's calls.
"""
import math

import torch

own = False
DEV = "cuda"
EPS = 1e-5
COEF = (0.01, 0.001)  # of the balance loss and of the z loss
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


# ---- cases ---------------------------------------------------------------------------

def listed():
    return [
        # one token: latent -> hidden with a bias, added to the residual stream
        {"name": "linear_1", "op": "linear", "rows": 1, "K": 3584, "N": 7168, "act": "none", "bias": "f32",
         "res": "bf16", "pre": False},
        # the decode batch of the benchmark, hidden -> latent with an activation
        {"name": "linear_64", "op": "linear", "rows": 64, "K": 7168, "N": 3584, "act": "gelu_tanh", "bias": "bf16",
         "res": "none", "pre": False},
        # a ragged chunk, widths that are no multiple of a tile, fp32 stream, the pre-activation kept for training
        {"name": "linear_odd", "op": "linear", "rows": 331, "K": 1056, "N": 1000, "act": "gelu", "bias": "f32",
         "res": "f32", "pre": True},
        # a prefill or training chunk of the benchmark
        {"name": "linear_8192", "op": "linear", "rows": 8192, "K": 7168, "N": 3584, "act": "silu", "bias": "f32",
         "res": "none", "pre": True},
        # gradients of a small ragged layer
        {"name": "linear_back_odd", "op": "linear_back", "rows": 333, "K": 1056, "N": 1000, "act": "gelu",
         "bias": True},
        # gradients of the latent -> hidden projection for a training chunk
        {"name": "linear_back_4096", "op": "linear_back", "rows": 4096, "K": 3584, "N": 7168, "act": "silu",
         "bias": True},
        # one token of the residual stream
        {"name": "ln_1", "op": "ln", "T": 1, "H": 7168, "x": "bf16", "bias": True, "stats": False},
        # a training chunk of an fp32 stream, statistics kept for the gradient
        {"name": "ln_8192", "op": "ln", "T": 8192, "H": 7168, "x": "f32", "bias": True, "stats": True},
        # gradients at the latent width, odd row count, added to the fp32 stream's own gradient
        {"name": "ln_back_1001", "op": "ln_back", "T": 1001, "H": 3584, "x": "f32", "add": True},
        # gradients of a training chunk in bf16
        {"name": "ln_back_8192", "op": "ln_back", "T": 8192, "H": 7168, "x": "bf16", "add": True},
        # losses, counts and the router's whole gradient for a handful of tokens
        {"name": "balance_64", "op": "balance", "T": 64, "E": 896, "k": 16, "mask": False, "grad": True, "gate": True},
        # the same for the benchmark's largest batch, padded sequences among it
        {"name": "balance_32768", "op": "balance", "T": 32768, "E": 896, "k": 16, "mask": True, "grad": True,
         "gate": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_back", "ln", "ln_back", "balance"])
    if op in ("linear", "linear_back"):
        rows, K, N = _log(rng, 1, 8192), 8 * _log(rng, 8, 896), _log(rng, 64, 8192)
        rows = max(1, min(rows, int((2.0e11 if op == "linear" else 1.0e11) / (K * N))))
        c = {"op": op, "rows": rows, "K": K, "N": N, "act": rng.choice(ACTS)}
        if op == "linear":
            c.update(bias=rng.choice(["none", "f32", "bf16"]), res=rng.choice(["none", "bf16", "f32"]),
                     pre=rng.random() < 0.4)
        else:
            c.update(bias=rng.random() < 0.7)
        return c
    if op in ("ln", "ln_back"):
        c = {"op": op, "T": _log(rng, 1, 8192), "H": 8 * _log(rng, 16, 1024), "x": rng.choice(["bf16", "f32"])}
        if op == "ln":
            c.update(bias=rng.random() < 0.7, stats=rng.random() < 0.6)
        else:
            c.update(add=rng.random() < 0.6)
        return c
    E = _log(rng, 4, 2048)
    T = max(1, min(_log(rng, 1, 32768), 29000000 // E))
    grad = rng.random() < 0.75
    return {"op": op, "T": T, "E": E, "k": rng.randint(1, min(E, 16)), "mask": rng.random() < 0.5, "grad": grad,
            "gate": grad and rng.random() < 0.7}


# ---- inputs --------------------------------------------------------------------------

def _randn(g, *shape, dtype=torch.bfloat16, scale=1.0):
    return torch.randn(*shape, device=DEV, generator=g).mul_(scale).to(dtype)


TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    st = {"op": op, "case": dict(case)}
    if op in ("linear", "linear_back"):
        rows, K, N = case["rows"], case["K"], case["N"]
        st["x"], st["W"], st["act"] = _randn(g, rows, K), _randn(g, N, K, scale=K ** -0.5), case["act"]
        if op == "linear":
            st["bias"] = None if case["bias"] == "none" else _randn(g, N, dtype=TYPES[case["bias"]], scale=0.3)
            st["res"] = None if case["res"] == "none" else _randn(g, rows, N, dtype=TYPES[case["res"]], scale=2.0)
        else:
            # pre-activations are of order one, as stored by the forward pass
            st["pre"] = None if case["act"] == "none" else _randn(g, rows, N)
            st["dout"] = _randn(g, rows, N, scale=0.02)
        return st
    if op in ("ln", "ln_back"):
        T, H, dt = case["T"], case["H"], TYPES[case["x"]]
        # a residual stream: rows of different size and offset, a few outlier channels
        amp = torch.exp(0.5 * torch.randn(T, 1, device=DEV, generator=g))
        chan = 1 + 20 * (torch.rand(H, device=DEV, generator=g) < 0.002)
        shift = 0.3 * torch.randn(T, 1, device=DEV, generator=g)
        st["x"] = (torch.randn(T, H, device=DEV, generator=g) * amp * chan + shift).to(dt)
        st["w"] = 1 + 0.1 * torch.randn(H, device=DEV, generator=g)
        if op == "ln":
            st["b"] = 0.1 * torch.randn(H, device=DEV, generator=g) if case["bias"] else None
            st["stats"] = case["stats"]
        else:
            st["dy"] = _randn(g, T, H, scale=0.05)
            st["add"] = _randn(g, T, H, dtype=dt, scale=0.05) if case["add"] else None
            # what the forward pass kept: every row's mean and 1/sqrt(variance + eps)
            x = st["x"].double()
            m = x.mean(1)
            st["mean"] = m.float()
            st["rstd"] = (((x - m[:, None]) ** 2).mean(1) + EPS).rsqrt().float()
        return st
    T, E, k = case["T"], case["E"], case["k"]
    # a router in training: some experts more popular than others
    logits = torch.randn(T, E, device=DEV, generator=g) + 0.5 * torch.randn(E, device=DEV, generator=g)
    top, idx = logits.topk(k, dim=1)
    st["logits"], st["idx"] = logits, idx.to(torch.int32).contiguous()
    st["mask"] = None
    if case["mask"]:  # sequences of a batch, padded behind their ends: about a tenth of the tokens
        S = min(T, 64)
        L = -(-T // S)
        ends = L - (torch.rand(S, device=DEV, generator=g) ** 4 * L).long()
        m = (torch.arange(L, device=DEV) < ends[:, None]).reshape(-1)[:T].contiguous()
        m[0] = True
        st["mask"] = m
    st["grad"], st["w"], st["dw"] = case["grad"], None, None
    if case["gate"]:
        st["w"] = torch.softmax(top, 1).contiguous()
        st["dw"] = 1e-3 * torch.randn(T, k, device=DEV, generator=g)
    return st


# ---- one pass ------------------------------------------------------------------------

def _workspace(st, need):
    ws = st.get("ws")
    if ws is None:
        ws = st["ws"] = torch.zeros(max(need(), 256), dtype=torch.uint8, device=DEV)
    return ws


def _run_own(st):
    from top_routing_mxfp4_gb300 import lmoe
    op = st["op"]
    if op == "linear":
        x, W = st["x"], st["W"]
        ws = _workspace(st, lambda: lmoe.linear_act_workspace_size(x.shape[0], x.shape[1], W.shape[0]))
        return lmoe.linear_act_bf16(x, W, bias=st["bias"], act=st["act"], res=st["res"], pre=st["case"]["pre"], ws=ws)
    if op == "linear_back":
        x, W = st["x"], st["W"]
        ws = _workspace(st, lambda: lmoe.linear_act_backward_workspace_size(x.shape[0], x.shape[1], W.shape[0]))
        dx, dW, db = lmoe.linear_act_bf16_backward(st["dout"], x, W, act=st["act"], pre=st["pre"],
                                                   want_dbias=st["case"]["bias"], ws=ws)
        return [dx, dW] if db is None else [dx, dW, db]
    if op == "ln":
        return lmoe.layer_norm(st["x"], st["w"], st["b"], EPS, stats=st["stats"])
    if op == "ln_back":
        x = st["x"]
        ws = _workspace(st, lambda: lmoe.layer_norm_backward_workspace_size(x.shape[0], x.shape[1]))
        return lmoe.layer_norm_backward(st["dy"], x, st["mean"], st["rstd"], st["w"], add=st["add"], ws=ws)
    T, E = st["logits"].shape
    ws = _workspace(st, lambda: lmoe.balance_loss_workspace_size(T, E, st["idx"].shape[1]))
    return lmoe.balance_loss(st["logits"], st["idx"], mask=st["mask"], coef=COEF, grad=st["grad"], topk_w=st["w"],
                             dtopk_w=st["dw"], ws=ws)


def _act(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * torch.erfc(z * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        s = 1 / (1 + torch.exp(-c * (z + 0.044715 * z * z * z)))
        return s + z * s * (1 - s) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _run_plain(st):
    op = st["op"]
    if op == "linear":
        z = st["x"].float() @ st["W"].float().t()
        if st["bias"] is not None:
            z = z + st["bias"].float()
        out = _act(z, st["act"])
        if st["res"] is not None:
            out = out + st["res"].float()
        out = out.to(torch.bfloat16 if st["res"] is None else st["res"].dtype)
        return (out, z.to(torch.bfloat16)) if st["case"]["pre"] else out
    if op == "linear_back":
        dz = st["dout"].float()
        if st["pre"] is not None:
            dz = dz * _act_slope(st["pre"].float(), st["act"])
        out = [(dz @ st["W"].float()).to(torch.bfloat16), (dz.t() @ st["x"].float()).to(torch.bfloat16)]
        return out + [dz.sum(0)] if st["case"]["bias"] else out
    if op == "ln":
        x = st["x"].float()
        m = x.mean(1, keepdim=True)
        c = x - m
        rs = torch.rsqrt((c * c).mean(1, keepdim=True) + EPS)
        y = c * rs * st["w"]
        if st["b"] is not None:
            y = y + st["b"]
        y = y.to(torch.bfloat16)
        return (y, m[:, 0], rs[:, 0]) if st["stats"] else y
    if op == "ln_back":
        dy, rs = st["dy"].float(), st["rstd"][:, None]
        xh = (st["x"].float() - st["mean"][:, None]) * rs
        g = dy * st["w"]
        dx = rs * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
        if st["add"] is not None:
            dx = dx + st["add"].float()
        return dx.to(st["x"].dtype), (dy * xh).sum(0), dy.sum(0)
    l, idx = st["logits"], st["idx"].long()
    T, E = l.shape
    k = idx.shape[1]
    keep = torch.ones(T, dtype=torch.bool, device=l.device) if st["mask"] is None else st["mask"]
    n = keep.sum()
    counts = torch.zeros(E, dtype=torch.int32, device=l.device)
    counts.index_add_(0, idx.reshape(-1), keep[:, None].expand(T, k).reshape(-1).to(torch.int32))
    top = l.max(1, keepdim=True).values
    e = torch.exp(l - top)
    s = e.sum(1, keepdim=True)
    lse = (top + torch.log(s)) * keep[:, None]
    p = e / s * keep[:, None]
    f = counts.float() * E / (k * n)
    probs = p.sum(0) / n
    loss = torch.stack([(f * probs).sum(), (lse * lse).sum() / n])
    if not st["grad"]:
        return loss, counts, probs
    d = p * ((f - (p * f).sum(1, keepdim=True)) * (COEF[0] / n) + lse * (2 * COEF[1] / n))
    if st["w"] is not None:
        w, dw = st["w"], st["dw"]
        d.scatter_add_(1, idx, w * (dw - (w * dw).sum(1, keepdim=True)) * keep[:, None])
    return loss, counts, probs, d


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- the definition in 64 bits -------------------------------------------------------

def _phi(z):  # the normal distribution function, without the cancellation of 1 + erf
    return torch.special.erfc(-z / 2 ** 0.5) / 2


def exact(case, seed):
    st = prepare(case, seed)
    op, D = st["op"], torch.float64
    if op in ("linear", "linear_back"):
        act = case["act"]
        z = st["pre"].to(D) if op == "linear_back" and act != "none" else None
        if op == "linear":
            z = torch.mm(st["x"].to(D), st["W"].to(D).t())
            if case["bias"] != "none":
                z += st["bias"].to(D)
            a = {"none": lambda: z, "relu": lambda: torch.where(z > 0, z, 0 * z), "silu": lambda: z * torch.sigmoid(z),
                 "gelu": lambda: z * _phi(z),
                 "gelu_tanh": lambda: z * torch.sigmoid((8 / math.pi) ** 0.5 * z * (1 + 0.044715 * z ** 2))}[act]()
            if case["res"] != "none":
                a = a + st["res"].to(D)
            return (a, z) if case["pre"] else a
        dz = st["dout"].to(D)
        if act == "relu":
            dz = torch.where(z > 0, dz, 0 * dz)
        elif act == "silu":
            s = torch.sigmoid(z)
            dz = dz * (s + z * s * torch.sigmoid(-z))
        elif act == "gelu":
            dz = dz * (_phi(z) + z * torch.exp(-z ** 2 / 2) / (2 * math.pi) ** 0.5)
        elif act == "gelu_tanh":
            c = (8 / math.pi) ** 0.5
            u = c * z * (1 + 0.044715 * z ** 2)
            s = torch.sigmoid(u)
            dz = dz * (s + z * s * torch.sigmoid(-u) * c * (1 + 0.134145 * z ** 2))
        out = [torch.mm(dz, st["W"].to(D)), torch.mm(dz.t(), st["x"].to(D))]
        return out + [dz.sum(0)] if case["bias"] else out
    if op == "ln":
        x = st["x"].to(D)
        mean, var = x.mean(1), x.var(1, unbiased=False)
        rstd = 1 / (var + EPS).sqrt()
        y = (x - mean[:, None]) * rstd[:, None] * st["w"].to(D) + (st["b"].to(D) if case["bias"] else 0)
        return (y, mean, rstd) if case["stats"] else y
    if op == "ln_back":
        H = case["H"]
        dy, rstd = st["dy"].to(D), st["rstd"].to(D)[:, None]
        n = (st["x"].to(D) - st["mean"].to(D)[:, None]) * rstd
        dn = dy * st["w"].to(D)
        dx = (dn - (dn.sum(1, keepdim=True) + n * (dn * n).sum(1, keepdim=True)) / H) * rstd
        if case["add"]:
            dx += st["add"].to(D)
        return dx, (n * dy).sum(0), dy.sum(0)
    T, E, k = case["T"], case["E"], case["k"]
    keep = st["mask"] if case["mask"] else torch.ones(T, dtype=torch.bool, device=DEV)
    rows = keep.nonzero()[:, 0]
    n = len(rows)
    counts = torch.bincount(st["idx"][rows].reshape(-1), minlength=E)
    l = st["logits"][rows].to(D)
    p, lse = torch.softmax(l, 1), torch.logsumexp(l, 1)
    f = counts.to(D) * (E / (k * n))
    probs = p.mean(0)
    loss = torch.stack([f @ probs, (lse ** 2).mean()])
    counts = counts.to(torch.int32)
    if not case["grad"]:
        return loss, counts, probs
    d = p * (f - (p @ f)[:, None]) * (COEF[0] / n) + p * lse[:, None] * (2 * COEF[1] / n)
    if case["gate"]:
        w, dw = st["w"][rows].to(D), st["dw"][rows].to(D)
        d.scatter_add_(1, st["idx"][rows].long(), w * dw - w * (w * dw).sum(1, keepdim=True))
    out = torch.zeros(T, E, dtype=D, device=DEV)
    out[rows] = d
    return loss, counts, probs, out


# ---- what a pass cannot do without ---------------------------------------------------

def work(case):
    op = case["op"]
    size = {"none": 0, "bf16": 2, "f32": 4}
    if op in ("linear", "linear_back"):
        r, K, N = case["rows"], case["K"], case["N"]
        if op == "linear":
            out = size[case["res"]] or 2
            by = 2 * (r * K + N * K) + N * size[case["bias"]] + r * N * (size[case["res"]] + out + 2 * case["pre"])
            return {"bytes": by, "flops": 2 * r * K * N}
        by = 4 * (r * K + N * K) + r * N * (2 if case["act"] == "none" else 4) + 4 * N * case["bias"]
        return {"bytes": by, "flops": 4 * r * K * N}
    if op in ("ln", "ln_back"):
        n, H, s = case["T"] * case["H"], case["H"], size[case["x"]]
        if op == "ln":
            return {"bytes": n * (s + 2) + 4 * H * (1 + case["bias"]) + 8 * case["T"] * case["stats"], "flops": 8 * n}
        return {"bytes": n * (2 + 2 * s + s * case["add"]) + 12 * H + 8 * case["T"], "flops": 14 * n}
    T, E, k = case["T"], case["E"], case["k"]
    by = T * E * 4 * (1 + case["grad"]) + 4 * T * k * (1 + 2 * case["gate"]) + T * case["mask"] + 8 * E
    return {"bytes": by, "flops": T * E * (12 if case["grad"] else 6)}
