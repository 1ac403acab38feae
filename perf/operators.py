"""Workloads of the operators around the LatentMoE layer: norms with gate and residual, MXFP4 linear layers on bf16
rows, and bf16 products grouped by expert.

`run` computes a case in plain torch operations, or, where `own` is true, by the library's calls.
"""
import math

import torch

own = False
DEV = "cuda"
EPS = 1e-5


# ---- cases ---------------------------------------------------------------------------

def listed():
    return [
        # MXFP4 projections hidden <-> latent.  One token: latent 3584 -> hidden 7168.
        {"name": "linear_1", "op": "linear", "rows": 1, "K": 3584, "N": 7168},
        # a handful of tokens (short speculative drafts): hidden -> latent
        {"name": "linear_7", "op": "linear", "rows": 7, "K": 7168, "N": 3584},
        # the decode batch of the benchmark
        {"name": "linear_64", "op": "linear", "rows": 64, "K": 7168, "N": 3584},
        # widths that are no multiple of a tile, a ragged prefill chunk
        {"name": "linear_odd", "op": "linear", "rows": 331, "K": 1056, "N": 1000},
        # the residual stream around the block: one token, then norm of the next block
        {"name": "norm_1", "op": "norm", "T": 1, "H": 7168, "res": "bf16", "post": True, "gate": "channel", "next": True},
        # decode batch, fp32 stream, gate per token
        {"name": "norm_64", "op": "norm", "T": 64, "H": 7168, "res": "f32", "post": True, "gate": "token", "next": True},
        # prefill chunk, element-wise gate, stream in bf16
        {"name": "norm_8192", "op": "norm", "T": 8192, "H": 7168, "res": "bf16", "post": True, "gate": "full", "next": True},
        # norm before a block only, latent width, odd row count
        {"name": "prenorm_1001", "op": "prenorm", "T": 1001, "H": 3584, "res": "f32"},
        # bf16 experts, one token: 16 of 896 experts' gate and up matrices
        {"name": "swiglu_1", "op": "swiglu", "T": 1, "E": 896, "k": 16, "K": 3584, "N": 512, "skew": False},
        # decode batch: weighted down projection into per-pair fp32 rows
        {"name": "down_64", "op": "grouped", "T": 64, "E": 896, "k": 16, "K": 512, "N": 3584, "skew": False},
        # prefill chunk: gate and up of every expert, about 146 rows each
        {"name": "swiglu_8192", "op": "swiglu", "T": 8192, "E": 896, "k": 16, "K": 3584, "N": 512, "skew": False},
        # few, wide experts with a skewed load: compute-bound
        {"name": "grouped_skew", "op": "rows", "T": 4096, "E": 24, "k": 2, "K": 2048, "N": 4104, "skew": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "norm", "prenorm", "swiglu", "grouped", "rows"])
    if op == "linear":
        return {"op": op, "rows": _log(rng, 1, 512), "K": 32 * _log(rng, 8, 256), "N": _log(rng, 64, 8192)}
    if op in ("norm", "prenorm"):
        c = {"op": op, "T": _log(rng, 1, 8192), "H": 8 * _log(rng, 16, 1024), "res": rng.choice(["bf16", "f32"])}
        if op == "norm":
            c.update(post=rng.random() < 0.75, gate=rng.choice(["none", "channel", "token", "full"]),
                     next=rng.random() < 0.75)
        return c
    E = _log(rng, 4, 512)
    # widths of a few hundred to a few thousand; the bank and the products stay under the listed ones
    K, N = 8 * _log(rng, 32, 512), 8 * _log(rng, 16, 512)
    while E * K * N > 1.2e9:
        K, N = max(256, K // 16 * 8), max(128, N // 16 * 8)
    k = rng.randint(1, min(E, 16))
    T = max(1, min(_log(rng, 1, 8192), 120000 // k, int(2.3e11 / (k * K * N))))
    return {"op": op, "T": T, "E": E, "k": k, "K": K, "N": N, "skew": rng.random() < 0.3 and E <= 64}


# ---- inputs --------------------------------------------------------------------------

def _randn(g, *shape, dtype=torch.bfloat16, scale=1.0):
    return torch.randn(*shape, device=DEV, dtype=torch.float32 if math.prod(shape) < 1 << 28 else dtype,
                       generator=g).mul_(scale).to(dtype)


def _scale_atoms(sc):
    """E8M0 bytes [N][K/32] in the 512-byte atoms of the tensor-core layout: one atom per 128 rows x 128 columns."""
    N, B = sc.shape
    RT, KC = -(-N // 128), -(-B // 4)
    full = torch.zeros(RT * 128, KC * 4, dtype=torch.uint8, device=sc.device)
    full[:N, :B] = sc
    # row 32*j + i of an atom, block b at byte 16*i + 4*j + b
    return full.view(RT, 4, 32, KC, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op = case["op"]
    if op == "linear":
        rows, K, N = case["rows"], case["K"], case["N"]
        Kp = -(-K // 128) * 128
        q = torch.randint(0, 256, (N, Kp // 2), device=DEV, dtype=torch.uint8, generator=g)
        q[:, K // 2:] = 0
        # scale bytes as a checkpoint of this fan-in has them: weights of about 1/sqrt(K), a spread of a few octaves
        mid = 127 - int(round(math.log2(3 * math.sqrt(K))))
        sc = torch.randint(mid - 2, mid + 2, (N, K // 32), device=DEV, generator=g).to(torch.uint8)
        x = _randn(g, rows, K)
        return {"op": op, "x": x, "q": q.view(-1), "s": _scale_atoms(sc), "K": K, "N": N}
    if op in ("norm", "prenorm"):
        T, H = case["T"], case["H"]
        dt = torch.float32 if case["res"] == "f32" else torch.bfloat16
        # a residual stream: rows of different size, a few outlier channels
        amp = torch.exp(0.5 * torch.randn(T, 1, device=DEV, generator=g))
        chan = 1 + 20 * (torch.rand(H, device=DEV, generator=g) < 0.002)
        st = {"op": op, "r": (torch.randn(T, H, device=DEV, generator=g) * amp * chan).to(dt)}
        st["next_w"] = 1 + 0.1 * torch.randn(H, device=DEV, generator=g)
        if op == "prenorm":
            return st
        st["y"] = (torch.randn(T, H, device=DEV, generator=g) * amp * 0.3).to(torch.bfloat16)
        st["post_w"] = 1 + 0.1 * torch.randn(H, device=DEV, generator=g) if case["post"] else None
        st["next_w"] = st["next_w"] if case["next"] else None
        st["gate"] = {"none": lambda: None,
                      "channel": lambda: 0.5 + 0.1 * torch.randn(H, device=DEV, generator=g),
                      "token": lambda: torch.rand(T, 1, device=DEV, generator=g),
                      "full": lambda: torch.rand(T, H, device=DEV, generator=g).to(torch.bfloat16)}[case["gate"]]()
        st["scale"] = 0.22
        return st
    T, E, k, K, N = (case[n] for n in ("T", "E", "k", "K", "N"))
    P = T * k
    score = torch.rand(T, E, device=DEV, generator=g).log().neg().log().neg()  # Gumbel: top-k without replacement
    if case["skew"]:
        score = score - 1.2 * torch.log(torch.arange(1, E + 1, device=DEV).float())[torch.randperm(E, device=DEV, generator=g)]
    idx = score.topk(k, dim=1).indices
    flat = idx.reshape(-1)
    perm = torch.sort(flat, stable=True).indices.to(torch.int32)
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(counts, 0).to(torch.int32)
    st = {"op": op, "offsets": offsets, "perm": perm, "k": k, "most": int(counts.max())}
    st["W"] = _randn(g, E, N, K, scale=K ** -0.5)
    if op == "swiglu":
        st["U"] = _randn(g, E, N, K, scale=K ** -0.5)
    if op == "grouped":  # rows already in expert order (the gated product), a gate weight for each pair
        st["x"] = _randn(g, P, K)
        st["w"] = torch.softmax(torch.randn(T, k, device=DEV, generator=g), 1).contiguous()
    else:
        st["x"] = _randn(g, T, K)
    return st


# ---- one pass ------------------------------------------------------------------------

def _workspace(st, need):
    ws = st.get("ws")
    if ws is None or ws.numel() < need:
        ws = st["ws"] = torch.zeros(max(need, 256), dtype=torch.uint8, device=DEV)
    return ws


def _run_own(st):
    from top_routing_mxfp4_gb300 import lmoe
    op = st["op"]
    if op == "linear":
        x, N = st["x"], st["N"]
        ws = st.get("ws")
        if ws is None:
            ws = _workspace(st, lmoe.linear_mxfp4_workspace_size(x.shape[0], st["K"], N))
        return lmoe.linear_mxfp4(x, st["q"], st["s"], N, ws=ws)
    if op == "prenorm":
        return lmoe.rms_norm(st["r"], st["next_w"], EPS)
    if op == "norm":
        r, n = lmoe.residual_norm(st["y"], st["r"], post_w=st["post_w"], gate=st["gate"], scale=st["scale"],
                                  next_w=st["next_w"], eps=EPS)
        return [r] if n is None else [r, n]
    ws = st.get("ws")
    if ws is None:
        ws = _workspace(st, lmoe.grouped_workspace_size())
    if op == "swiglu":
        return lmoe.grouped_swiglu_bf16(st["x"], st["W"], st["U"], st["offsets"], st["perm"], st["k"], ws=ws)
    if op == "grouped":
        return lmoe.grouped_linear_bf16(st["x"], st["W"], st["offsets"], st["perm"], st["k"], gather=False,
                                        row_w=st["w"], ws=ws)
    return lmoe.grouped_linear_bf16(st["x"], st["W"], st["offsets"], st["perm"], st["k"], ws=ws)


def _dequant(q, s, N, K):
    Kp = -(-K // 128) * 128
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=q.device)
    b = q.view(N, Kp // 2)
    v = grid[torch.stack([b & 15, b >> 4], -1).view(N, Kp).long()]
    RT, KC = -(-N // 128), Kp // 128
    e = s.view(RT, KC, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(RT * 128, KC * 4)[:N]
    sc = torch.exp2(e.float() - 127)
    return (v.view(N, Kp // 32, 32) * sc[..., None]).view(N, Kp)[:, :K]


def _rms(v, w):
    return v * torch.rsqrt((v * v).mean(-1, keepdim=True) + EPS) * w


def _products(x, mats, st):
    """x rows (fp32) in expert order against each row's own matrix; one fp32 [P][N] tensor for each bank in mats."""
    P, E = x.shape[0], mats[0].shape[0]
    off = st["offsets"].long()
    q = torch.arange(P, device=x.device)
    e = torch.searchsorted(off[1:].contiguous(), q, right=True)
    if P <= E // 4:  # few rows: only their experts' matrices are read
        return [torch.matmul(W[e].float(), x[:, :, None])[:, :, 0] for W in mats]
    most = st["most"]
    at = (off[:-1, None] + torch.arange(most, device=x.device)).clamp_(max=P - 1)
    xb = x[at]  # padded to the longest group; rows of the next group in the padding are not taken back
    return [torch.bmm(xb, W.float().transpose(1, 2))[e, q - off[e]] for W in mats]


def _run_plain(st):
    op = st["op"]
    if op == "linear":
        return (st["x"].float() @ _dequant(st["q"], st["s"], st["N"], st["K"]).t()).to(torch.bfloat16)
    if op == "prenorm":
        return _rms(st["r"].float(), st["next_w"]).to(torch.bfloat16)
    if op == "norm":
        y, g = st["y"].float(), st["gate"]
        if st["post_w"] is not None:
            y = _rms(y, st["post_w"])
        if g is not None:
            y = y * g.float()
        r = (st["r"].float() + st["scale"] * y).to(st["r"].dtype)
        return [r] if st["next_w"] is None else [r, _rms(r.float(), st["next_w"]).to(torch.bfloat16)]
    perm = st["perm"].long()
    if op == "grouped":
        (y,) = _products(st["x"].float(), [st["W"]], st)
        return y * st["w"].view(-1)[perm][:, None]
    x = st["x"][perm // st["k"]].float()
    if op == "rows":
        return _products(x, [st["W"]], st)[0].to(torch.bfloat16)
    a, b = _products(x, [st["W"], st["U"]], st)
    return (a / (1 + torch.exp(-a)) * b).to(torch.bfloat16)


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---- the definition in 64 bits -------------------------------------------------------

def exact(case, seed):
    st = prepare(case, seed)
    op, D = st["op"], torch.float64
    if op == "linear":
        N, K = st["N"], st["K"]
        Kp, KC = -(-K // 128) * 128, -(-K // 128)
        n = torch.arange(N, device=DEV)[:, None]
        c = torch.arange(K, device=DEV)[None, :]
        byte = st["q"].long()[n * (Kp // 2) + c // 2]
        code = (byte >> (4 * (c & 1))) & 15
        ex, m = (code >> 1) & 3, (code & 1).to(D)
        mag = torch.where(ex == 0, 0.5 * m, (1 + 0.5 * m) * torch.exp2(ex.to(D) - 1))
        r, blk = n % 128, c // 32
        sb = st["s"].long()[((n // 128) * KC + blk // 4) * 512 + 16 * (r % 32) + 4 * (r // 32) + blk % 4]
        W = torch.where(code >= 8, -mag, mag) * torch.exp2(sb.to(D) - 127)
        return st["x"].to(D) @ W.t()
    if op == "prenorm":
        v = st["r"].to(D)
        return v / (v.square().sum(1, keepdim=True) / v.shape[1] + EPS).sqrt() * st["next_w"].to(D)
    if op == "norm":
        y = st["y"].to(D)
        if case["post"]:
            y = y / (y.square().sum(1, keepdim=True) / y.shape[1] + EPS).sqrt() * st["post_w"].to(D)
        if case["gate"] != "none":
            y = y * st["gate"].to(D)
        r = st["r"].to(D) + st["scale"] * y
        if not case["next"]:
            return [r]
        v = r.to(st["r"].dtype).to(D)  # the stored stream is what the next norm reads
        return [r, v / (v.square().sum(1, keepdim=True) / v.shape[1] + EPS).sqrt() * st["next_w"].to(D)]
    off, perm = st["offsets"].tolist(), st["perm"].long()
    if 2 * case["T"] * case["k"] * case["K"] * case["N"] * (2 if op == "swiglu" else 1) > 4e12:
        return None
    out = torch.empty(len(perm), case["N"], dtype=D, device=DEV)
    for e in range(case["E"]):
        a, b = off[e], off[e + 1]
        if a == b:
            continue
        x = (st["x"][a:b] if op == "grouped" else st["x"][perm[a:b] // st["k"]]).to(D)
        y = x @ st["W"][e].to(D).t()
        if op == "grouped":
            y = y * st["w"].reshape(-1)[perm[a:b]].to(D)[:, None]
        if op == "swiglu":
            y = y * torch.sigmoid(y) * (x @ st["U"][e].to(D).t())
        out[a:b] = y
    return out


# ---- what a pass cannot do without ---------------------------------------------------

def work(case):
    op = case["op"]
    if op == "linear":
        r, K, N = case["rows"], case["K"], case["N"]
        return {"bytes": N * K * 17 // 32 + 2 * r * (K + N), "flops": 2 * r * K * N}
    if op in ("norm", "prenorm"):
        n, H = case["T"] * case["H"], case["H"]
        rb = 4 if case["res"] == "f32" else 2
        if op == "prenorm":
            return {"bytes": n * (rb + 2) + 4 * H, "flops": 4 * n}
        by = n * (2 + 2 * rb + (2 if case["next"] else 0)) + 4 * H * (bool(case["post"]) + bool(case["next"]))
        by += {"none": 0, "channel": 4 * H, "token": 4 * case["T"], "full": 2 * n}[case["gate"]]
        return {"bytes": by, "flops": 10 * n}
    T, E, k, K, N = (case[n] for n in ("T", "E", "k", "K", "N"))
    P, mats = T * k, 2 if op == "swiglu" else 1
    touched = E * (1 - (1 - k / E) ** T)  # expected, at a uniform load
    rows = P * K if op == "grouped" else T * K
    return {"bytes": int(touched * mats * N * K * 2) + 2 * rows + P * N * (4 if op == "grouped" else 2) + 4 * P,
            "flops": 2 * P * mats * N * K}
