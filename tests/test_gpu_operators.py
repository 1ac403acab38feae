"""Norms around the block, the MXFP4 linear on bf16 rows and the bf16 products
grouped by expert, against plain torch in 64 bits.

Tolerances (u = 2^-24, half a step of fp32; a bf16 result is off by at most
half a step, 2^-8 of its value):
  norms      a row's sum of squares is fp32 with at most 64 + 11 additions on
             any element's way and one rounding per square, so its relative
             error is below 80 u and that of rsqrt(mean + eps) below 44 u with
             the division, the add and the root's own rounding; three more
             products: below 64 u in all.
  products   every product and every sum in the accumulation is rounded at
             most once, in any order: |error| <= (K + 2) u sum_c |x_c w_c|
             (each term passes at most K additions).  The MXFP4 linear may
             hold x as two 8-bit parts, within 2^-22 of its 32-block's largest
             magnitude, which adds 2^-22 sum_blocks amax sum |w|.
  silu       the exponential, the add and the division: below 16 u of h.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
HALF = 2.0 ** -8  # half a bf16 step, relative
D = torch.float64


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def randn(g, *shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(*shape, device=DEV, generator=g) * scale).to(dtype)


def guarded(shape, dtype, fill=77.0):
    """A tensor with a sentinel row of 64 elements before and behind it, and the check that they stay."""
    n = int(np.prod(shape))
    buf = torch.full((n + 128,), fill, dtype=dtype, device=DEV)
    view = buf[64:64 + n].view(shape)

    def intact():
        return bool((buf[:64] == fill).all()) and bool((buf[64 + n:] == fill).all())

    return view, intact


def within(got, ref, tol):
    got = got.to(D)
    assert bool(torch.isfinite(got).all())
    bad = (got - ref).abs() > tol
    assert not bool(bad.any()), f"{int(bad.sum())} of {bad.numel()} beyond the bound, worst {float(((got - ref).abs() / tol.clamp_min(1e-300)).max()):.2f}x"


# ---- norms --------------------------------------------------------------------------

def norm_ref(v, w, eps):
    return v / (v.square().mean(1, keepdim=True) + eps).sqrt() * w.to(D)


@pytest.mark.parametrize("T,H", [(1, 8), (1, 7168), (3, 40), (5, 256), (4, 264), (2500, 520), (2, 1024), (3, 1032),
                                 (7, 4104), (400, 7168), (305, 3584), (2, 8192), (3, 8200), (2, 16384), (2, 32768)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_rms_norm(cuda_lib, T, H, dt):
    g = gen(T * 7 + H)
    x = randn(g, T, H, dtype=dt, scale=3.0)
    w = randn(g, H, dtype=torch.float32)
    out, intact = guarded((T, H), torch.bfloat16)
    cuda_lib.rms_norm(x, w, 1e-5, out=out)
    ref = norm_ref(x.to(D), w, 1e-5)
    within(out, ref, ref.abs() * (HALF + 64 * U) * (1 + HALF))
    assert intact()


@pytest.mark.parametrize("T,H", [(1, 7168), (64, 7168), (3, 72), (9, 1000), (306, 2056), (2, 12288), (3000, 512)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gate", ["none", "channel", "token", "full"])
@pytest.mark.parametrize("post,nxt", [(True, True), (False, True), (True, False), (False, False)])
def test_residual_norm(cuda_lib, T, H, dt, gate, post, nxt):
    g = gen(T + H)
    y, res = randn(g, T, H, scale=0.7), randn(g, T, H, dtype=dt, scale=2.0)
    pw = randn(g, H, dtype=torch.float32) if post else None
    nw = randn(g, H, dtype=torch.float32) if nxt else None
    gt = {"none": None, "channel": randn(g, H, dtype=torch.float32), "token": randn(g, T, 1, dtype=torch.float32),
          "full": randn(g, T, H)}[gate]
    ro, intact_r = guarded((T, H), dt)
    no, intact_n = guarded((T, H), torch.bfloat16)
    r, n = cuda_lib.residual_norm(y, res, post_w=pw, gate=gt, scale=0.3, next_w=nw, eps=1e-6, res_out=ro,
                                  next_out=no if nxt else None)
    s = y.to(D) if pw is None else norm_ref(y.to(D), pw, 1e-6)
    add = float(np.float32(0.3)) * (s if gt is None else s * gt.to(D))
    ref = res.to(D) + add
    half = HALF if dt == torch.bfloat16 else U
    # the add's own fp32 rounding, the products' error, then the stored type's half step of the computed value
    tol = add.abs() * 64 * U + ref.abs() * U
    within(r, ref, tol + (ref.abs() + tol) * half)
    assert intact_r() and intact_n()
    if nxt:
        ref = norm_ref(r.to(D), nw, 1e-6)
        within(n, ref, ref.abs() * (HALF + 64 * U) * (1 + HALF))
    else:
        assert n is None


def test_residual_norm_in_place_and_zero_rows(cuda_lib):
    g = gen(5)
    T, H = 37, 7168
    y, res, w = randn(g, T, H), randn(g, T, H, dtype=torch.float32), randn(g, H, dtype=torch.float32)
    y[3] = 0
    res[5] = 0
    y[5] = 0
    a = cuda_lib.residual_norm(y, res, post_w=w, scale=0.5, next_w=w)
    y2, r2 = y.clone(), res.clone()
    cuda_lib.residual_norm(y2, r2, post_w=w, scale=0.5, next_w=w, res_out=r2, next_out=y2)
    assert torch.equal(a[0], r2) and torch.equal(a[1], y2)
    assert torch.equal(a[0][3], res[3])
    assert not bool(a[0][5].any()) and not bool(a[1][5].any())


def test_norm_of_a_row_with_a_nan_stays_in_that_row(cuda_lib):
    g = gen(6)
    y, res, w = randn(g, 9, 512), randn(g, 9, 512), randn(g, 512, dtype=torch.float32)
    clean = cuda_lib.residual_norm(y, res, post_w=w, next_w=w)
    y[4, 17] = float("nan")
    r, n = cuda_lib.residual_norm(y, res, post_w=w, next_w=w)
    keep = [i for i in range(9) if i != 4]
    assert bool(r[4].isnan().all()) and bool(n[4].isnan().all())
    assert torch.equal(r[keep], clean[0][keep]) and torch.equal(n[keep], clean[1][keep])


# ---- MXFP4 linear -------------------------------------------------------------------

GRID = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], dtype=D)


def mx_weights(lmoe, g, N, K, lo=-8, hi=-3):
    """Random canonical MXFP4 matrix -> (tensor-core codes, scales, the fp64 matrix)."""
    codes = torch.randint(0, 16, (N, K), device=DEV, generator=g)
    sc = torch.randint(127 + lo, 127 + hi, (N, K // 32), device=DEV, generator=g)
    W = GRID.to(DEV)[codes].view(N, K // 32, 32) * torch.exp2(sc.to(D) - 127)[..., None]
    q = (codes[:, 0::2] | (codes[:, 1::2] << 4)).to(torch.uint8).contiguous()
    qt, st = lmoe.repack_mxfp4(q, sc.to(torch.uint8).contiguous(), 1, N, K)
    return qt, st, W.view(N, K)


def linear_tol(x, W, ref):
    K = x.shape[1]
    ax, aw = x.to(D).abs(), W.abs()
    amax = ax.view(-1, K // 32, 32).amax(2, keepdim=True).expand(-1, -1, 32).reshape(-1, K)
    return ref.abs() * HALF + ((K + 2) * U * (ax @ aw.t()) + 2.0 ** -22 * (amax @ aw.t())) * (1 + HALF)


def check_linear(lmoe, x, W, q, s):
    rows, N = x.shape[0], W.shape[0]
    out, intact = guarded((rows, N), torch.bfloat16)
    ws = torch.zeros(lmoe.linear_mxfp4_workspace_size(rows, x.shape[1], N), dtype=torch.uint8, device=DEV)
    lmoe.linear_mxfp4(x, q, s, N, out=out, ws=ws)
    ref = x.to(D) @ W.t()
    within(out, ref, linear_tol(x, W, ref))
    assert lmoe.last_device_status(ws) == lmoe.OK
    assert intact()
    return out, ref


@pytest.mark.parametrize("rows", [1, 2, 7, 8, 9, 16, 17, 33, 64, 65, 130, 257])
@pytest.mark.parametrize("K,N", [(32, 16), (96, 7), (160, 129), (1056, 1000), (3584, 256)])
def test_linear_mxfp4(cuda_lib, rows, K, N):
    g = gen(rows * 31 + K + N)
    q, s, W = mx_weights(cuda_lib, g, N, K)
    out, ref = check_linear(cuda_lib, randn(g, rows, K), W, q, s)
    # as a whole the error is the output's rounding
    assert float((out.to(D) - ref).norm()) <= HALF * float(ref.norm())


@pytest.mark.parametrize("rows,K,N", [(1, 3584, 7168), (5, 7168, 3584), (64, 7168, 3584), (1, 64, 1), (3, 128, 20000),
                                      (1025, 512, 384), (40, 16384, 72)])
def test_linear_mxfp4_wide(cuda_lib, rows, K, N):
    g = gen(rows + K)
    q, s, W = mx_weights(cuda_lib, g, N, K)
    check_linear(cuda_lib, randn(g, rows, K), W, q, s)


# enough tiles that 128-row ones are taken: several a CTA, a long K, ragged rows and columns
@pytest.mark.parametrize("rows,K,N", [(161, 384, 14330), (383, 1632, 14337), (513, 7168, 2600), (1000, 1600, 2050)])
def test_linear_mxfp4_large_tiles(cuda_lib, rows, K, N):
    g = gen(rows + K + N)
    q, s, W = mx_weights(cuda_lib, g, N, K)
    check_linear(cuda_lib, randn(g, rows, K), W, q, s)


@pytest.mark.parametrize("rows", [3, 24])
def test_linear_mxfp4_keeps_every_bit_of_x(cuda_lib, rows):
    """One nonzero weight per output: out is x times it, exactly, for every
    element within 2^-14 of its block's largest, and within 2^-22 of that
    magnitude for the smallest ones."""
    K = 256
    g = gen(rows)
    x = randn(g, rows, K) * torch.exp2(torch.randint(-13, 1, (rows, K), device=DEV, generator=g)).to(torch.bfloat16)
    x[0, 64:96] = 0
    x[1, 100] = 2.0 ** 90
    x[2, 200] = 2.0 ** -120
    q = torch.zeros(K, K // 2, dtype=torch.uint8, device=DEV)
    c = torch.arange(K, device=DEV)
    q[c, c // 2] = torch.where(c % 2 == 0, 0x02, 0x20).to(torch.uint8)  # code 2 = 1.0 on the diagonal
    s = torch.full((K, K // 32), 127, dtype=torch.uint8, device=DEV)
    qt, st = cuda_lib.repack_mxfp4(q, s, 1, K, K)
    out = cuda_lib.linear_mxfp4(x, qt, st, K).to(D)
    xd = x.to(D)
    amax = xd.abs().view(rows, K // 32, 32).amax(2, keepdim=True).expand(-1, -1, 32).reshape(rows, K)
    near = xd.abs() >= amax * 2.0 ** -13
    assert torch.equal(out[near], xd[near])
    # the output's own rounding is exact or half a step of a value this small
    assert bool(((out - xd).abs() <= amax * 2.0 ** -22 + xd.abs() * HALF).all())


def test_linear_mxfp4_extreme_scales(cuda_lib):
    """Scale bytes from 0 to 254: products far below and far above 1."""
    g = gen(9)
    N, K, rows = 48, 128, 6
    codes = torch.randint(0, 16, (N, K), device=DEV, generator=g)
    sc = torch.randint(0, 255, (N, 1), device=DEV, generator=g).expand(N, K // 32).contiguous()
    sc[0], sc[1], sc[2] = 0, 254, 1
    W = (GRID.to(DEV)[codes].view(N, K // 32, 32) * torch.exp2(sc.to(D) - 127)[..., None]).view(N, K)
    q = (codes[:, 0::2] | (codes[:, 1::2] << 4)).to(torch.uint8).contiguous()
    qt, st = cuda_lib.repack_mxfp4(q, sc.to(torch.uint8), 1, N, K)
    x = randn(g, rows, K, scale=2.0 ** -8)
    out = cuda_lib.linear_mxfp4(x, qt, st, N).to(D)
    ref = x.to(D) @ W.t()
    # sums below fp32's normal range may be flushed: 2^-126 per term
    tol = linear_tol(x, W, ref) + K * 2.0 ** -126
    assert bool(((out - ref).abs() <= tol).all())


@pytest.mark.parametrize("rows", [4, 40])
def test_linear_mxfp4_nonfinite_rows_stay_apart(cuda_lib, rows):
    """A NaN or an infinity in a row of x makes that row's outputs NaN (an
    infinity may also stay one), and no other row's."""
    g = gen(11)
    q, s, W = mx_weights(cuda_lib, g, 200, 256)
    x = randn(g, rows, 256)
    clean = cuda_lib.linear_mxfp4(x, q, s, 200)
    x[1, 5], x[2, 250] = float("nan"), float("inf")
    out = cuda_lib.linear_mxfp4(x, q, s, 200)
    assert not bool(torch.isfinite(out[1]).any())
    assert not bool(torch.isfinite(out[2][W[:, 250] != 0]).any())
    keep = [i for i in range(rows) if i not in (1, 2)]
    assert torch.equal(out[keep], clean[keep])


# ---- products grouped by expert -----------------------------------------------------

def make_groups(counts, k, g):
    """Pairs of T tokens in expert order for the given counts (their sum a multiple of k)."""
    P = sum(counts)
    assert P % k == 0
    perm = torch.randperm(P, device=DEV, generator=g).to(torch.int32)
    off = torch.tensor([0] + list(np.cumsum(counts)), dtype=torch.int32, device=DEV)
    return off, perm, P // k


def grouped_ref(x, W, off, src):
    P, N = len(src), W.shape[1]
    y, mag = torch.zeros(P, N, dtype=D, device=DEV), torch.zeros(P, N, dtype=D, device=DEV)
    o = off.tolist()
    for e in range(W.shape[0]):
        a, b = o[e], o[e + 1]
        if a < b:
            xe = x[src[a:b]].to(D)
            y[a:b], mag[a:b] = xe @ W[e].to(D).t(), xe.abs() @ W[e].to(D).abs().t()
    return y, mag


COUNTS = {
    "one_row": [0, 1, 0],
    "decode": [1, 0, 2, 1, 0, 0, 3, 1, 16, 0, 17, 0, 1, 0, 6],
    "edges": [15, 16, 17, 31, 32, 33, 0, 127, 128, 129, 255, 256, 257, 0, 64],
    "one_big": [0, 0, 1000, 0],
    "last_empty": [40, 0, 0],
    "single": [48],
}


@pytest.mark.parametrize("name", list(COUNTS))
@pytest.mark.parametrize("K,N", [(8, 1), (72, 40), (200, 257), (1024, 128), (64, 136)])
def test_grouped_linear(cuda_lib, name, K, N):
    counts = COUNTS[name]
    k = 4 if sum(counts) % 4 == 0 else 1
    g = gen(K + N + len(counts))
    off, perm, T = make_groups(counts, k, g)
    P = T * k
    x, W = randn(g, T, K), randn(g, len(counts), N, K, scale=K ** -0.5)
    ws = torch.zeros(cuda_lib.grouped_workspace_size(), dtype=torch.uint8, device=DEV)
    out, intact = guarded((P, N), torch.bfloat16)
    cuda_lib.grouped_linear_bf16(x, W, off, perm, k, out=out, ws=ws)
    ref, mag = grouped_ref(x, W, off, (perm // k).long())
    acc = (K + 2) * U * mag
    within(out, ref, ref.abs() * HALF + acc * (1 + HALF))
    assert intact()
    # rows in expert order, weighted, fp32: the rows lmoe_combine takes
    xr, row_w = randn(g, P, K), torch.rand(P, device=DEV, generator=g)
    out32, intact = guarded((P, N), torch.float32)
    cuda_lib.grouped_linear_bf16(xr, W, off, perm, k, gather=False, row_w=row_w, out=out32, ws=ws)
    ref, mag = grouped_ref(xr, W, off, torch.arange(P, device=DEV))
    w = row_w.to(D)[perm.long()][:, None]
    within(out32, ref * w, ((K + 2) * U * mag * w + (ref * w).abs() * U) * (1 + U) + 1e-300)
    assert intact()
    # no permutation at all, fp32 rows
    o2 = cuda_lib.grouped_linear_bf16(xr, W, off, out=torch.empty(P, N, device=DEV), ws=ws)
    within(o2, ref, (K + 2) * U * mag + 1e-300)
    assert cuda_lib.last_device_status(ws) == cuda_lib.OK


@pytest.mark.parametrize("name", list(COUNTS))
@pytest.mark.parametrize("K,I", [(8, 1), (72, 40), (264, 200), (1024, 64), (128, 129)])
def test_grouped_swiglu(cuda_lib, name, K, I):
    counts = COUNTS[name]
    k = 2 if sum(counts) % 2 == 0 else 1
    g = gen(K + I)
    off, perm, T = make_groups(counts, k, g)
    P = T * k
    x = randn(g, T, K)
    Wg, Wu = (randn(g, len(counts), I, K, scale=2 * K ** -0.5) for _ in range(2))
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    out, intact = guarded((P, I), torch.bfloat16)
    cuda_lib.grouped_swiglu_bf16(x, Wg, Wu, off, perm, k, out=out, ws=ws)
    src = (perm // k).long()
    a, ma = grouped_ref(x, Wg, off, src)
    b, mb = grouped_ref(x, Wu, off, src)
    da, db = (K + 2) * U * ma, (K + 2) * U * mb
    s = a * torch.sigmoid(a)
    ref = s * b
    # |silu'| <= 1.1
    tol = 1.1 * da * (b.abs() + db) + (s.abs() + 1.1 * da) * db + 16 * U * ref.abs()
    within(out, ref, ref.abs() * HALF + tol * (1 + HALF) + 1e-300)
    assert intact()
    assert cuda_lib.last_device_status(ws) == cuda_lib.OK


@pytest.mark.parametrize("gather", [True, False])
@pytest.mark.parametrize("swiglu", [True, False])
def test_grouped_pairs_with_short_tails(cuda_lib, gather, swiglu):
    """Large groups whose last row tile holds 1 to 33 rows, so that the second CTA
    of a pair has none of them, over many items and several runs: every run the
    same, and right."""
    counts = [257, 513, 260, 769, 272, 273, 288, 289, 512, 1025, 258, 261, 0, 256, 521, 264]
    g = gen(31)
    off, perm, P = make_groups(counts, 1, g)
    K, N = 192, 1000
    x = randn(g, P, K)
    W, V = randn(g, len(counts), N, K, scale=K ** -0.5), randn(g, len(counts), N, K, scale=K ** -0.5)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    pm = perm if gather else None
    call = (lambda: cuda_lib.grouped_swiglu_bf16(x, W, V, off, pm, 1, ws=ws)) if swiglu else \
        (lambda: cuda_lib.grouped_linear_bf16(x, W, off, pm, 1, ws=ws))
    out = call()
    for _ in range(20):
        assert torch.equal(call(), out)
    assert cuda_lib.last_device_status(ws) == cuda_lib.OK
    src = perm.long() if gather else torch.arange(P, device=DEV)
    a, ma = grouped_ref(x, W, off, src)
    da = (K + 2) * U * ma
    if not swiglu:
        return within(out, a, a.abs() * HALF + da * (1 + HALF))
    b, mb = grouped_ref(x, V, off, src)
    db = (K + 2) * U * mb
    s = a * torch.sigmoid(a)
    tol = 1.1 * da * (b.abs() + db) + (s.abs() + 1.1 * da) * db + 16 * U * (s * b).abs()
    within(out, s * b, (s * b).abs() * HALF + tol * (1 + HALF) + 1e-300)


def test_grouped_many_experts(cuda_lib):
    g = gen(3)
    E, T, k, K, N = 896, 64, 16, 192, 144
    idx = torch.rand(T, E, device=DEV, generator=g).topk(k, 1).indices.to(torch.int32)
    counts, off, perm, inv, _ = cuda_lib.permute(idx, E)
    x, W = randn(g, T, K), randn(g, E, N, K, scale=K ** -0.5)
    out = cuda_lib.grouped_linear_bf16(x, W, off, perm, k)
    ref, mag = grouped_ref(x, W, off, (perm // k).long())
    within(out, ref, ref.abs() * HALF + (K + 2) * U * mag * (1 + HALF))


def test_grouped_rows_outside_the_groups_stay(cuda_lib):
    g = gen(4)
    off = torch.tensor([3, 10, 10, 45], dtype=torch.int32, device=DEV)  # rows 0..2 and 45..59 are in no group
    x, W = randn(g, 60, 128), randn(g, 3, 96, 128)
    out = torch.full((60, 96), 5.0, dtype=torch.bfloat16, device=DEV)
    cuda_lib.grouped_linear_bf16(x, W, off, out=out)
    ref, mag = grouped_ref(x, W, off, torch.arange(60, device=DEV))
    assert bool((out[:3] == 5).all()) and bool((out[45:] == 5).all())
    within(out[3:45], ref[3:45], ref[3:45].abs() * HALF + 130 * U * mag[3:45] * (1 + HALF))


def test_grouped_nan_row_stays_apart(cuda_lib):
    g = gen(8)
    off = torch.tensor([0, 20, 39], dtype=torch.int32, device=DEV)
    x, W = randn(g, 39, 136), randn(g, 2, 72, 136)
    clean = cuda_lib.grouped_linear_bf16(x, W, off)
    x[19, 3] = float("nan")
    out = cuda_lib.grouped_linear_bf16(x, W, off)
    assert bool(out[19].isnan().all())
    keep = [i for i in range(39) if i != 19]
    assert torch.equal(out[keep], clean[keep])


@pytest.mark.parametrize("what", ["perm_high", "perm_low", "offset_high", "offset_back", "offset_negative"])
@pytest.mark.parametrize("swiglu", [False, True])
def test_grouped_bad_indices_are_reported(cuda_lib, what, swiglu):
    """Bad groups and rows: a status, nothing out of bounds, and the groups that are right keep their results."""
    g = gen(12)
    off = torch.tensor([0, 8, 24, 40], dtype=torch.int32, device=DEV)
    perm = torch.arange(40, dtype=torch.int32, device=DEV)
    if what == "perm_high":
        perm[30] = 4000
    elif what == "perm_low":
        perm[30] = -7
    elif what == "offset_high":
        off[3] = 4000
    elif what == "offset_back":
        off[3] = 20
    else:
        off[0] = -3
    x, W = randn(g, 40, 64), randn(g, 3, 80, 64)
    ws = torch.zeros(256, dtype=torch.uint8, device=DEV)
    out, intact = guarded((40, 80), torch.bfloat16)
    if swiglu:
        cuda_lib.grouped_swiglu_bf16(x, W, W, off, perm, 1, out=out, ws=ws)
    else:
        cuda_lib.grouped_linear_bf16(x, W, off, perm, 1, out=out, ws=ws)
    assert cuda_lib.last_device_status(ws) == cuda_lib.ERR_DEVICE_CHECK
    assert intact()
    if not swiglu:  # group 1 (rows 8..23) is good in every case
        ref = x[8:24].to(D) @ W[1].to(D).t()
        within(out[8:24], ref, ref.abs() * HALF + 66 * U * (x[8:24].to(D).abs() @ W[1].to(D).abs().t()) * (1 + HALF))


def test_outputs_past_32_bit_offsets(cuda_lib):
    """More than 2^31 output elements: the last rows are right."""
    g = gen(40)
    # 66000 rows x 33000 outputs
    P, N = 66000, 33000
    x, W = randn(g, P, 32), randn(g, 2, N, 32)
    off = torch.tensor([0, 30000, P], dtype=torch.int32, device=DEV)
    out = cuda_lib.grouped_linear_bf16(x, W, off)
    for rows, e in ((slice(29990, 30000), 0), (slice(P - 300, P), 1)):
        ref = x[rows].to(D) @ W[e].to(D).t()
        within(out[rows], ref, ref.abs() * HALF + 34 * U * (x[rows].to(D).abs() @ W[e].to(D).abs().t()) * (1 + HALF))
    del out
    q, s, Wm = mx_weights(cuda_lib, g, N, 32)
    out = cuda_lib.linear_mxfp4(x, q, s, N)
    rows = slice(P - 130, P)
    ref = x[rows].to(D) @ Wm.t()
    within(out[rows], ref, linear_tol(x[rows], Wm, ref))
    del out
    T, H = 270000, 8192
    y = torch.randn(T, H, device=DEV, dtype=torch.bfloat16, generator=g)
    w = randn(g, H, dtype=torch.float32)
    n = cuda_lib.rms_norm(y, w)
    ref = norm_ref(y[-3:].to(D), w, 1e-5)
    within(n[-3:], ref, ref.abs() * (HALF + 64 * U) * (1 + HALF))


# ---- streams, graphs, repeats -------------------------------------------------------

def _calls(lmoe, g):
    """One call of each operator on fixed inputs, as (function of keyword arguments, its workspace bytes or None)."""
    q, s, _ = mx_weights(lmoe, g, 512, 1024)
    off, perm, T = make_groups([3, 0, 50, 1, 10], 4, g)
    x, xm, xb = randn(g, T, 256), randn(g, 3, 1024), randn(g, 100, 1024)
    W, V = randn(g, 5, 136, 256), randn(g, 5, 136, 256)
    y, r, w = randn(g, 33, 1024), randn(g, 33, 1024, dtype=torch.float32), randn(g, 1024, dtype=torch.float32)
    # many items: handed out by the counter in the workspace, for single CTAs and for pairs
    off1, perm1, T1 = make_groups([2, 1] * 32, 1, g)
    off2, perm2, T2 = make_groups([700, 300, 513, 5], 1, g)
    x1, W1, x2, W2 = randn(g, T1, 64), randn(g, 64, 1300, 64), randn(g, T2, 64), randn(g, 4, 10000, 64)
    return [
        (lambda **a: lmoe.rms_norm(r, w, **a), None),
        (lambda **a: lmoe.residual_norm(y, r, post_w=w, next_w=w, scale=0.5, **a)[1], None),
        (lambda **a: lmoe.linear_mxfp4(xm, q, s, 512, **a), lmoe.linear_mxfp4_workspace_size(3, 1024, 512)),
        (lambda **a: lmoe.linear_mxfp4(xb, q, s, 512, **a), lmoe.linear_mxfp4_workspace_size(100, 1024, 512)),
        (lambda **a: lmoe.grouped_linear_bf16(x, W, off, perm, 4, **a), 256),
        (lambda **a: lmoe.grouped_swiglu_bf16(x, W, V, off, perm, 4, **a), 256),
        (lambda **a: lmoe.grouped_linear_bf16(x1, W1, off1, perm1, 1, **a), 256),
        (lambda **a: lmoe.grouped_linear_bf16(x2, W2, off2, perm2, 1, **a), 256),
        (lambda **a: lmoe.grouped_swiglu_bf16(x2, W2, W2, off2, perm2, 1, **a), 256),
    ]


def test_operators_repeat_bit_for_bit(cuda_lib):
    for f, _ in _calls(cuda_lib, gen(20)):
        a = f()
        assert all(torch.equal(a, f()) for _ in range(5))


def test_operators_on_another_stream(cuda_lib):
    side = torch.cuda.Stream(DEV)
    for f, _ in _calls(cuda_lib, gen(21)):
        a = f()
        torch.cuda.synchronize()
        b = f(stream=side)
        with torch.cuda.stream(side):
            c = f()
        side.synchronize()
        assert torch.equal(a, b) and torch.equal(a, c)


def test_operators_captured_and_replayed(cuda_lib):
    """Each operator in two graphs, with a workspace each, replayed at once on two streams."""
    streams = [torch.cuda.Stream(DEV) for _ in range(2)]
    for f, need in _calls(cuda_lib, gen(22)):
        want = f()
        torch.cuda.synchronize()
        graphs = []
        for _ in range(2):
            kw = {} if need is None else {"ws": torch.zeros(need, dtype=torch.uint8, device=DEV)}
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr):
                outs = [f(**kw) for _ in range(3)]
            graphs.append((gr, outs, kw))
        for _ in range(3):
            for st, (gr, _, _) in zip(streams, graphs):
                with torch.cuda.stream(st):
                    gr.replay()
        torch.cuda.synchronize()
        for _, outs, _ in graphs:
            assert all(torch.equal(want, o) for o in outs)
