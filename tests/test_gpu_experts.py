"""The expert layer's calls against their definitions in 64 bits (GPU only):
token sort and combine, expert products, routing gradient, and a layer of them
forward and backward."""
import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

import pytest
import torch

import moe_expert_routing_token_b200 as moe
from tests import expert_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, I32, D = torch.bfloat16, torch.float32, torch.int32, torch.float64


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dtype=BF, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def routing(M, k, E, g, missing=0.0):
    ids = torch.rand(M, E, generator=g, device=DEV).argsort(1)[:, :k].to(I32)
    if missing:
        ids = torch.where(torch.rand(M, k, generator=g, device=DEV) < missing, -1, ids).to(I32)
    w = torch.rand(M, k, generator=g, device=DEV) + 0.1
    _, offsets, _, scatter, _ = moe.expert_permutation(ids.contiguous(), E)
    return w, ids.contiguous(), offsets, scatter


# ---------------------------------------------------------------- tokens to experts and back

TOKENS = [  # M, k, E, H, share of pairs without a place
    (1, 1, 1, 1, 0.0), (1, 8, 8, 7168, 0.0), (3, 2, 8, 8, 0.0), (5, 1, 4, 33, 0.0), (17, 6, 160, 1031, 0.4),
    (64, 8, 256, 7168, 0.0), (129, 9, 16, 514, 0.2), (40, 32, 64, 260, 0.9), (7, 3, 8, 12, 1.0), (300, 40, 64, 72, 0.1),
    (1025, 8, 256, 2052, 0.5)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,k,E,H,missing", TOKENS)
def test_gather(M, k, E, H, missing, dtype):
    g = gen(M * 31 + H)
    _, _, offsets, scatter = routing(M, k, E, g, missing)
    x = randn(g, M, H, dtype=dtype)
    canary = torch.full((M * k, H), 7.0, dtype=dtype, device=DEV)
    out = moe.gather_tokens(x, scatter, k, out=canary.clone())
    want = canary.clone()
    at = scatter.long()
    pair = (at >= 0).nonzero()[:, 0]
    want[at[pair]] = x[pair // k]
    assert torch.equal(out, want)           # rows behind the last segment as they were
    n = int(offsets[-1])
    assert torch.equal(moe.gather_tokens(x, scatter, k)[:n], want[:n])

    dsorted = randn(g, M * k, H, dtype=dtype)
    dsorted[n:] = float("nan")              # belongs to nobody
    ref.within(moe.gather_tokens_backward(dsorted, scatter, k), ref.combine(dsorted, scatter, None, None, k))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("M,k,E,H,missing", TOKENS)
def test_combine(M, k, E, H, missing, residual, dtype):
    g = gen(M * 37 + H)
    w, _, offsets, scatter = routing(M, k, E, g, missing)
    n = int(offsets[-1])
    y, r = randn(g, M * k, H, dtype=dtype), randn(g, M, H, dtype=dtype) if residual else None
    y[n:] = float("inf")
    w[(scatter.view(M, k) < 0)] = float("nan")   # weights of pairs without a place are not used
    ref.within(moe.combine_tokens(y, scatter, w, residual=r), ref.combine(y, scatter, w.nan_to_num(0.0), r, k))

    dout = randn(g, M, H, dtype=dtype)
    canary = torch.full((M * k, H), -3.0, dtype=dtype, device=DEV)
    dy, dw = moe.combine_tokens_backward(dout, y, scatter, w, grad_y=canary.clone())
    rows, placed = ref.rows_of(y, scatter, k)
    dot = rows * dout.to(D)[:, None, :]
    ref.within(dw, (dot.sum(2), (H + 8) * ref.U24 * dot.abs().sum(2)))
    assert bool((dw[~placed] == 0).all())
    pair = (scatter >= 0).nonzero()[:, 0]
    v = dout.to(D)[pair // k] * w.reshape(-1)[pair, None].to(D)
    ref.within(dy[scatter[pair].long()], (v, (ref.half_step(dtype) + ref.U24) * v.abs()))
    assert torch.equal(dy[n:], canary[n:])


def test_token_rows_at_every_alignment():
    """Rows that begin at any element of their storage: the widest accesses
    that still reach them are taken."""
    M, k, E, H = 37, 4, 16, 264
    g = gen(5)
    w, _, _, scatter = routing(M, k, E, g)
    for dtype in (BF, F32):
        for shift in (0, 1, 2, 3, 4, 8):
            buf = randn(g, M * H + 16, dtype=dtype)
            x = buf[shift:shift + M * H].view(M, H)
            out = torch.empty(M * k * H + 16, dtype=dtype, device=DEV)[shift:shift + M * k * H].view(M * k, H)
            moe.gather_tokens(x, scatter, k, out=out)
            assert torch.equal(out[scatter.long()], x.repeat_interleave(k, 0))
            ref.within(moe.combine_tokens(out, scatter, w, residual=x), ref.combine(out, scatter, w, x, k))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("H", [64, 257, 288, 289, 385, 577, 768, 1154, 2308, 2881, 20011])
def test_rows_of_many_widths(H, dtype):
    """Widths around whole segments of every access size."""
    M, k, E = 43, 5, 16
    g = gen(H)
    w, _, _, scatter = routing(M, k, E, g)
    x, r, dout = randn(g, M, H, dtype=dtype), randn(g, M, H, dtype=dtype), randn(g, M, H, dtype=dtype)
    xs = moe.gather_tokens(x, scatter, k)
    assert torch.equal(xs[scatter.long()], x.repeat_interleave(k, 0))
    y = randn(g, M * k, H, dtype=dtype)
    ref.within(moe.combine_tokens(y, scatter, w, residual=r), ref.combine(y, scatter, w, r, k))
    ref.within(moe.gather_tokens_backward(y, scatter, k), ref.combine(y, scatter, None, None, k))
    dy, dw = moe.combine_tokens_backward(dout, y, scatter, w)
    rows, _ = ref.rows_of(y, scatter, k)
    dot = rows * dout.to(D)[:, None, :]
    ref.within(dw, (dot.sum(2), (H + 8) * ref.U24 * dot.abs().sum(2)))
    v = dout.to(D).repeat_interleave(k, 0) * w.reshape(-1, 1).to(D)
    ref.within(dy[scatter.long()], (v, (ref.half_step(dtype) + ref.U24) * v.abs()))


def test_token_offsets_pass_32_bits():
    """Row offsets beyond 2^32 bytes and 2^31 elements."""
    M, k, E, H = 40000, 8, 8, 7168
    g = gen(6)
    ids = torch.arange(8, dtype=I32, device=DEV).repeat(M, 1)
    _, _, _, scatter, _ = moe.expert_permutation(ids, E)
    x = randn(g, M, H)
    xs = moe.gather_tokens(x, scatter, k)
    assert torch.equal(xs[-M:], x) and torch.equal(xs[:M], x)
    w = torch.full((M, k), 0.125, device=DEV)
    assert torch.equal(moe.combine_tokens(xs, scatter, w), x)   # eighths of one value sum exactly
    del xs
    torch.cuda.empty_cache()


def test_empty_batches():
    e = torch.empty(0, 64, dtype=BF, device=DEV)
    s = torch.empty(0, dtype=I32, device=DEV)
    assert moe.gather_tokens(e, s, 4).shape == (0, 64)
    assert moe.gather_tokens_backward(e, s, 4).shape == (0, 64)
    w = torch.empty(0, 4, device=DEV)
    assert moe.combine_tokens(e, s, w).shape == (0, 64)
    off = torch.zeros(3, dtype=I32, device=DEV)
    W = torch.zeros(2, 16, 64, dtype=BF, device=DEV)
    assert moe.expert_matmul(e, W, off).shape == (0, 16)
    dw, db = moe.expert_matmul_grad_weight(torch.empty(0, 16, dtype=BF, device=DEV), e, off, bias_grad=True)
    torch.cuda.synchronize()
    assert bool((dw == 0).all()) and bool((db == 0).all())
    assert moe.topk_backward(torch.empty(0, 2, device=DEV), torch.empty(0, 8, device=DEV),
                             torch.empty(0, 2, dtype=I32, device=DEV), "softmax", True).shape == (0, 8)


# ---------------------------------------------------------------- expert products

SEGMENTS = {
    "one row": [1],
    "dense": [300],
    "uneven": [0, 1, 127, 0, 128, 129, 15, 16, 17, 0],
    "long": [257, 3, 512, 256],
    "none": [0, 0, 0],
    "many": [i % 5 for i in range(160)],
}


def product(name, K, N, seed, spare=13):
    """Offsets, rows and weight; `spare` rows behind the last segment hold NaN."""
    counts = SEGMENTS[name]
    g = gen(seed)
    offsets = torch.tensor([0] + counts, device=DEV).cumsum(0).to(I32)
    P = sum(counts) + spare
    x = randn(g, P, K)
    x[sum(counts):] = float("nan")
    return g, len(counts), P, offsets, x


SHAPES = [(8, 8), (64, 128), (72, 136), (200, 264), (1032, 520), (2048, 256)]
FORMS = [  # activation, gated, bias, residual, preact
    ("none", False, False, False, False), ("silu", True, False, False, True), ("gelu", False, True, True, False),
    ("silu", False, True, False, True), ("gelu", True, True, True, True), ("none", True, False, True, False)]


@pytest.mark.parametrize("name", list(SEGMENTS))
@pytest.mark.parametrize("K,N", SHAPES)
@pytest.mark.parametrize("act,gated,bias,residual,preact", FORMS)
def test_expert_matmul(name, K, N, act, gated, bias, residual, preact):
    g, E, P, off, x = product(name, K, N, K + N)
    Nz = 2 * N if gated else N
    w = randn(g, E, Nz, K, scale=K ** -0.5)
    b = randn(g, E, Nz, dtype=F32) if bias else None
    r = randn(g, P, N) if residual else None
    out = torch.full((P, N), 5.0, dtype=BF, device=DEV)
    kept = torch.full((P, Nz), 6.0, dtype=BF, device=DEV) if preact else None
    got = moe.expert_matmul(x, w, off, bias=b, activation=act, gated=gated, residual=r, out=out, preact_out=kept)
    n = int(off[-1])
    want = ref.matmul(x, w, off, b, act, gated, r)
    ref.within(out[:n], tuple(t[:n] for t in want["out"]))
    assert bool((out[n:] == 5.0).all())
    if preact:
        assert got[1] is kept
        ref.within(kept[:n], tuple(t[:n] for t in want["preact"]))
        assert bool((kept[n:] == 6.0).all())


@pytest.mark.parametrize("name", list(SEGMENTS))
@pytest.mark.parametrize("K,N", SHAPES)
@pytest.mark.parametrize("act,gated,through", [("none", False, False), ("silu", True, True), ("gelu", False, True),
                                               ("silu", False, True), ("gelu", True, True), ("none", True, True)])
def test_expert_matmul_grad_input(name, K, N, act, gated, through):
    g, E, P, off, dy = product(name, N, K, K + N + 1)
    w = randn(g, E, N, K, scale=N ** -0.5)
    Kz = 2 * K if gated else K
    z = randn(g, P, Kz, scale=2.0) if through else None
    out = torch.full((P, Kz), 5.0, dtype=BF, device=DEV)
    moe.expert_matmul_grad_input(dy, w, off, preact=z, activation=act, gated=gated, out=out)
    n = int(off[-1])
    ref.within(out[:n], tuple(t[:n] for t in ref.grad_input(dy, w, off, z, act, gated)))
    assert bool((out[n:] == 5.0).all())


@pytest.mark.parametrize("name", list(SEGMENTS))
@pytest.mark.parametrize("K,N", SHAPES)
@pytest.mark.parametrize("dtype,bias", [(BF, True), (F32, False), (F32, True)])
def test_expert_matmul_grad_weight(name, K, N, dtype, bias):
    g, E, P, off, x = product(name, K, N, K + N + 2)
    dy = randn(g, P, N)
    dy[int(off[-1]):] = float("inf")
    got = moe.expert_matmul_grad_weight(dy, x, off, bias_grad=bias, dtype=dtype)
    dw, db = ref.grad_weight(dy, x, off, E, dtype)
    ref.within(got[0] if bias else got, dw)
    if bias:
        ref.within(got[1], db)


def test_grad_weight_keeps_neighbours_apart():
    """An expert's sum takes nothing of the next segment's rows, whatever they
    hold: infinities stay in their own expert."""
    off = torch.tensor([0, 70, 135, 200], dtype=I32, device=DEV)
    g = gen(11)
    dy, x = randn(g, 200, 136), randn(g, 200, 72)
    x[70:135] = float("inf")
    dw, db = moe.expert_matmul_grad_weight(dy, x, off, bias_grad=True, dtype=F32)
    good = torch.cat([x[:70], torch.zeros_like(x[70:135]), x[135:]])
    want, want_b = ref.grad_weight(dy, good, off, 3, F32)
    for e in (0, 2):
        ref.within(dw[e], (want[0][e], want[1][e]))
    assert not bool(dw[1].isfinite().any())
    ref.within(db, want_b)


@pytest.mark.parametrize("offsets", [[0, 5, 3, 9], [-4, 2, 100, 100], [7, 7, 7, 7], [50, 60, 70, 80]])
def test_offsets_outside_the_rows(offsets):
    """Offsets that no permutation gives: nothing outside the tensors is
    touched, and experts with a proper range inside [0, P] are served."""
    P, K, N = 40, 72, 136
    g = gen(12)
    off = torch.tensor(offsets, dtype=I32, device=DEV)
    buf = torch.full((P + 64, N), 3.0, dtype=BF, device=DEV)
    x, w = randn(g, P, K), randn(g, 3, N, K)
    moe.expert_matmul(x, w, off, out=buf[32:32 + P])
    dw = moe.expert_matmul_grad_weight(buf[32:32 + P], x, off)
    torch.cuda.synchronize()
    assert bool((buf[:32] == 3.0).all()) and bool((buf[32 + P:] == 3.0).all()) and dw.shape == (3, N, K)
    served = [(e, max(0, min(P, a)), max(0, min(P, b))) for e, (a, b) in enumerate(zip(offsets, offsets[1:]))]
    rows = torch.zeros(P, device=DEV)
    for _, a, b in served:
        rows[a:max(a, b)] += 1
    for e, a, b in served:
        own = [p for p in range(a, b) if rows[p] == 1]
        if own:
            one = ref.matmul(x, w[e:e + 1], [0, P], None, "none", False, None)["out"]
            ref.within(buf[32:32 + P][own], tuple(t[own] for t in one))
    assert bool((buf[32:32 + P][rows == 0] == 3.0).all())


@pytest.mark.parametrize("counts,K,N,gated", [
    ([0, 1, 0, 0, 1, 0, 0, 0], 1024, 512, True),       # one token: four pairs of CTAs to a tile
    ([3], 520, 8, False), ([32, 0, 33, 1], 4096, 136, False), ([1] * 12, 4160, 264, False),
    ([5, 0, 31, 2], 264, 520, True), ([17], 7168, 256, False)])
def test_few_rows_long_reductions(counts, K, N, gated):
    """Calls small enough that pairs of CTAs share a tile's reduction: against
    the definition, and the same bits each time."""
    g = gen(K + N)
    off = torch.tensor([0] + counts, device=DEV).cumsum(0).to(I32)
    P, E = sum(counts), len(counts)
    x, w = randn(g, P, K), randn(g, E, 2 * N if gated else N, K, scale=K ** -0.5)
    b, r = randn(g, E, w.shape[1], dtype=F32), randn(g, P, N)
    out = moe.expert_matmul(x, w, off, bias=b, activation="silu", gated=gated, residual=r)
    ref.within(out, ref.matmul(x, w, off, b, "silu", gated, r)["out"])
    for _ in range(3):
        assert torch.equal(moe.expert_matmul(x, w, off, bias=b, activation="silu", gated=gated, residual=r), out)
    dy, w2 = randn(g, P, K), randn(g, E, K, N, scale=K ** -0.5)
    dx = moe.expert_matmul_grad_input(dy, w2, off)
    ref.within(dx, ref.grad_input(dy, w2, off, None, "none", False))
    assert torch.equal(moe.expert_matmul_grad_input(dy, w2, off), dx)


@pytest.mark.parametrize("E", [1000, 1024])
def test_most_experts(E):
    g = gen(E)
    counts = torch.randint(0, 4, (E,), generator=g, device=DEV)
    counts[::7] = 0
    counts[E // 2] = 300
    off = torch.zeros(E + 1, dtype=I32, device=DEV)
    off[1:] = counts.cumsum(0)
    P, K, N = int(off[-1]), 72, 40
    x, w = randn(g, P, K), randn(g, E, N, K)
    ref.within(moe.expert_matmul(x, w, off), ref.matmul(x, w, off, None, "none", False, None)["out"])
    dy = randn(g, P, N)
    ref.within(moe.expert_matmul_grad_input(dy, w, off), ref.grad_input(dy, w, off, None, "none", False))
    dw, db = moe.expert_matmul_grad_weight(dy, x, off, bias_grad=True)
    want, want_b = ref.grad_weight(dy, x, off, E, BF)
    ref.within(dw, want)
    ref.within(db, want_b)


def test_product_offsets_pass_32_bits():
    """More than 2^31 values in the output, the preactivation and the weight's
    gradient: their last rows against the definition."""
    g = gen(31)
    P, K, N = 270000, 64, 8192
    off = torch.tensor([0, 130000, P], dtype=I32, device=DEV)
    x, w = randn(g, P, K), randn(g, 2, N, K, scale=0.125)
    out, kept = moe.expert_matmul(x, w, off, activation="silu", return_preact=True)
    want = ref.matmul(x[-300:], w[1:], [0, 300], None, "silu", False, None)
    ref.within(out[-300:], want["out"])
    ref.within(kept[-300:], want["preact"])
    dx = moe.expert_matmul_grad_input(out, w, off)
    ref.within(dx[-300:], ref.grad_input(out[-300:], w[1:], [0, 300], None, "none", False))
    del out, kept, dx, x, w
    E, N, K = 300, 4096, 2048
    off = torch.arange(E + 1, dtype=I32, device=DEV) * 3
    dy, x = randn(g, 3 * E, N), randn(g, 3 * E, K)
    dw = moe.expert_matmul_grad_weight(dy, x, off)
    ref.within(dw[-2:], ref.grad_weight(dy[-6:], x[-6:], [0, 3, 6], 2, BF)[0])
    del dw
    torch.cuda.empty_cache()


def test_expert_matmul_spread_values():
    """Preactivations far into both tails, where expf over- and underflows."""
    g = gen(13)
    x = randn(g, 64, 64, scale=30.0)
    w = randn(g, 1, 128, 64)
    off = torch.tensor([0, 64], dtype=I32, device=DEV)
    for act in ("silu", "gelu"):
        for gated in (False, True):
            out = moe.expert_matmul(x, w, off, activation=act, gated=gated)
            ref.within(out, ref.matmul(x, w, off, None, act, gated, None)["out"])
            z = randn(g, 64, 128 if gated else 64, scale=60.0)
            w2 = w[:, :, :64].contiguous()
            dy = randn(g, 64, 128)
            ref.within(moe.expert_matmul_grad_input(dy, w2, off, preact=z, activation=act, gated=gated),
                       ref.grad_input(dy, w2, off, z, act, gated))


# ---------------------------------------------------------------- the router's gradient

ROUTES = [("softmax", False, 1.0, 0.0), ("softmax", True, 2.5, 0.0), ("softmax", False, 2.5, 30.0),
          ("softmax", True, 1.0, 5.0), ("sigmoid", False, 1.0, 0.0), ("sigmoid", True, 2.5, 0.0)]


def choice(M, k, E, dtype, seed, scale=2.0):
    g = gen(seed)
    x = randn(g, M, E, dtype=dtype, scale=scale)
    ids = (x + torch.rand(M, E, generator=g, device=DEV)).topk(k, dim=1).indices.to(I32).contiguous()
    return x, ids, torch.randn(M, k, generator=g, device=DEV)


def check_topk(x, ids, dw, scoring, renorm, rsf, cap, got):
    xd = x.to(D).requires_grad_()
    (want,) = torch.autograd.grad((ref.routed(xd, ids, scoring, renorm, rsf, cap) * dw.to(D)).sum(), xd)
    xd = xd.detach()
    z = cap * torch.tanh(xd / cap) if cap else xd
    p = torch.special.expit(z) if scoring == "sigmoid" else torch.softmax(z, 1)
    # Relative error of a score: its exponent's argument is rounded (|z - max|,
    # and tanhf and the products around it by 4 units of cap), expf, the
    # division and a sum of positive terms, E / 32 + 5 deep, a few units more.
    depth = 64 + x.shape[1] / 32
    eps = (depth + 2 * (z.amax(1, keepdim=True) - z.amin(1, keepdim=True)) + 8 * abs(cap)) * ref.U24
    chosen = p.gather(1, ids.long())
    v = chosen / chosen.sum(1, keepdim=True) if renorm else chosen
    g = rsf * dw.to(D).abs()
    # every term of the formula with its sign taken off
    lump = (g * v).sum(1, keepdim=True)
    size = torch.zeros_like(p)
    if scoring == "softmax" and not renorm:
        size = p * lump
        size.scatter_add_(1, ids.long(), chosen * g)
    elif scoring == "softmax":
        size.scatter_add_(1, ids.long(), v * (g + lump))
    elif renorm:
        size.scatter_add_(1, ids.long(), (g + lump) * v)
    else:
        size.scatter_add_(1, ids.long(), g * chosen)
    slope = 1 - torch.tanh(xd / cap) ** 2 if cap else torch.ones_like(xd)
    # The 64-bit value's own error: the dense softmax's derivative with
    # renormalisation is a difference of terms of at most lump, exactly 0 off
    # the chosen experts but computed in fewer than 16 roundings of 2^-53 each.
    d = 3 * eps * size * slope + 8 * ref.U24 * size + 2.0 ** -48 * lump
    ref.within(got, (want, d + ref.half_step(x.dtype) * (want.abs() + d) + 2.0 ** -126))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scoring,renorm,rsf,cap", ROUTES)
@pytest.mark.parametrize("M,k,E", [(1, 1, 1), (1, 2, 8), (5, 8, 8), (33, 6, 160), (64, 8, 256), (129, 32, 1024),
                                   (7, 3, 37), (1000, 4, 64), (4099, 8, 256)])
def test_topk_backward(M, k, E, scoring, renorm, rsf, cap, dtype):
    x, ids, dw = choice(M, k, E, dtype, M + E)
    out = torch.full_like(x, float("nan"))
    got = moe.topk_backward(dw, x, ids, scoring, renorm, rsf, softcap=cap, out=out)
    check_topk(x, ids, dw, scoring, renorm, rsf, cap, got)


@pytest.mark.parametrize("scoring,renorm,rsf,cap", ROUTES)
def test_topk_backward_against_differences(scoring, renorm, rsf, cap):
    """Along random directions, against central differences of the 64-bit
    routing weights: truncation h^2 / 6 times a third derivative below 10
    units of the values, rounding 2^-52 / h."""
    x, ids, dw = choice(50, 6, 160, F32, 3)
    got = moe.topk_backward(dw, x, ids, scoring, renorm, rsf, softcap=cap).to(D)
    h = 1e-4
    for seed in range(4):
        d = torch.randn(x.shape, generator=gen(seed), device=DEV, dtype=D)
        diff = (ref.routed(x.to(D) + h * d, ids, scoring, renorm, rsf, cap)
                - ref.routed(x.to(D) - h * d, ids, scoring, renorm, rsf, cap)) / (2 * h)
        want = (diff * dw.to(D)).sum(1)
        size = (got.abs() * d.abs()).sum(1) + rsf * dw.to(D).abs().sum(1)
        assert bool(((got * d).sum(1) - want).abs().le(2e-5 * size).all())


def test_topk_backward_saturated_logits():
    for scoring, renorm, rsf, cap in ROUTES:
        x, ids, dw = choice(40, 8, 256, F32, 9, scale=30.0)
        got = moe.topk_backward(dw, x, ids, scoring, renorm, rsf, softcap=cap)
        check_topk(x, ids, dw, scoring, renorm, rsf, cap, got)


def test_topk_backward_ids_outside_and_twice():
    """Ids outside [0, E) are left out of every sum; an id given twice adds up."""
    x, ids, dw = choice(20, 4, 32, F32, 4)
    for scoring, renorm, rsf, cap in ROUTES:
        whole = moe.topk_backward(dw, x, ids, scoring, renorm, rsf, softcap=cap)
        shared = torch.cat([ids, torch.full_like(ids[:, :1], 32), torch.full_like(ids[:, :1], -1)], 1).contiguous()
        more = torch.cat([dw, torch.full_like(dw[:, :2], float("nan"))], 1).contiguous()
        assert torch.equal(moe.topk_backward(more, x, shared, scoring, renorm, rsf, softcap=cap), whole)
        if not renorm:
            twice = torch.cat([ids, ids], 1).contiguous()
            halves = torch.cat([dw, dw], 1).contiguous()
            ref.within(moe.topk_backward(halves, x, twice, scoring, renorm, rsf, softcap=cap),
                       (2 * whole.to(D), 1e-5 * whole.to(D).abs() + 1e-7))
        none = torch.full_like(ids, -1)
        assert bool((moe.topk_backward(dw, x, none, scoring, renorm, rsf, softcap=cap) == 0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_topk_backward_of_the_routing_calls(dtype):
    """The gradients of what the routing calls return, on unaligned rows too."""
    M, E = 301, 160
    x = randn(gen(21), M * E + 8, dtype=dtype)[1:1 + M * E].view(M, E)
    dw = torch.randn(M, 6, generator=gen(22), device=DEV)
    w, ids = moe.grouped_topk(x, 6, False, 8, 3, 1.0)
    check_topk(x, ids, dw, "softmax", False, 1.0, 0.0, moe.topk_backward(dw, x, ids, "softmax", False))
    w, ids = moe.biased_grouped_topk(x, randn(gen(23), E, dtype=F32, scale=0.05), 6, True, 8, 4, 2.5)
    check_topk(x, ids, dw, "sigmoid", True, 2.5, 0.0, moe.topk_backward(dw, x, ids, "sigmoid", True, 2.5))
    v = ref.routed(x.to(D), ids, "sigmoid", True, 2.5, 0.0)
    assert float((w.to(D) - v).abs().max()) < 1e-2


def test_operands_and_outputs_on_other_devices_are_refused():
    x, s, w = torch.zeros(4, 8, device=DEV), torch.zeros(8, dtype=I32, device=DEV), torch.zeros(4, 2, device=DEV)
    for call in (lambda: moe.gather_tokens(x, s.cpu(), 2), lambda: moe.gather_tokens(x, s, 2, out=torch.zeros(8, 8)),
                 lambda: moe.gather_tokens(x, s, 2, out=torch.zeros(8, 8, dtype=BF, device=DEV)),
                 lambda: moe.gather_tokens(x, s, 2, out=torch.zeros(8, 16, device=DEV)[:, ::2]),
                 lambda: moe.combine_tokens(torch.zeros(8, 8, device=DEV), s, w.cpu()),
                 lambda: moe.combine_tokens(torch.zeros(8, 8, device=DEV), s, w, residual=torch.zeros(4, 8))):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(NotImplementedError, match="multiples of 8"):
        moe.expert_matmul(torch.zeros(4, 12, dtype=BF, device=DEV), torch.zeros(1, 8, 12, dtype=BF, device=DEV),
                          torch.zeros(2, dtype=I32, device=DEV))


# ---------------------------------------------------------------- the calls together

def layer(x, logits, W1, b1, W2, dout, k):
    """Forward and backward of one layer; every value a training step keeps."""
    E = W1.shape[0]
    w, ids = moe.topk_softmax(logits, k, True)
    _, offsets, _, scatter, _ = moe.expert_permutation(ids, E)
    xs = moe.gather_tokens(x, scatter, k)
    h, z = moe.expert_matmul(xs, W1, offsets, bias=b1, activation="silu", gated=True, return_preact=True)
    y = moe.expert_matmul(h, W2, offsets)
    out = moe.combine_tokens(y, scatter, w, residual=x)
    dy, dw = moe.combine_tokens_backward(dout, y, scatter, w)
    dz = moe.expert_matmul_grad_input(dy, W2, offsets, preact=z, activation="silu", gated=True)
    dW2 = moe.expert_matmul_grad_weight(dy, h, offsets)
    dxs = moe.expert_matmul_grad_input(dz, W1, offsets)
    dW1, db1 = moe.expert_matmul_grad_weight(dz, xs, offsets, bias_grad=True)
    dx = moe.gather_tokens_backward(dxs, scatter, k)
    dlogits = moe.topk_backward(dw, logits, ids, "softmax", True)
    return dict(ids=ids, out=out, dx=dx, dW1=dW1, db1=db1, dW2=dW2, dlogits=dlogits)


def layer_inputs(M, k, E, H, F, seed):
    g = gen(seed)
    return (randn(g, M, H), randn(g, M, E, dtype=F32), randn(g, E, 2 * F, H, scale=H ** -0.5),
            randn(g, E, 2 * F, dtype=F32, scale=0.3), randn(g, E, H, F, scale=F ** -0.5), randn(g, M, H), k)


def layer_in_64_bits(x, logits, W1, b1, W2, dout, k, ids):
    leaves = [t.to(D).requires_grad_() for t in (x, logits, W1, b1, W2)]
    x, logits, W1, b1, W2 = leaves
    w = ref.routed(logits, ids, "softmax", True, 1.0, 0.0)
    rows = []
    for j in range(k):
        e = ids[:, j].long()
        z = torch.einsum("mh,mnh->mn", x, W1[e]) + b1[e]
        F = z.shape[1] // 2
        rows.append(w[:, j:j + 1] * torch.einsum("mf,mhf->mh", ref.f(z[:, :F], "silu") * z[:, F:], W2[e]))
    out = x + sum(rows)
    dx, dlogits, dW1, db1, dW2 = torch.autograd.grad((out * dout.to(D)).sum(), leaves)
    return dict(out=out.detach(), dx=dx - dout.to(D), dW1=dW1, db1=db1, dW2=dW2, dlogits=dlogits)


@pytest.mark.parametrize("M,k,E,H,F", [(1, 2, 8, 64, 32), (77, 4, 32, 136, 72), (200, 2, 4, 256, 264)])
def test_layer_against_64_bits(M, k, E, H, F):
    """Norm-wise: each value passes at most six roundings to bf16 on its way
    (xs is exact; z, h, y, dy, dz, dxs and itself), each off by at most half a
    step of 2^-8, and the products keep their relative size."""
    inp = layer_inputs(M, k, E, H, F, M + H)
    got = layer(*inp)
    want = layer_in_64_bits(*inp, got["ids"])
    for name, v in want.items():
        off = float((got[name].to(D) - v).norm() / v.norm())
        assert off <= 6 * ref.half_step(BF), (name, off)


def test_layer_gradients_against_differences():
    """Along random directions of each leaf, against central differences of the
    64-bit layer: the bound of the test above on the gradient's norm times the
    direction's, and h^2 times a third derivative."""
    inp = layer_inputs(48, 2, 4, 72, 40, 5)
    got = layer(*inp)
    x, logits, W1, b1, W2, dout, k = inp

    def value(*leaves):
        a, lg, A, c, B = leaves
        w = ref.routed(lg, got["ids"], "softmax", True, 1.0, 0.0)
        total = a
        for j in range(k):
            e = got["ids"][:, j].long()
            z = torch.einsum("mh,mnh->mn", a, A[e]) + c[e]
            F = z.shape[1] // 2
            total = total + w[:, j:j + 1] * torch.einsum("mf,mhf->mh", ref.f(z[:, :F], "silu") * z[:, F:], B[e])
        return (total * dout.to(D)).sum()

    leaves = [t.to(D) for t in (x, logits, W1, b1, W2)]
    grads = [got["dx"].to(D) + dout.to(D)] + [got[n].to(D) for n in ("dlogits", "dW1", "db1", "dW2")]
    h = 1e-4
    for i, grad in enumerate(grads):
        for seed in range(3):
            d = torch.randn(grad.shape, generator=gen(seed + 7 * i), device=DEV, dtype=D)
            up, down = list(leaves), list(leaves)
            up[i], down[i] = leaves[i] + h * d, leaves[i] - h * d
            want = float(value(*up) - value(*down)) / (2 * h)
            bound = 6 * ref.half_step(BF) * float(grad.norm() * d.norm()) + 1e-5 * abs(want)
            assert abs(float((grad * d).sum()) - want) <= bound, (i, seed)


FIRST_CALL = """
import torch, moe_expert_routing_token_b200 as moe
d = "cuda:0"
x, w = torch.ones(40, 1024, device=d).bfloat16(), torch.ones(2, 64, 1024, device=d).bfloat16()
off = torch.tensor([0, 30, 40], dtype=torch.int32, device=d)
out, dw = torch.zeros(40, 64, device=d).bfloat16(), torch.zeros(2, 64, 1024, device=d).bfloat16()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    moe.expert_matmul(x, w, off, out=out)
    moe.expert_matmul_grad_weight(out, x, off, out=dw)
assert float(out.abs().sum()) == 0
graph.replay()
torch.cuda.synchronize()
assert bool((out == 1024).all()) and bool((dw[0] == 1024 * 30).all()) and bool((dw[1] == 1024 * 10).all())
"""


def test_first_calls_inside_a_capture():
    """What the library looks up once per device it may look up while a stream
    is capturing."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, capture_output=True, text=True, timeout=300)
    assert done.returncode == 0, done.stderr[-2000:]


def test_layer_captured_replayed_and_on_another_stream():
    """One graph of the whole layer, replayed on new inputs, while eager calls
    of the same layer run on a second stream: the same bits as eager calls
    alone."""
    a, b = layer_inputs(130, 4, 16, 200, 136, 1), layer_inputs(130, 4, 16, 200, 136, 2)
    alone = [layer(*a), layer(*b)]
    torch.cuda.synchronize()
    static = [t.clone() if torch.is_tensor(t) else t for t in a]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = layer(*static)
    for _ in range(3):
        for k, inp in enumerate((a, b)):
            for s, t in zip(static, inp):
                if torch.is_tensor(s):
                    s.copy_(t)
            side.wait_stream(torch.cuda.current_stream())
            graph.replay()
            with torch.cuda.stream(side):
                beside = layer(*inp)
            torch.cuda.synchronize()
            for name in held:
                assert torch.equal(held[name], alone[k][name]), name
                assert torch.equal(beside[name], alone[k][name]), name


def test_layers_of_two_threads():
    """Two threads call the layer at once, each on a stream of its own: the
    same bits as one after the other."""
    inputs = [layer_inputs(97, 4, 16, 200, 136, 3), layer_inputs(3, 2, 16, 264, 40, 4)]
    alone = [layer(*i) for i in inputs]
    torch.cuda.synchronize()

    def run(i):
        with torch.cuda.stream(torch.cuda.Stream()):
            done = [layer(*inputs[i]) for _ in range(20)]
            torch.cuda.current_stream().synchronize()
        return done

    with ThreadPoolExecutor(2) as pool:
        for i, done in enumerate(pool.map(run, range(2))):
            for got in done:
                for name in got:
                    assert torch.equal(got[name], alone[i][name]), (i, name)


def test_no_watchdog_trips():
    assert moe.watchdog_trips() == 0
