"""The routing gradient (moe_topk_backward) where a caller meets it: behind each
routing call, behind a shared-expert slot, at saturated softcaps and at logits far
below zero (GPU only)."""
import inspect
import re
import textwrap

import pytest
import torch

import moe_expert_routing_token_b200 as moe
from tests import expert_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, I32, D = torch.bfloat16, torch.float32, torch.int32, torch.float64
U24 = ref.U24


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dtype=F32, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(dtype)


def definition(x, ids, g, scoring, renorm, cap, mag=None):
    """(value, bound) in 64 bits of the gradient of sum_j g_j w_j with respect to
    the logits x, for weights without a scaling factor.  ``mag``: magnitudes that
    g was summed from, where it is a sum itself.

    The bound follows the formula term by term, each with its sign taken off.  A
    score, or the chosen ones' shares of their sum, is off by its exponent's
    argument (one rounding of it, and of the capped logits by 4 units of cap:
    tanhf and the products around it), expf (2 units in the last place) and a sum
    of positive terms with a division, fewer than 64 + E / 32 roundings.  At most
    three such factors meet in a term.  The cap's slope is 1 / cosh(t)^2 at
    t = x / cap, rounded: 2 |t| units, and 16 for an exponential, its products
    and a division."""
    x = x.to(D)
    ids, g = ids.long(), g.to(D)
    mag = g.abs() if mag is None else mag.to(D)
    t = x / cap if cap else torch.zeros_like(x)
    z = cap * torch.tanh(t) if cap else x
    slope = 1 / torch.cosh(t) ** 2
    zj = z.gather(1, ids)
    if scoring == "softmax" and not renorm:
        p, spread = torch.softmax(z, 1), z.amax(1, keepdim=True) - z.amin(1, keepdim=True)
        v, every = p.gather(1, ids), p
    elif scoring == "softmax":
        v, spread = torch.softmax(zj, 1), zj.amax(1, keepdim=True) - zj.amin(1, keepdim=True)
    else:
        log_p = torch.nn.functional.logsigmoid(zj)
        q = torch.special.expit(-zj)
        v = torch.softmax(log_p, 1) if renorm else log_p.exp()
        spread = zj.amax(1, keepdim=True) - zj.amin(1, keepdim=True) if renorm else torch.zeros_like(zj[:, :1])
    mean = (g * v).sum(1, keepdim=True)
    lump = (mag * v).sum(1, keepdim=True)
    value, size = torch.zeros_like(x), torch.zeros_like(x)
    if scoring == "softmax" and not renorm:
        value = -every * mean
        size = every * lump
        value.scatter_add_(1, ids, v * g)
        size.scatter_add_(1, ids, v * mag)
    elif scoring == "softmax":
        value.scatter_add_(1, ids, v * (g - mean))
        size.scatter_add_(1, ids, v * (mag + lump))
    elif renorm:
        value.scatter_add_(1, ids, v * (g - mean) * q)
        size.scatter_add_(1, ids, v * (mag + lump) * q)
    else:
        value.scatter_add_(1, ids, v * g * q)
        size.scatter_add_(1, ids, v * mag * q)
    eps = (64 + x.shape[1] / 32 + 2 * spread + 8 * abs(cap)) * U24
    return value * slope, (3 * eps + (2 * t.abs() + 16) * U24) * size * slope


def check(got, value, bound):
    """To the rounding of got's type, and 2^-120 where fp32 leaves its normal range."""
    ref.within(got, (value, bound + ref.half_step(got.dtype) * (value.abs() + bound) + 2.0 ** -120))


def route(M, k, E, dtype, seed, scale=2.0):
    g = gen(seed)
    x = randn(g, M, E, dtype=dtype, scale=scale)
    ids = torch.rand(M, E, generator=g, device=DEV).argsort(1)[:, :k].to(I32).contiguous()
    return x, ids, randn(g, M, k)


# ---------------------------------------------------------------- behind the calls that make weights

def shown(after):
    """The indented example of topk_backward's documentation that follows ``after``."""
    doc = inspect.getdoc(moe.topk_backward)
    assert after in doc
    lines = doc[doc.index(after):].split("::\n", 1)[1].strip("\n").split("\n")
    n = next((i for i, line in enumerate(lines) if line and not line.startswith("    ")), len(lines))
    return textwrap.dedent("\n".join(lines[:n]))


@pytest.mark.parametrize("factor", [None, 2.5])
@pytest.mark.parametrize("scoring,renorm", [("softmax", False), ("softmax", True), ("sigmoid", False),
                                            ("sigmoid", True)])
@pytest.mark.parametrize("k", [1, 2, 6])
def test_behind_a_shared_expert_slot(k, scoring, renorm, factor):
    """The documented lines, run as they stand, give the gradient of the weights
    that the layer used: the routing's, its last slot overwritten with the sum of
    the others."""
    M, E, rsf = 70, 160, 2.5
    x, _, dw = route(M, k, E, F32, 3)
    if scoring == "softmax":
        w, ids = moe.grouped_topk(x, k, renorm, 8, 3, rsf)
    else:
        w, ids = moe.biased_grouped_topk(x, randn(gen(4), E, scale=0.05), k, renorm, 8, 4, rsf)
    before, given = ids.clone(), dw.clone()
    names = dict(moe=moe, w=w, ids=ids, logits=x, dw=dw, E=E, num_shared=2, factor=factor, scoring=scoring,
                 renormalize=renorm, rsf=rsf, pick=torch.randint(0, 2, (M,), generator=gen(5), device=DEV, dtype=I32))
    exec(shown("fill_shared_expert_slot"), names)
    assert bool((ids[:, -1] >= E).all()) and torch.equal(ids[:, :-1], before[:, :-1])
    # as a function of the logits: every slot's gradient reaches the slots its weight was made of
    g, mag = given.to(D), given.to(D).abs()
    if factor is not None:
        g, mag = [torch.cat([a[:, :-1] + a[:, -1:] / factor, torch.zeros_like(a[:, -1:])], 1) for a in (g, mag)]
    check(names["dlogits"], *definition(x, before, rsf * g, scoring, renorm, 0.0, rsf * mag))
    # and by differences of the filled weights along a direction
    h, d = 1e-4, torch.randn(M, E, generator=gen(6), device=DEV, dtype=D)

    def value(logits):
        v = ref.routed(logits, before, scoring, renorm, rsf, 0.0)
        if factor is not None:
            v = torch.cat([v[:, :-1], v[:, :-1].sum(1, keepdim=True) / factor], 1)
        return (v * given.to(D)).sum(1)

    want = (value(x.to(D) + h * d) - value(x.to(D) - h * d)) / (2 * h)
    size = (names["dlogits"].to(D) * d).abs().sum(1) + rsf * given.to(D).abs().sum(1)
    assert bool(((names["dlogits"].to(D) * d).sum(1) - want).abs().le(2e-5 * size).all())


def softmax_weights(x, ids):
    return torch.softmax(x, 1).gather(1, ids.long())


def sigmoid_weights(x, ids):
    p = torch.special.expit(x.gather(1, ids.long()))
    return p / p.sum(1, keepdim=True)


def top1_weight(x, ids):
    z = 30.0 * torch.tanh(x / 30.0)
    return 1 / torch.exp(z - z.gather(1, ids.long())).sum(1, keepdim=True)


# routing call -> (its result on hidden rows, renormalize, softcap, its weights' definition)
CALLS = {
    "topk_softmax": (lambda h, W, x: (*moe.topk_softmax(x, 6, False), x), False, 0.0, softmax_weights),
    "grouped_topk": (lambda h, W, x: (*moe.grouped_topk(x, 6, False, 8, 3), x), False, 0.0, softmax_weights),
    "biased_grouped_topk": (lambda h, W, x: (*moe.biased_grouped_topk(x, None, 6, True, 8, 4), x), True, 0.0,
                            sigmoid_weights),
    "fused_router_topk": (lambda h, W, x: moe.fused_router_topk(h, W, None, 6, True, 8, 4, weight_layout="ek",
                                                                return_logits=True), True, 0.0, sigmoid_weights),
    "fused_router_top1": (lambda h, W, x: moe.fused_router_top1(h, W, softcap=30.0, return_logits=True), False, 30.0,
                          top1_weight),
}


@pytest.mark.parametrize("name", list(CALLS))
def test_scoring_documented_for_each_routing_call(name):
    """With the scoring that the documentation names for a routing call,
    topk_backward is the gradient of the weights that call returns."""
    doc = " ".join(inspect.getdoc(moe.topk_backward).split())
    named = {call: scoring for scoring, calls in re.findall(r'"(softmax|sigmoid)" for ((?:``\w+``(?:, | and )?)+)', doc)
             for call in re.findall(r"``(\w+)``", calls)}
    assert set(named) == set(CALLS)
    call, renorm, cap, weights = CALLS[name]
    g = gen(7)
    h, W = randn(g, 200, 512, dtype=BF), randn(g, 256, 512, dtype=BF, scale=0.1)
    w, ids, x = call(h, W, h.float() @ W.float().T)
    xd = x.to(D).requires_grad_()
    v = weights(xd, ids)
    # a weight is a score of the routing kernels' own, to a part in 10^5
    assert bool((w.to(D) - v).abs().le(1e-5 * v).all())
    dw = randn(g, *w.shape)
    (want,) = torch.autograd.grad((v * dw.to(D)).sum(), xd)
    _, bound = definition(x, ids, dw, named[name], renorm, cap)
    # 2^-48: the 64-bit derivative's own roundings where terms cancel
    check(moe.topk_backward(dw, x, ids, named[name], renorm, softcap=cap), want,
          bound + 2.0 ** -48 * dw.to(D).abs().sum(1, keepdim=True))


@pytest.mark.parametrize("factor,scoring", [(2.5, "sigmoid"), (None, "softmax")])
def test_a_layer_with_a_shared_expert(factor, scoring):
    """Route, fill the last slot, run the layer on E + 2 experts forward and backward,
    the documented lines for the router: against autograd of all of it in 64 bits, to
    six roundings to bf16 (half a step is 2^-8) by the norm."""
    M, k, E, H, F, rsf = 90, 3, 8, 128, 64, 2.5
    g = gen(31)
    x, dout = randn(g, M, H, dtype=BF), randn(g, M, H, dtype=BF)
    W1, W2 = randn(g, E + 2, 2 * F, H, dtype=BF, scale=H ** -0.5), randn(g, E + 2, H, F, dtype=BF, scale=F ** -0.5)
    logits = randn(g, M, E)
    w, ids = (moe.topk_softmax(logits, k, True) if scoring == "softmax"
              else moe.biased_grouped_topk(logits, None, k, True, 1, 1, rsf))
    rsf = 1.0 if scoring == "softmax" else rsf
    before = ids.clone()
    pick = torch.randint(0, 2, (M,), generator=g, device=DEV, dtype=I32)

    example = shown("fill_shared_expert_slot").split("\n")
    cut = next(i for i, line in enumerate(example) if line.startswith("#"))
    names = dict(moe=moe, w=w, ids=ids, logits=logits, E=E, num_shared=2, factor=factor, pick=pick, scoring=scoring,
                 renormalize=True, rsf=rsf)
    exec("\n".join(example[:cut]), names)
    _, offsets, _, scatter, _ = moe.expert_permutation(ids, E + 2)
    xs = moe.gather_tokens(x, scatter, k)
    h, z = moe.expert_matmul(xs, W1, offsets, activation="silu", gated=True, return_preact=True)
    y = moe.expert_matmul(h, W2, offsets)
    out = moe.combine_tokens(y, scatter, w, residual=x)
    dy, names["dw"] = moe.combine_tokens_backward(dout, y, scatter, w)
    exec("\n".join(example[cut:]), names)

    leaf = logits.to(D).requires_grad_()
    v = ref.routed(leaf, before, scoring, True, rsf, 0.0)
    if factor is not None:
        v = torch.cat([v[:, :-1], v[:, :-1].sum(1, keepdim=True) / factor], 1)
    total, xd = x.to(D), x.to(D)
    for j in range(k):
        e = ids[:, j].long()
        zz = torch.einsum("mh,mnh->mn", xd, W1.to(D)[e])
        total = total + v[:, j:j + 1] * torch.einsum("mf,mhf->mh", ref.f(zz[:, :F], "silu") * zz[:, F:], W2.to(D)[e])
    (want,) = torch.autograd.grad((total * dout.to(D)).sum(), leaf)
    for got, exact in ((out, total.detach()), (names["dlogits"], want)):
        assert float((got.to(D) - exact).norm() / exact.norm()) <= 6 * 2.0 ** -8


@pytest.mark.parametrize("scoring,renorm", [("softmax", False), ("softmax", True), ("sigmoid", True)])
def test_of_a_result_in_ascending_ids(scoring, renorm):
    """sort_topk_by_id moves weights and ids together; so does their gradient."""
    M, k, E = 50, 6, 160
    x, _, dw = route(M, k, E, F32, 23)
    w, ids = (moe.topk_softmax(x, k, renorm) if scoring == "softmax"
              else moe.biased_grouped_topk(x, None, k, renorm, 1, 1, 1.0))
    moe.sort_topk_by_id(w, ids)
    v = ref.routed(x.to(D), ids, scoring, renorm, 1.0, 0.0)
    assert bool((w.to(D) - v).abs().le(1e-5 * v).all())
    check(moe.topk_backward(dw, x, ids, scoring, renorm), *definition(x, ids, dw, scoring, renorm, 0.0))


# ---------------------------------------------------------------- the ends of the logits' range

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("centre", [-80.0, -87.5, -88.5, -90.0, -104.0, -200.0, -1e30])
@pytest.mark.parametrize("scoring,renorm", [("sigmoid", True), ("sigmoid", False), ("softmax", True),
                                            ("softmax", False)])
@pytest.mark.parametrize("k", [1, 4, 12, 32])
def test_logits_far_below_zero(k, scoring, renorm, centre, dtype):
    """Rows whose sigmoids are below fp32's normal range, or vanish: the chosen
    experts' shares of their sum, and with them the gradient, are those of any
    other row."""
    x, ids, dw = route(50, k, 64, dtype, 13)
    x = (x.to(D) + centre).to(dtype)
    got = moe.topk_backward(dw, x, ids, scoring, renorm)
    check(got, *definition(x, ids, dw, scoring, renorm, 0.0))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("E", [64, 37, 1024])
@pytest.mark.parametrize("scoring,renorm,cap", [("sigmoid", True, 0.0), ("sigmoid", False, 0.0), ("softmax", True, 0.0),
                                                ("softmax", False, 0.0), ("softmax", True, 30.0),
                                                ("softmax", False, 30.0)])
def test_masked_logits(scoring, renorm, cap, E, dtype):
    """Logits of -inf (masked experts) have no gradient and take no part in the
    others'; a row of nothing else gets zeros.  A NaN stays in its row."""
    k = 6
    x, ids, dw = route(40, k, E, dtype, 17)
    low = float("-inf")
    x[0] = low                                      # a masked token
    x[1].scatter_(0, ids[1].long(), low)            # nothing chosen is left
    x[2, int(ids[2, 0])] = low                      # one of the chosen
    x[3] = low
    x[3, int(ids[3, 2])] = -1.5                     # all but one of them
    x[4].masked_fill_(torch.rand(E, generator=gen(18), device=DEV) < 0.5, low)
    x[5, int(ids[5, 1])] = float("nan")
    got = moe.topk_backward(dw, x, ids, scoring, renorm, softcap=cap)
    # a finite logit that far down has the same scores and slopes, to 2^-280
    value, bound = definition(torch.where(x == low, -1e4 if cap else -200.0, x.to(D)), ids, dw, scoring, renorm, cap)
    gone = (x == low).all(1) | ((x.gather(1, ids.long()) == low).all(1) if renorm or scoring == "sigmoid" else False)
    value[gone], bound[gone] = 0.0, 0.0
    value[x == low] = 0.0
    plain = [r for r in range(40) if r != 5]
    check(got[plain], value[plain], bound[plain])
    assert bool(got[5].isnan().any())
    if cap:  # a capped -inf is a score like others, with no slope
        assert bool((got[plain][x[plain] == low] == 0).all())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("cap", [5.0, 30.0, -30.0])
@pytest.mark.parametrize("k,E", [(1, 8), (8, 256), (20, 37)])
def test_softcap_slope_keeps_its_precision(k, E, cap, renorm, dtype):
    """Logits up to 25 caps out, where the slope 1 / cosh(t)^2 is down to 1e-21: a
    relative bound, slope and all."""
    x, ids, dw = route(60, k, E, dtype, 11, scale=8 * abs(cap))
    x = x.clamp(-25 * abs(cap), 25 * abs(cap))
    got = moe.topk_backward(dw, x, ids, "softmax", renorm, softcap=cap)
    check(got, *definition(x, ids, dw, "softmax", renorm, cap))
