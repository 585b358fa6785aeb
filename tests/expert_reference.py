"""The expert layer's operators in 64 bits, one segment or slot at a time, and
the error bounds that their fp32 kernels are held to."""
import math

import torch

D = torch.float64
U24 = 2.0 ** -24


def half_step(dtype):
    """Largest rounding error relative to the value."""
    return torch.finfo(dtype).eps / 2


def segments(offsets):
    off = [int(v) for v in offsets]
    return [(e, a, b) for e, (a, b) in enumerate(zip(off, off[1:])) if b > a]


def f(z, act):
    if act == "silu":
        return z * torch.special.expit(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    return z


def df(z, act):
    if act == "silu":
        p = torch.special.expit(z)
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    return torch.ones_like(z)


def sum_bound(n):
    """Error of a tensor-core sum of n exact products relative to the sum of
    their magnitudes: 16 products a step, the running sum cut (not rounded) to
    24 bits at each, and 16 more such steps for the products aligned to the
    largest of a step and the joining of parts."""
    return (math.ceil(n / 16) + 16) * 2 * U24


# |f'| <= 1.13 for both activations.  act_error is absolute: an approximate
# exponential (its argument carries roundings of z) and reciprocal, and GELU's
# fitted ratio, a few units of 2^-23 of the result's largest term.  It is wide far
# into the tails; tests/test_gpu_expert_accuracy.py bounds those relative to them.
SLOPE = 1.13


def act_error(z, act):
    return (8 + z.abs()) * 2 * U24 * (z.abs() + 1) if act != "none" else torch.zeros_like(z)


def matmul(x, w, offsets, bias, act, gated, residual):
    """{name: (value, bound)} of out and preact; rows behind the last segment
    are left NaN."""
    P, Nz = x.shape[0], w.shape[1]
    N = Nz // 2 if gated else Nz
    z = torch.full((P, Nz), float("nan"), dtype=D, device=x.device)
    dz = torch.zeros_like(z)
    for e, a, b in segments(offsets):
        xe, we = x[a:b].to(D), w[e].to(D)
        z[a:b] = xe @ we.T
        size = xe.abs() @ we.abs().T
        if bias is not None:
            z[a:b] += bias[e].to(D)
            size = size + bias[e].to(D).abs()
        dz[a:b] = sum_bound(x.shape[1] + 16) * size
    bf = half_step(torch.bfloat16)
    preact = (z, dz + bf * (z.abs() + dz))
    if gated:
        g, u, dg, du = z[:, :N], z[:, N:], dz[:, :N], dz[:, N:]
        h = f(g, act) * u
        fg = SLOPE * dg + act_error(g, act)
        dh = fg * (u.abs() + du) + f(g, act).abs() * du + 2 * U24 * h.abs()
    else:
        h, dh = f(z, act), SLOPE * dz + act_error(z, act)
    if residual is not None:
        h = h + residual.to(D)
        dh = dh + U24 * h.abs()
    return {"out": (h, dh + bf * (h.abs() + dh)), "preact": preact}


def grad_input(dy, w, offsets, preact, act, gated):
    P, K = dy.shape[0], w.shape[2]
    q = torch.full((P, K), float("nan"), dtype=D, device=dy.device)
    dq = torch.zeros_like(q)
    for e, a, b in segments(offsets):
        q[a:b] = dy[a:b].to(D) @ w[e].to(D)
        dq[a:b] = sum_bound(dy.shape[1]) * (dy[a:b].to(D).abs() @ w[e].to(D).abs())
    bf = half_step(torch.bfloat16)

    def through(m, dm):
        v = q * m
        d = dq * (m.abs() + dm) + q.abs() * dm + 2 * U24 * v.abs()
        return v, d + bf * (v.abs() + d)

    if preact is None:
        return q, dq + bf * (q.abs() + dq)
    z = preact.to(D)
    if not gated:
        return through(df(z, act), act_error(z, act))
    g, u = z[:, :K], z[:, K:]
    parts = [through(u * df(g, act), u.abs() * act_error(g, act)), through(f(g, act), act_error(g, act))]
    return tuple(torch.cat(p, dim=1) for p in zip(*parts))


def grad_weight(dy, x, offsets, E, dtype):
    dw = torch.zeros(E, dy.shape[1], x.shape[1], dtype=D, device=dy.device)
    dd = torch.zeros_like(dw)
    db = torch.zeros(E, dy.shape[1], dtype=D, device=dy.device)
    ddb = torch.zeros_like(db)
    for e, a, b in segments(offsets):
        g, xe = dy[a:b].to(D), x[a:b].to(D)
        dw[e] = g.T @ xe
        dd[e] = sum_bound(b - a) * (g.abs().T @ xe.abs())
        db[e] = g.sum(0)
        ddb[e] = (b - a) * U24 * g.abs().sum(0)
    u = half_step(dtype)
    return (dw, dd + u * (dw.abs() + dd)), (db, ddb + U24 * db.abs())


def rows_of(y, scatter, k):
    """(M, k, H) rows of the pairs in 64 bits, zeros for pairs without a
    place, and which have one."""
    at = scatter.long().view(-1, k)
    placed = at >= 0
    return torch.where(placed[:, :, None], y[at.clamp(min=0)].to(D), 0.0), placed


def combine(y, scatter, weights, residual, k):
    rows, _ = rows_of(y, scatter, k)
    terms = rows if weights is None else rows * weights.to(D)[:, :, None]
    v, size = terms.sum(1), terms.abs().sum(1)
    if residual is not None:
        v, size = v + residual.to(D), size + residual.to(D).abs()
    d = (k + 1) * U24 * size  # one rounding per term and one for the residual
    return v, d + half_step(y.dtype) * (v.abs() + d)


def routed(x, ids, scoring, renorm, rsf, softcap):
    """Routing weights of 64-bit logits for fixed ids (all inside [0, E))."""
    z = softcap * torch.tanh(x / softcap) if softcap else x
    p = torch.special.expit(z) if scoring == "sigmoid" else torch.softmax(z, dim=1)
    w = p.gather(1, ids.long())
    return rsf * (w / w.sum(1, keepdim=True) if renorm else w)


def within(got, value_bound, where=None):
    value, bound = value_bound
    got = got.to(D)
    if where is not None:
        got, value, bound = got[where], value[where], bound[where]
    bad = ~((got - value).abs() <= bound)
    assert not bool(bad.any()), (
        f"{int(bad.sum())} of {bad.numel()} values out of bounds, first at {bad.nonzero()[0].tolist()}: "
        f"{float(got[bad][0])} for {float(value[bad][0])} +- {float(bound[bad][0])}")
