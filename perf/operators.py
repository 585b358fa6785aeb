"""Measured cases of the expert layer's operators: tokens sorted by expert and back, the experts' products, and the
gradients down to the router's logits.

A case names its operator in ``"op"``:

    gather         rows of x copied to their places in expert order
    gather_grad    its gradient: each token sums the rows of its places
    combine        each token's rows of y, weighted and summed, plus a residual
    combine_grad   its gradients: rows of y and routing weights
    matmul         x W_e^T over the experts' segments, with bias, activation (gated or not) and residual
    matmul_dx      its input gradient, through the activation in front of it
    matmul_dw      its weight and bias gradients
    topk_grad      gradient of the routing weights with respect to the router's logits

``M`` tokens choose ``k`` of ``E_all`` experts, of which the first ``E`` are held here (one device's share where
experts are spread over devices; pairs of other experts have no place).
"""
import math

import torch

own = False

BF16, F32 = torch.bfloat16, torch.float32
DTYPES = {"bf16": BF16, "f32": F32}


def listed():
    """Hidden sizes, expert counts, top-k and token counts of the routing workloads (7168 with 256 experts and 8
    slots, 160 with 6, 8 with 2); the experts' inner sizes are generic."""
    return [
        # a long prefill or training batch: bandwidth counts
        dict(name="gather prefill", op="gather", M=16384, k=8, E=256, E_all=256, H=7168, dtype="bf16"),
        # training in fp32 on an odd width, an eighth of the experts held here
        dict(name="gather grad ragged", op="gather_grad", M=8191, k=6, E=20, E_all=160, H=1031, dtype="f32"),
        # a decode batch brought back, added to the residual stream
        dict(name="combine decode", op="combine", M=64, k=8, E=256, E_all=256, H=7168, dtype="bf16", residual=True),
        # backward of the combine of a training batch
        dict(name="combine grad", op="combine_grad", M=8192, k=8, E=256, E_all=256, H=7168, dtype="bf16"),
        # a small layer, one token: latency of a single call
        dict(name="matmul one token", op="matmul", M=1, k=2, E=8, E_all=8, K=1024, N=512, act="silu", gated=True,
             bias=False, residual=False, preact=False),
        # first product of a decode batch: the experts' weights are read once, little else
        dict(name="matmul decode", op="matmul", M=64, k=8, E=32, E_all=256, K=7168, N=2048, act="silu", gated=True,
             bias=False, residual=False, preact=False),
        # first product of a training batch, its inputs to the activation kept for the backward pass
        dict(name="matmul train", op="matmul", M=4096, k=8, E=32, E_all=32, K=7168, N=2048, act="silu", gated=True,
             bias=False, residual=False, preact=True),
        # second product on uneven sizes, with every part of the epilogue
        dict(name="matmul bias residual", op="matmul", M=1500, k=6, E=160, E_all=160, K=1544, N=5128, act="gelu",
             gated=False, bias=True, residual=True, preact=False),
        # input gradient of the second product, through the gated activation
        dict(name="matmul grad input", op="matmul_dx", M=4096, k=8, E=32, E_all=32, K=2048, N=7168, act="silu",
             gated=True),
        # weight and bias gradients of the second product
        dict(name="matmul grad weight", op="matmul_dw", M=4096, k=8, E=32, E_all=32, K=2048, N=7168, bias=True),
        # the router's gradients: of a small batch through the dense softmax, of a training batch
        dict(name="topk grad softmax", op="topk_grad", M=64, k=6, E=160, E_all=160, dtype="f32", scoring="softmax",
             renorm=False, rsf=1.0, softcap=0.0),
        dict(name="topk grad", op="topk_grad", M=16384, k=8, E=256, E_all=256, dtype="bf16", scoring="sigmoid",
             renorm=True, rsf=2.5, softcap=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """A case of the same ranges: every operator, from one token to the largest batch that costs no more than the
    listed ones."""
    op = rng.choice(["gather", "gather_grad", "combine", "combine_grad", "matmul", "matmul", "matmul_dx", "matmul_dw",
                     "topk_grad"])
    E_all, k = rng.choice([(8, 2), (32, 4), (160, 6), (256, 8)])
    if op == "topk_grad":
        scoring = rng.choice(["softmax", "sigmoid"])
        return dict(op=op, M=_log(rng, 1, 16384), k=k, E=E_all, E_all=E_all, dtype=rng.choice(["bf16", "f32"]),
                    scoring=scoring, renorm=rng.random() < 0.5, rsf=rng.choice([1.0, 2.5]),
                    softcap=30.0 if scoring == "softmax" and rng.random() < 0.3 else 0.0)
    share = rng.choice([1, 1, 2, 8])
    E, least = E_all // share, 1 if share == 1 else -(-8 * share // k)  # a few pairs have a place here
    if not op.startswith("matmul"):
        dtype = rng.choice(["bf16", "f32"])
        H = _log(rng, 64, 7168)
        if rng.random() < 0.5:
            H = -(-H // 64) * 64
        most = min(16384, 16384 * 7168 * 8 * 2 // (H * k * (2 if dtype == "bf16" else 4) * 2))
        case = dict(op=op, M=_log(rng, least, most), k=k, E=E, E_all=E_all, H=H, dtype=dtype)
        if op == "combine":
            case["residual"] = rng.random() < 0.5
        return case
    gated = rng.random() < 0.5 and op != "matmul_dw"
    K = 8 * _log(rng, 16, 896)
    N = 8 * _log(rng, 16, 640)
    while E * K * N * (2 if gated and op == "matmul" else 1) > 32 * 7168 * 4096:
        K, N = max(128, K // 16 * 8), max(128, N // 16 * 8)
    flops = 2 * K * N * (2 if gated and op == "matmul" else 1) * k * E / E_all
    case = dict(op=op, M=_log(rng, least, max(least, min(8192, int(0.9e12 / flops)))), k=k, E=E, E_all=E_all, K=K, N=N)
    if op == "matmul_dw":
        return dict(case, bias=rng.random() < 0.5)
    case.update(act=rng.choice(["silu", "gelu"] if gated else ["none", "silu", "gelu"]), gated=gated)
    if op == "matmul":
        case.update(bias=rng.random() < 0.5, residual=rng.random() < 0.4, preact=rng.random() < 0.3)
    return case


def _route(case, gen):
    """A routing result of mildly uneven load and its expert order: what the routing and permutation calls give.
    Returns weights (M, k), ids (M, k), offsets (E + 1), gather (P), scatter (P), placed pairs, largest segment."""
    M, k, E, E_all = case["M"], case["k"], case["E"], case["E_all"]
    dev = "cuda"
    score = torch.randn(M, E_all, generator=gen, device=dev) + 0.15 * torch.randn(E_all, generator=gen, device=dev)
    top, ids = score.topk(k, dim=1)
    weights = torch.softmax(top, dim=1).contiguous()
    ids = torch.where(ids < E, ids, -1).to(torch.int32).contiguous()
    flat = ids.reshape(-1).long()
    order = torch.sort(torch.where(flat < 0, E, flat), stable=True).indices
    counts = torch.bincount(flat + 1, minlength=E + 1)[1:]
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=dev)
    offsets[1:] = counts.cumsum(0)
    n = int(offsets[-1])
    scatter = torch.full((M * k,), -1, dtype=torch.int32, device=dev)
    scatter[order[:n]] = torch.arange(n, dtype=torch.int32, device=dev)
    return weights, ids, offsets, order.to(torch.int32), scatter, n, max(1, int(counts.max()))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))

    def rand(*shape, scale=1.0, dtype=BF16):
        return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)

    M, k, E, op = case["M"], case["k"], case["E"], case["op"]
    weights, ids, offsets, gather, scatter, n, most = _route(case, gen)
    s = dict(case=case, weights=weights, ids=ids, offsets=offsets, gather=gather, scatter=scatter, n=n, most=most)
    P = M * k
    if op == "topk_grad":
        s["logits"] = rand(M, E, scale=2.0, dtype=DTYPES[case["dtype"]])
        s["ids"] = s["logits"].topk(k, dim=1).indices.to(torch.int32).contiguous()
        s["dweights"] = rand(M, k, dtype=F32)
        return s
    if not op.startswith("matmul"):
        H, dtype = case["H"], DTYPES[case["dtype"]]
        if op == "gather":
            s["x"], s["out"] = rand(M, H, dtype=dtype), torch.zeros(P, H, dtype=dtype, device="cuda")
        elif op == "gather_grad":
            s["dsorted"] = rand(P, H, dtype=dtype)
        else:
            s["y"] = rand(P, H, dtype=dtype)
            if op == "combine":
                s["residual"] = rand(M, H, dtype=dtype) if case["residual"] else None
            else:
                s["dout"], s["out"] = rand(M, H, dtype=dtype), torch.zeros(P, H, dtype=dtype, device="cuda")
        return s
    K, N = case["K"], case["N"]
    if op == "matmul":
        Nw = 2 * N if case["gated"] else N
        s["x"], s["W"] = rand(P, K), torch.empty(E, Nw, K, dtype=BF16, device="cuda")
        s["bias"] = rand(E, Nw, scale=0.5, dtype=F32) if case["bias"] else None
        s["residual"] = rand(P, N) if case["residual"] else None
        s["out"] = torch.zeros(P, N, dtype=BF16, device="cuda")
        s["preact"] = torch.zeros(P, Nw, dtype=BF16, device="cuda") if case["preact"] else None
    elif op == "matmul_dx":
        Kz = 2 * K if case["gated"] else K
        s["dy"], s["W"] = rand(P, N), torch.empty(E, N, K, dtype=BF16, device="cuda")
        s["preact"] = rand(P, Kz) if case["act"] != "none" or case["gated"] else None
        s["out"] = torch.zeros(P, Kz, dtype=BF16, device="cuda")
    else:
        s["dy"], s["x"] = rand(P, N), rand(P, K)
    if "W" in s:
        # a trained layer's scale: outputs of about one
        s["W"].normal_(0.0, 1.0 / math.sqrt(s["W"].shape[2] if op == "matmul" else N), generator=gen)
    return s


# ---------------------------------------------------------------- one pass


def run(s):
    return _own(s) if own else PLAIN[s["case"]["op"]](s, s["case"])


def _own(s):
    import moe_expert_routing_token_b200 as moe

    c = s["case"]
    op, k = c["op"], c["k"]
    if op == "gather":
        return moe.gather_tokens(s["x"], s["scatter"], k, out=s["out"])
    if op == "gather_grad":
        return moe.gather_tokens_backward(s["dsorted"], s["scatter"], k)
    if op == "combine":
        return moe.combine_tokens(s["y"], s["scatter"], s["weights"], residual=s["residual"])
    if op == "combine_grad":
        return moe.combine_tokens_backward(s["dout"], s["y"], s["scatter"], s["weights"], grad_y=s["out"])
    if op == "matmul":
        return moe.expert_matmul(s["x"], s["W"], s["offsets"], bias=s["bias"], activation=c["act"], gated=c["gated"],
                                 residual=s["residual"], out=s["out"], preact_out=s["preact"])
    if op == "matmul_dx":
        return moe.expert_matmul_grad_input(s["dy"], s["W"], s["offsets"], preact=s["preact"], activation=c["act"],
                                            gated=c["gated"], out=s["out"])
    if op == "matmul_dw":
        return moe.expert_matmul_grad_weight(s["dy"], s["x"], s["offsets"], bias_grad=c["bias"])
    return moe.topk_backward(s["dweights"], s["logits"], s["ids"], c["scoring"], c["renorm"], c["rsf"],
                             softcap=c["softcap"])


# ---------------------------------------------------------------- plain forms


def _gather(s, c):
    s["out"][: s["n"]] = s["x"][s["gather"][: s["n"]].long() // c["k"]]
    return s["out"]


def _rows(s, c, y):
    """Each pair's row of y in fp32, zero for pairs without a place: (M, k, H)."""
    at = s["scatter"].long().view(c["M"], c["k"])
    return torch.where((at >= 0)[:, :, None], y[at.clamp(min=0)].float(), 0.0), at >= 0


def _gather_grad(s, c):
    rows, _ = _rows(s, c, s["dsorted"])
    return rows.sum(1).to(s["dsorted"].dtype)


def _combine(s, c):
    rows, _ = _rows(s, c, s["y"])
    out = (rows * s["weights"][:, :, None]).sum(1)
    if s["residual"] is not None:
        out = out + s["residual"].float()
    return out.to(s["y"].dtype)


def _combine_grad(s, c):
    rows, placed = _rows(s, c, s["y"])
    dweights = (rows * s["dout"].float()[:, None, :]).sum(2)
    at = s["gather"][: s["n"]].long()
    s["out"][: s["n"]] = (s["weights"].reshape(-1)[at][:, None] * s["dout"][at // c["k"]].float()).to(s["out"].dtype)
    return s["out"], torch.where(placed, dweights, 0.0)


def _padded(s, c, x):
    """The segments of x, padded to the largest one: (E, most, columns) fp32; and each sorted row's place in it."""
    off = s["offsets"].long()
    at = off[:-1, None] + torch.arange(s["most"], device=off.device)
    x_pad = torch.where((at < off[1:, None])[:, :, None], x[at.clamp(max=x.shape[0] - 1)].float(), 0.0)
    row = torch.arange(s["n"], device=off.device)
    e = torch.bucketize(row, off[1:], right=True)
    return x_pad, e * s["most"] + row - off[e], e


def _act(z, act):
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    return z


def _act_grad(z, act):
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    return torch.ones_like(z)


def _matmul(s, c):
    x_pad, at, e = _padded(s, c, s["x"])
    z = torch.bmm(x_pad, s["W"].float().transpose(1, 2)).reshape(-1, s["W"].shape[1])[at]
    if s["bias"] is not None:
        z = z + s["bias"][e]
    if s["preact"] is not None:
        s["preact"][: s["n"]] = z.to(BF16)
    h = _act(z[:, : c["N"]], c["act"]) * z[:, c["N"]:] if c["gated"] else _act(z, c["act"])
    if s["residual"] is not None:
        h = h + s["residual"][: s["n"]].float()
    s["out"][: s["n"]] = h.to(BF16)
    return (s["out"], s["preact"]) if s["preact"] is not None else s["out"]


def _matmul_dx(s, c):
    dy_pad, at, _ = _padded(s, c, s["dy"])
    q = torch.bmm(dy_pad, s["W"].float()).reshape(-1, c["K"])[at]
    if s["preact"] is not None:
        z = s["preact"][: s["n"]].float()
        g = z[:, : c["K"]]
        if c["gated"]:
            q = torch.cat([q * z[:, c["K"]:] * _act_grad(g, c["act"]), q * _act(g, c["act"])], dim=1)
        else:
            q = q * _act_grad(g, c["act"])
    s["out"][: s["n"]] = q.to(BF16)
    return s["out"]


def _matmul_dw(s, c):
    dy_pad, _, _ = _padded(s, c, s["dy"])
    x_pad, _, _ = _padded(s, c, s["x"])
    dW = torch.bmm(dy_pad.transpose(1, 2), x_pad).to(BF16)
    return (dW, dy_pad.sum(1)) if c["bias"] else dW


def _topk_grad(s, c):
    x, ids = s["logits"].float(), s["ids"].long()
    g = c["rsf"] * s["dweights"]
    slope = 1.0
    if c["softcap"]:
        t = torch.tanh(x / c["softcap"])
        x, slope = t * c["softcap"], 1.0 - t * t
    dense = torch.zeros_like(x)
    if c["scoring"] == "softmax" and not c["renorm"]:
        e = torch.exp(x - x.amax(1, keepdim=True))
        p = e / e.sum(1, keepdim=True)
        pj = p.gather(1, ids)
        dz = p * (dense.scatter(1, ids, g) - (g * pj).sum(1, keepdim=True))
    elif c["scoring"] == "softmax":
        xj = x.gather(1, ids)
        v = torch.exp(xj - xj.amax(1, keepdim=True))
        v = v / v.sum(1, keepdim=True)
        dz = dense.scatter(1, ids, v * (g - (g * v).sum(1, keepdim=True)))
    else:
        p = 1.0 / (1.0 + torch.exp(-x.gather(1, ids)))
        if c["renorm"]:
            total = p.sum(1, keepdim=True)
            g = (g - (g * p).sum(1, keepdim=True) / total) / total
        dz = dense.scatter(1, ids, g * p * (1.0 - p))
    return (dz * slope).to(s["logits"].dtype)


PLAIN = {"gather": _gather, "gather_grad": _gather_grad, "combine": _combine, "combine_grad": _combine_grad,
         "matmul": _matmul, "matmul_dx": _matmul_dx, "matmul_dw": _matmul_dw, "topk_grad": _topk_grad}


# ---------------------------------------------------------------- what a pass cannot do without


def work(case):
    M, k, E, op = case["M"], case["k"], case["E"], case["op"]
    P = M * k
    n = P * E / case["E_all"]  # pairs placed here, on average
    if op == "topk_grad":
        b = 2 if case["dtype"] == "bf16" else 4
        dense = case["scoring"] == "softmax" and not case["renorm"]
        return {"bytes": M * E * b + (M * E * b if dense else P * b) + 8 * P, "flops": (6 * M * E if dense else 0) + 12 * P}
    if not op.startswith("matmul"):
        H, b = case["H"], 2 if case["dtype"] == "bf16" else 4
        token, rows = M * H * b, n * H * b
        return {"gather": {"bytes": token + rows + 4 * P, "flops": 0},
                "gather_grad": {"bytes": token + rows + 4 * P, "flops": n * H},
                "combine": {"bytes": token * (2 if case.get("residual") else 1) + rows + 8 * P, "flops": 2 * n * H},
                "combine_grad": {"bytes": token + 2 * rows + 12 * P, "flops": 3 * n * H}}[op]
    K, N = case["K"], case["N"]
    active = E * (1.0 - (1.0 - 1.0 / case["E_all"]) ** P)  # experts with a row, on average
    if op == "matmul":
        Nw = 2 * N if case["gated"] else N
        size = n * K * 2 + active * Nw * K * 2 + n * N * 2 * (2 if case["residual"] else 1)
        size += (active * Nw * 4 if case["bias"] else 0) + (n * Nw * 2 if case["preact"] else 0)
        return {"bytes": size, "flops": 2.0 * n * Nw * K}
    if op == "matmul_dx":
        Kz = 2 * K if case["gated"] else K
        through = case["act"] != "none" or case["gated"]
        return {"bytes": n * N * 2 + active * N * K * 2 + n * Kz * 2 * (2 if through else 1), "flops": 2.0 * n * N * K}
    return {"bytes": n * (N + K) * 2 + E * N * K * 2 + (E * N * 4 if case["bias"] else 0), "flops": 2.0 * n * N * K}


# ---------------------------------------------------------------- the definitions in 64 bits


def _ranges(s):
    off = s["offsets"].tolist()
    return [(e, a, b) for e, (a, b) in enumerate(zip(off, off[1:])) if b > a]


def _f(z, act):
    if act == "silu":
        return z * torch.special.expit(z)
    if act == "gelu":
        return z * torch.special.ndtr(z)
    return z


def _df(z, act):
    if act == "silu":
        p = torch.special.expit(z)
        return p + z * p * torch.special.expit(-z)
    if act == "gelu":
        return torch.special.ndtr(z) + z * torch.exp(-z.square() / 2) * (2 * math.pi) ** -0.5
    return torch.ones_like(z)


def exact(case, seed):
    s = prepare(case, seed)
    c, D = case, torch.float64
    op, M, k, n = c["op"], c["M"], c["k"], s["n"]
    pair = s["gather"][:n].long()
    token, w = pair // k, s["weights"].reshape(-1).to(D)
    if op == "gather":
        out = torch.zeros(M * k, c["H"], dtype=D, device="cuda")
        out[:n] = s["x"].to(D).index_select(0, token)
        return out
    if op == "gather_grad":
        return torch.zeros(M, c["H"], dtype=D, device="cuda").index_add_(0, token, s["dsorted"][:n].to(D))
    if op == "combine":
        out = torch.zeros(M, c["H"], dtype=D, device="cuda") if s["residual"] is None else s["residual"].to(D)
        return out.index_add_(0, token, s["y"][:n].to(D) * w[pair, None])
    if op == "combine_grad":
        dy, dw = torch.zeros(M * k, c["H"], dtype=D, device="cuda"), torch.zeros(M * k, dtype=D, device="cuda")
        for a in range(0, n, 16384):
            b = min(n, a + 16384)
            d = s["dout"].index_select(0, token[a:b]).to(D)
            dy[a:b] = d * w[pair[a:b], None]
            dw[pair[a:b]] = torch.linalg.vecdot(d, s["y"][a:b].to(D))
        return dy, dw.view(M, k)
    if op == "matmul":
        out = torch.zeros(M * k, c["N"], dtype=D, device="cuda")
        kept = torch.zeros(M * k, s["W"].shape[1], dtype=D, device="cuda") if c["preact"] else None
        for e, a, b in _ranges(s):
            z = s["x"][a:b].to(D) @ s["W"][e].to(D).T
            if c["bias"]:
                z += s["bias"][e].to(D)
            if kept is not None:
                kept[a:b] = z
            if c["gated"]:
                gate, up = z.chunk(2, dim=1)
                z = _f(gate, c["act"]) * up
            else:
                z = _f(z, c["act"])
            out[a:b] = z if s["residual"] is None else z + s["residual"][a:b].to(D)
        return (out, kept) if kept is not None else out
    if op == "matmul_dx":
        out = torch.zeros(s["out"].shape, dtype=D, device="cuda")
        for e, a, b in _ranges(s):
            q = s["dy"][a:b].to(D) @ s["W"][e].to(D)
            if s["preact"] is None:
                out[a:b] = q
            elif c["gated"]:
                gate, up = s["preact"][a:b].to(D).chunk(2, dim=1)
                out[a:b, : c["K"]] = q * up * _df(gate, c["act"])
                out[a:b, c["K"]:] = q * _f(gate, c["act"])
            else:
                out[a:b] = q * _df(s["preact"][a:b].to(D), c["act"])
        return out
    if op == "matmul_dw":
        dW = torch.zeros(c["E"], c["N"], c["K"], dtype=D, device="cuda")
        db = torch.zeros(c["E"], c["N"], dtype=D, device="cuda")
        for e, a, b in _ranges(s):
            d = s["dy"][a:b].to(D)
            dW[e] = d.T @ s["x"][a:b].to(D)
            db[e] = d.sum(0)
        return (dW, db) if c["bias"] else dW
    # the routing weights as a function of the logits, differentiated
    x = s["logits"].to(D).requires_grad_()
    z = c["softcap"] * torch.tanh(x / c["softcap"]) if c["softcap"] else x
    p = torch.special.expit(z) if c["scoring"] == "sigmoid" else torch.softmax(z, dim=1)
    chosen = torch.take_along_dim(p, s["ids"].long(), dim=1)
    if c["renorm"]:
        chosen = chosen / chosen.sum(1, keepdim=True)
    return torch.autograd.grad((chosen * c["rsf"] * s["dweights"].to(D)).sum(), x)[0]
