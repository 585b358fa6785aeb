"""Accuracy of the expert layer's sums and activations where a bound on the worst
case says little: error in the mean of long dot products, activations far into
their tails (GPU only)."""
import math

import pytest
import torch

import moe_expert_routing_token_b200 as moe
from tests import expert_reference as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF, F32, I32, D = torch.bfloat16, torch.float32, torch.int32, torch.float64
U24 = ref.U24


def randn(g, *shape, dtype=F32):
    return torch.randn(*shape, generator=g, device=DEV).to(dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M,k,H", [(1024, 4, 7168), (1024, 4, 2890), (1100, 4, 1031), (512, 8, 7167), (600, 8, 4098),
                                   (64, 8, 7168)])
def test_weight_gradients_error_in_the_mean(M, k, H, dtype):
    """grad_weights, fp32 whatever the rows' type, by the root mean square.

    A rounding to 24 bits is off by 2^-24 / sqrt(3) of the spacing's half, 0.425 *
    2^-24 of the value in the mean over mantissas (sqrt(3 / (8 ln 2) / 3)).  A sum
    of n terms of random signs passes through partial sums of n / 2 times a term's
    variance in the mean: one chain is off by 0.425 * 2^-24 sqrt(n / 2) of the
    result.  Summed in blocks of b, blocks in turn, 32 lanes at the end, that is
    sqrt(b / 2 + n / (2 b) + 5); for the n = H / 32 values of a lane it is below
    sqrt(26) up to H = 7168 with any b of 8 to 32 (one chain: sqrt(117)).  The
    mean of 4096 errors is known to 3%: a bound at sqrt(28)."""
    g = torch.Generator(device=DEV).manual_seed(H)
    scatter = torch.randperm(M * k, generator=g, device=DEV).to(I32)
    dout, y, w = randn(g, M, H, dtype=dtype), randn(g, M * k, H, dtype=dtype), randn(g, M, k)
    _, dw = moe.combine_tokens_backward(dout, y, scatter, w)
    want = torch.stack([(y[scatter.view(M, k)[:, j].long()].to(D) * dout.to(D)).sum(1) for j in range(k)], 1)
    off = float((dw.to(D) - want).norm() / want.norm())
    assert off <= 0.425 * U24 * math.sqrt(28), off / U24


def values_of_bf16(low, high):
    """Every bf16 value between, in rows of 64 (filled up with zeros)."""
    v = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(BF).float()
    v = v[(v >= low) & (v <= high) & (v.abs() >= 2.0 ** -20)]
    v = torch.nn.functional.pad(v, (0, -len(v) % 64)).view(-1, 64)
    return v.to(BF).to(DEV)


def exact(z, act):
    """f and f' in 64 bits, with the normal distribution from erfc: from erf, as
    1 + erf, it cancels in the tail."""
    if act == "silu":
        p, q = torch.special.expit(z), torch.special.expit(-z)
        return z * p, p + z * p * q
    normal = 0.5 * torch.special.erfc(-z / math.sqrt(2))
    return z * normal, normal + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


def activation_bounds(z, act):
    """Error of f and f' at an exact z, relative to their terms.

    GELU: Phi(-|z|) = density * ratio; the density's exponent z^2 / 2 is rounded
    twice, z^2 units of 2^-24; ex2 (4 units), the fitted ratio (12 units, 20 for
    its Horner steps and the reciprocal) and products make 48.  f = max(z, 0) -
    |z| Phi(-|z|) and f' = z phi + Phi join them with a rounding of the result;
    Phi = 1 - Phi(-z) for z > 0 with one more of 1.
    SiLU: p = 1 / (1 + exp(-z)); exp's argument is rounded by 2 |z| units, and
    matters by 1 - p; ex2, sum and reciprocal make 12.  f = z p; f' = p + f (1 - p),
    where 1 - p is off by p's error.
    Exponentials and reciprocals below 2^-126 are 0."""
    u = z.abs()
    value, rate = exact(z, act)
    if act == "gelu":
        phi = torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
        tail = 0.5 * torch.special.erfc(u / math.sqrt(2))
        e = z * z + 48
        f = U24 * (e * u * tail + value.abs())
        slope = U24 * (e * tail + e * u * phi + rate.abs() + (z > 0))
    else:
        p, q = torch.special.expit(z), torch.special.expit(-z)
        e = U24 * p * (2 * u * q + 12)
        f = u * e + U24 * u * p
        slope = e + f * q + u * p * (e + U24 * (q + (z > 0))) + U24 * (rate.abs() + p * u * q)
    end = (1 + u) * 2.0 ** -125
    return f + end, slope + end


@pytest.mark.parametrize("act,low,high", [("gelu", -14.5, 14.5), ("silu", -100.0, 100.0)])
@pytest.mark.parametrize("gated", [False, True])
def test_activations_at_every_bf16_value(gated, act, low, high):
    """An identity weight makes the preactivations exact: f and f' are held to
    bounds relative to their own terms, down to where the tails leave fp32."""
    z = values_of_bf16(low, high)
    P = z.shape[0]
    off = torch.tensor([0, P], dtype=I32, device=DEV)
    one = torch.eye(64, device=DEV, dtype=BF)[None]
    f, df = exact(z.to(D), act)
    ef, edf = activation_bounds(z.to(D), act)
    bf = ref.half_step(BF)
    floor = 2.0 ** -133  # bf16's own spacing at the end of its range

    def check(got, value, bound):
        ref.within(got, (value, bound + bf * (value.abs() + bound) + floor))

    if gated:  # the other factor is a bias of one
        weight = torch.cat([one, torch.zeros_like(one)], 1).contiguous()
        bias = torch.cat([torch.zeros(1, 64, device=DEV), torch.ones(1, 64, device=DEV)], 1)
        check(moe.expert_matmul(z, weight, off, bias=bias, activation=act, gated=True), f, ef)
    else:
        check(moe.expert_matmul(z, one, off, activation=act), f, ef)
    dy = torch.ones_like(z)
    if gated:
        both = torch.cat([z, torch.ones_like(z)], 1).contiguous()
        got = moe.expert_matmul_grad_input(dy, one, off, preact=both, activation=act, gated=True)
        check(got[:, :64], df, edf)
        check(got[:, 64:], f, ef)
    else:
        check(moe.expert_matmul_grad_input(dy, one, off, preact=z, activation=act), df, edf)


LONG = [([5000], 264, 136), ([8192, 0, 2048, 2049, 4096], 256, 256), ([40000, 3, 17000], 72, 264), ([131077], 256, 64)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("positive", [False, True])
@pytest.mark.parametrize("counts,K,N", LONG)
def test_weight_gradients_of_many_rows(counts, K, N, positive, dtype):
    """The tensor core cuts its running sum at each step of 16 rows, by up to a unit
    of 2^-23; a part of 2048 rows (16384 for bf16 results) is summed that way, parts
    are joined with rounded additions.  So the error relative to the sum of the
    terms' magnitudes does not grow with the rows beyond a part's steps and half a
    unit per part.  For random signs, by the root mean square: a running sum of i of
    n steps is sqrt(i / n) of the part's in the mean, 2/3 n units of 2^-23 in all at
    the most."""
    g = torch.Generator(device=DEV).manual_seed(sum(counts))
    off = torch.tensor([0] + counts, device=DEV).cumsum(0).to(I32)
    P, part = sum(counts), 2048 if dtype == F32 else 16384
    dy, x = randn(g, P, N, dtype=BF), randn(g, P, K, dtype=BF)
    if positive:
        dy, x = dy.abs(), x.abs()
    dw = moe.expert_matmul_grad_weight(dy, x, off, dtype=dtype)
    for e, (a, b) in enumerate(zip(off.tolist(), off.tolist()[1:])):
        want, size = (torch.zeros(N, K, dtype=D, device=DEV) for _ in range(2))
        for c in range(a, b, 32768):
            d, r = dy[c:min(b, c + 32768)].to(D), x[c:min(b, c + 32768)].to(D)
            want += d.T @ r
            size += d.abs().T @ r.abs()
        parts = -(-(b - a) // part)
        bound = (ref.sum_bound(min(b - a, part)) + parts * U24) * size
        ref.within(dw[e], (want, bound + ref.half_step(dtype) * (want.abs() + bound)))
        if dtype == F32 and not positive and b > a:
            mean = (2 / 3 * (min(b - a, part) / 16 + 16) * 2 + math.sqrt(parts)) * U24
            assert float((dw[e].to(D) - want).norm() / want.norm()) <= mean
    if len(counts) == 1:
        assert torch.equal(moe.expert_matmul_grad_weight(dy, x, off, dtype=dtype), dw)
