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
