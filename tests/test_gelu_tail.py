"""The fitted ratio behind the expert products' GELU, from the source's constants
(CPU only)."""
import os
import re

import numpy as np
import torch

SOURCE = os.path.join(os.path.dirname(__file__), "..", "moe_expert_routing_token_b200", "csrc", "expert_matmul.cu")


def coefficients():
    """Numerator and denominator of mills(), highest power first."""
    text = open(SOURCE).read()
    body = text[text.index("float2 mills("):]
    body = body[:body.index("return")]
    numbers = [[np.float32(v) for line in body.split("\n") if re.search(rf"\b{name} = ", line)
                for v in re.findall(r"(\d+\.\d+)f", line)] for name in ("p", "q")]
    assert [len(n) for n in numbers] == [4, 5]
    return numbers


def ratio(p, q, t):
    def horner(c):
        v = np.full_like(t, c[0])
        for a in c[1:]:
            v = (v.astype(np.float64) * t + a).astype(np.float32)  # a fused multiply-add: one rounding
        return v

    return (horner(p) / horner(q)).astype(np.float64)


def error(p, q):
    t = np.linspace(0, 14, 1400001).astype(np.float32)
    want = np.sqrt(np.pi / 2) * torch.special.erfcx(torch.from_numpy(t).double() / 2 ** 0.5).numpy()
    return float(np.abs(ratio(p, q, t) / want - 1).max())


def test_the_fit_over_its_range():
    """12 units of 2^-24 for the fit and 20 for its steps: what the bound of the GPU
    test of the activations takes for them."""
    assert error(*coefficients()) <= 32 * 2.0 ** -24


def test_a_wrong_coefficient_is_seen():
    p, q = coefficients()
    for c in (p, q):
        for i in range(len(c)):
            kept = c[i]
            c[i] = np.float32(kept * 1.0001)
            assert error(p, q) > 32 * 2.0 ** -24
            c[i] = kept
