"""Refusals of the expert layer's calls: by the C library before any CUDA
call, and by the binding (CPU only)."""
import pytest
import torch

import moe_expert_routing_token_b200 as moe

P = 4096  # a non-null, aligned dummy address; never dereferenced on these paths


@pytest.fixture(scope="module")
def lib():
    return moe.lib()


def refused(lib, status, want, needle):
    assert status == want
    assert needle in lib.moe_last_error().decode()


@pytest.mark.parametrize("args,want,needle", [
    # (x, dtype, M, H, scatter, k, sorted, stream)
    ((P, 3, 4, 8, P, 2, P, None), 1, "dtype"),
    ((P, 0, -1, 8, P, 2, P, None), 1, "M=-1"),
    ((P, 0, 4, 0, P, 2, P, None), 1, "H=0"),
    ((P, 0, 4, 8, P, 0, P, None), 1, "k=0"),
    ((P, 0, 1 << 30, 8, P, 2, P, None), 2, "2^31"),
    ((P, 0, 1 << 62, 8, P, 2, P, None), 2, "2^31"),
    ((None, 0, 4, 8, P, 2, P, None), 1, "null"),
    ((P, 0, 4, 8, None, 2, P, None), 1, "null"),
    ((P, 0, 4, 8, P, 2, None, None), 1, "null"),
    ((P + 2, 0, 4, 8, P, 2, P, None), 1, "aligned"),
    ((P + 1, 1, 4, 8, P, 2, P, None), 1, "aligned"),
    ((P, 1, 4, 8, P + 2, 2, P, None), 1, "aligned"),
])
def test_gather_tokens(lib, args, want, needle):
    refused(lib, lib.moe_gather_tokens(*args), want, needle)
    refused(lib, lib.moe_gather_tokens_backward(*args), want, needle)


def test_combine_tokens(lib):
    # (y, dtype, M, H, scatter, k, weights, residual, out, stream)
    call = lib.moe_combine_tokens
    refused(lib, call(P, 5, 4, 8, P, 2, P, None, P, None), 1, "dtype")
    refused(lib, call(P, 0, 4, 8, P, 2, None, None, P, None), 1, "null")
    refused(lib, call(P, 0, 4, 8, P, 2, P, P + 2, P, None), 1, "aligned")
    refused(lib, call(P, 0, 1 << 40, 8, P, 2, P, None, P, None), 2, "2^31")
    assert call(None, 0, 0, 8, None, 2, None, None, None, None) == 0
    # (grad_out, y, dtype, M, H, scatter, k, weights, grad_y, grad_weights, stream)
    back = lib.moe_combine_tokens_backward
    refused(lib, back(P, P, 0, 4, 8, P, 2, P, P, None, None), 1, "null")
    refused(lib, back(P, None, 0, 4, 8, P, 2, P, P, P, None), 1, "null")
    refused(lib, back(P, P, 0, 4, -8, P, 2, P, P, P, None), 1, "H=-8")
    assert back(None, None, 1, 0, 8, None, 2, None, None, None, None) == 0


def test_expert_matmul(lib):
    def call(x=P, w=P, off=P, rows=64, K=64, N=64, E=4, bias=None, act=0, gated=0, residual=None, out=P, preact=None):
        return lib.moe_expert_matmul(x, w, off, rows, K, N, E, bias, act, gated, residual, out, preact, None)

    refused(lib, call(rows=-1), 1, "P=-1")
    refused(lib, call(K=0), 1, "K=0")
    refused(lib, call(E=0), 1, "E=0")
    refused(lib, call(act=3), 1, "activation 3")
    refused(lib, call(act=-1), 1, "activation -1")
    refused(lib, call(gated=2), 1, "gated 2")
    refused(lib, call(K=60), 2, "multiples of 8")
    refused(lib, call(N=4), 2, "multiples of 8")
    refused(lib, call(E=1025), 2, "E=1025")
    refused(lib, call(rows=1 << 31), 2, "2^31")
    for name in ("x", "w", "off", "out"):
        refused(lib, call(**{name: None}), 1, "null")
    for name in ("x", "w", "out", "residual", "preact"):
        refused(lib, call(**{name: P + 8}), 1, "aligned")
    refused(lib, call(bias=P + 2), 1, "aligned")
    assert call(rows=0, x=None, w=None, off=None, out=None) == 0


def test_expert_matmul_gradients(lib):
    def dx(dy=P, w=P, off=P, rows=64, K=64, N=64, E=4, preact=None, act=0, gated=0, out=P):
        return lib.moe_expert_matmul_grad_input(dy, w, off, rows, K, N, E, preact, act, gated, out, None)

    refused(lib, dx(act=1), 1, "preact")
    refused(lib, dx(gated=1), 1, "preact")
    refused(lib, dx(preact=P + 2), 1, "aligned")
    refused(lib, dx(N=63), 2, "multiples of 8")
    assert dx(rows=0, dy=None, w=None, off=None, out=None) == 0

    def dw(dy=P, x=P, off=P, rows=64, K=64, N=64, E=4, dtype=1, out=P, db=None):
        return lib.moe_expert_matmul_grad_weight(dy, x, off, rows, K, N, E, dtype, out, db, None)

    refused(lib, dw(dtype=2), 1, "dtype")
    refused(lib, dw(dy=None), 1, "null")
    refused(lib, dw(rows=0, dy=None, x=None, out=None), 1, "null")
    refused(lib, dw(out=P + 4), 1, "aligned")
    refused(lib, dw(db=P + 1), 1, "aligned")
    refused(lib, dw(E=2000), 2, "E=2000")


def test_topk_backward(lib):
    def call(g=P, x=P, dtype=0, ids=P, M=4, E=8, k=2, scoring=0, renorm=1, rsf=1.0, cap=0.0, out=P):
        return lib.moe_topk_backward(g, x, dtype, ids, M, E, k, scoring, renorm, rsf, cap, out, None)

    refused(lib, call(dtype=9), 1, "dtype")
    refused(lib, call(M=-2), 1, "M must")
    refused(lib, call(k=0), 1, "positive")
    refused(lib, call(scoring=2), 1, "scoring")
    refused(lib, call(rsf=float("inf")), 1, "scaling")
    refused(lib, call(cap=float("nan")), 1, "softcap")
    refused(lib, call(scoring=1, cap=30.0), 1, "softmax scoring only")
    refused(lib, call(E=1025), 2, "E=1025")
    refused(lib, call(k=33), 2, "k=33")
    refused(lib, call(M=1 << 60, k=8), 2, "2^31")
    for name in ("g", "x", "ids", "out"):
        refused(lib, call(**{name: None}), 1, "null")
    assert call(M=0, g=None, x=None, ids=None, out=None) == 0


def t(*shape, dtype=torch.bfloat16):
    return torch.zeros(*shape, dtype=dtype)


I32, I64, F16, F32 = torch.int32, torch.int64, torch.float16, torch.float32


# The binding looks at shapes, types and layouts before the device, so CPU
# tensors reach every refusal; right ones are refused for the device alone.
@pytest.mark.parametrize("call,needle", [
    (lambda: moe.gather_tokens(t(8, 4).T, t(8, dtype=I32), 2), "contiguous 2-D"),
    (lambda: moe.gather_tokens(t(4), t(8, dtype=I32), 2), "contiguous 2-D"),
    (lambda: moe.gather_tokens(t(4, 8, dtype=F16), t(8, dtype=I32), 2), "dtype"),
    (lambda: moe.gather_tokens(t(4, 8), t(7, dtype=I32), 2), "scatter_indx"),
    (lambda: moe.gather_tokens(t(4, 8), t(0, dtype=I32), 0), "positive"),
    (lambda: moe.gather_tokens(t(4, 8), t(8, dtype=I64), 2), "scatter_indx"),
    (lambda: moe.gather_tokens(t(4, 8), t(8, dtype=I32), 1 << 40), "out of range"),
    (lambda: moe.gather_tokens(t(4, 8), t(8, dtype=I32), 2), "x must be a CUDA tensor"),
    (lambda: moe.gather_tokens_backward(t(7, 8), t(7, dtype=I32), 2), "grad_sorted"),
    (lambda: moe.gather_tokens_backward(t(8, 8), t(8, dtype=I32), 2), "CUDA"),
    (lambda: moe.combine_tokens(t(8, 8), t(8, dtype=I32), t(4, 2)), "topk_weights"),
    (lambda: moe.combine_tokens(t(8, 8), t(8, dtype=I32), t(8, dtype=F32)), "topk_weights"),
    (lambda: moe.combine_tokens(t(9, 8), t(8, dtype=I32), t(4, 2, dtype=F32)), "y must have"),
    (lambda: moe.combine_tokens(t(8, 8), t(8, dtype=I32), t(4, 2, dtype=F32), residual=t(4, 8, dtype=F32)), "residual"),
    (lambda: moe.combine_tokens(t(8, 8), t(8, dtype=I32), t(4, 2, dtype=F32), residual=t(8, 8)), "residual"),
    (lambda: moe.combine_tokens(t(8, 8), t(8, dtype=I32), t(4, 2, dtype=F32)), "CUDA"),
    (lambda: moe.combine_tokens_backward(t(4, 8), t(8, 8, dtype=F32), t(8, dtype=I32), t(4, 2, dtype=F32)),
     "y must be"),
    (lambda: moe.combine_tokens_backward(t(5, 8), t(8, 8), t(8, dtype=I32), t(4, 2, dtype=F32)), "grad_out must have"),
    (lambda: moe.combine_tokens_backward(t(4, 8), t(8, 8), t(8, dtype=I32), t(4, 2, dtype=F32)), "CUDA"),
    (lambda: moe.expert_matmul(t(4, 8, dtype=F32), t(2, 8, 8), t(3, dtype=I32)), "x must be bfloat16"),
    (lambda: moe.expert_matmul(t(4, 8), t(2, 8, 16), t(3, dtype=I32)), "columns"),
    (lambda: moe.expert_matmul(t(4, 8), t(2, 8, 8, dtype=F16), t(3, dtype=I32)), "weight must be"),
    (lambda: moe.expert_matmul(t(4, 8), t(2, 8, 8).transpose(1, 2), t(3, dtype=I32)), "weight must be"),
    (lambda: moe.expert_matmul(t(4, 8), t(2, 8, 8), t(4, dtype=I32)), "weight must be"),
    (lambda: moe.expert_matmul(t(4, 8), t(2, 8, 8), t(1, dtype=I32)), "expert_offsets"),
    (lambda: moe.expert_matmul(t(4, 8), t(2, 8, 8), t(3, dtype=I64)), "expert_offsets"),
    (lambda: moe.expert_matmul(t(4, 8), t(2, 8, 8), t(3, dtype=I32), activation="tanh"), "activation"),
    (lambda: moe.expert_matmul(t(4, 8), t(2, 9, 8), t(3, dtype=I32), gated=True), "odd"),
    (lambda: moe.expert_matmul(t(4, 8), t(2, 8, 8), t(3, dtype=I32), bias=t(2, 8)), "bias"),
    (lambda: moe.expert_matmul(t(4, 8), t(2, 16, 8), t(3, dtype=I32), residual=t(4, 8)), "residual"),
    (lambda: moe.expert_matmul(t(4, 8), t(2, 8, 8), t(3, dtype=I32)), "CUDA"),
    (lambda: moe.expert_matmul_grad_input(t(4, 8), t(2, 8, 8), t(3, dtype=I32), activation="silu"), "preact"),
    (lambda: moe.expert_matmul_grad_input(t(4, 8), t(2, 8, 8), t(3, dtype=I32), gated=True), "preact"),
    (lambda: moe.expert_matmul_grad_input(t(4, 8), t(2, 8, 8), t(3, dtype=I32), preact=t(4, 8), gated=True), "preact"),
    (lambda: moe.expert_matmul_grad_input(t(4, 8), t(2, 16, 8), t(3, dtype=I32)), "columns"),
    (lambda: moe.expert_matmul_grad_input(t(4, 8), t(2, 8, 8), t(3, dtype=I32)), "CUDA"),
    (lambda: moe.expert_matmul_grad_weight(t(4, 8), t(5, 8), t(3, dtype=I32)), "x must be"),
    (lambda: moe.expert_matmul_grad_weight(t(4, 8), t(4), t(3, dtype=I32)), "2-D"),
    (lambda: moe.expert_matmul_grad_weight(t(4, 8), t(4, 8), t(3, dtype=I32), dtype=F16), "dtype"),
    (lambda: moe.expert_matmul_grad_weight(t(4, 8), t(4, 8), t(3, dtype=I32), out=t(2, 8, 8, dtype=F16)), "dtype"),
    (lambda: moe.expert_matmul_grad_weight(t(4, 8), t(4, 8), t(3, dtype=I32)), "CUDA"),
    (lambda: moe.topk_backward(t(4, 2, dtype=F32), t(4, 8), t(4, 2, dtype=I32), "tanh", True), "scoring"),
    (lambda: moe.topk_backward(t(4, 3, dtype=F32), t(4, 8), t(4, 2, dtype=I32), "softmax", True), "grad_weights"),
    (lambda: moe.topk_backward(t(4, 2, dtype=F32), t(4, 8), t(4, 2, dtype=I64), "softmax", True), "topk_ids"),
    (lambda: moe.topk_backward(t(4, 2, dtype=F32), t(4, 8), t(8, dtype=I32), "softmax", True), "topk_ids"),
    (lambda: moe.topk_backward(t(4, 2, dtype=F32), t(4, 8), t(4, 2, dtype=I32), "softmax", True), "CUDA"),
])
def test_binding(call, needle):
    with pytest.raises(ValueError, match=needle):
        call()


def test_binding_wants_tensors_and_numbers():
    for call in (lambda: moe.gather_tokens([1], t(8, dtype=I32), 2), lambda: moe.gather_tokens(t(4, 8), None, 2),
                 lambda: moe.gather_tokens(t(4, 8), t(8, dtype=I32), "2"),
                 lambda: moe.topk_backward(t(4, 2, dtype=F32), t(4, 8), t(4, 2, dtype=I32), "softmax", True, "1")):
        with pytest.raises(TypeError):
            call()


def test_the_binding_calls_this_library():
    """Both bindings reach one copy of the library."""
    with open("/proc/self/maps") as f:
        paths = {line.split()[-1] for line in f if "libmoe_routing" in line}
    assert len(paths) == 1
