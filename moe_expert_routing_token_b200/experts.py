"""Binding of the expert layer around the routing: tokens sorted by expert and
brought back, the experts' products, and the gradients down to the router's
logits.

One layer, forward and backward (``moe.`` stands for this package)::

    w, ids = moe.topk_softmax(logits, k, True)
    _, offsets, _, scatter, _ = moe.expert_permutation(ids, E)
    xs = moe.gather_tokens(x, scatter, k)
    h, z = moe.expert_matmul(xs, W1, offsets, activation="silu", gated=True, return_preact=True)
    y = moe.expert_matmul(h, W2, offsets)
    out = moe.combine_tokens(y, scatter, w, residual=x)

    dy, dw = moe.combine_tokens_backward(dout, y, scatter, w)
    dz = moe.expert_matmul_grad_input(dy, W2, offsets, preact=z, activation="silu", gated=True)
    dW2 = moe.expert_matmul_grad_weight(dy, h, offsets)
    dxs = moe.expert_matmul_grad_input(dz, W1, offsets)
    dW1 = moe.expert_matmul_grad_weight(dz, xs, offsets)
    dx = dout + moe.gather_tokens_backward(dxs, scatter, k)
    dlogits = moe.topk_backward(dw, logits, ids, "softmax", True)

Each function checks its tensors, allocates what ``out`` arguments do not
give, and calls the C entry point on the operands' device and current stream.
Rows behind the last expert's segment are not written: freshly allocated
outputs hold anything there.  Outputs must not overlap inputs.  A tensor that
was made on another stream is the caller's to order and, where it is freed
early, to ``record_stream``.
"""
from __future__ import annotations

import torch

from .routing import (MOE_ACT_GELU, MOE_ACT_NONE, MOE_ACT_SILU, MOE_OK, MOE_SCORE_SIGMOID, MOE_SCORE_SOFTMAX, _check,
                      _cuda_2d, _dtype_code, _on, lib)

ACTIVATIONS = {"none": MOE_ACT_NONE, "silu": MOE_ACT_SILU, "gelu": MOE_ACT_GELU}
SCORINGS = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}


def _activation(name: str) -> int:
    code = ACTIVATIONS.get(name)
    if code is None:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, not {name!r}")
    return code


def _call(name: str, index: int, *args) -> None:
    """The C entry point ``name`` on the current stream of device ``index``.

    A small call's time is the host's: the raw handle is
    torch.cuda.current_stream(index).cuda_stream without the Python object
    around it, the device is switched only where it has to be, and devices are
    compared by number."""
    fn = getattr(lib(), name)
    if torch._C._cuda_getDevice() == index:
        st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with _on(torch.device("cuda", index)):
            st = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if st != MOE_OK:
        _check(st, name)


def _like(t, name: str, like: torch.Tensor, shape, dtype) -> torch.Tensor:
    """The given tensor, checked, or a new one on ``like``'s device."""
    if t is None:
        return like.new_empty(shape) if dtype is like.dtype else like.new_empty(shape, dtype=dtype)
    _expect(t, name, shape, dtype, like.get_device())
    return t


def _expect(t: torch.Tensor, name: str, shape, dtype, index: int) -> None:
    if not (t.shape == shape and t.dtype is dtype and t.get_device() == index and t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {tuple(shape)} {dtype} tensor on cuda:{index}")


def _rows(t: torch.Tensor, name: str) -> int:
    """A contiguous 2-D CUDA tensor's device number."""
    index = t.get_device()
    if index < 0 or t.dim() != 2 or not t.is_contiguous():
        _cuda_2d(t, name)
    return index


def _scatter(scatter_indx: torch.Tensor, pairs: int, index: int) -> None:
    if not (scatter_indx.dtype is torch.int32 and scatter_indx.numel() == pairs and scatter_indx.is_contiguous()
            and scatter_indx.get_device() == index):
        raise ValueError(f"scatter_indx must be a contiguous int32 tensor of {pairs} places on cuda:{index}")


def _tokens_of(rows: torch.Tensor, k: int, name: str) -> int:
    if k < 1 or rows.shape[0] % k:
        raise ValueError(f"{name} must have a row for each of the tokens' {k} slots")
    return rows.shape[0] // k


def gather_tokens(x: torch.Tensor, scatter_indx: torch.Tensor, topk: int, out=None) -> torch.Tensor:
    """Token rows (M, H) to their places in expert order: (M * topk, H), by the
    scatter indices of ``expert_permutation`` (moe_gather_tokens)."""
    dev = _rows(x, "x")
    M, H = x.shape
    topk = int(topk)
    code = _dtype_code(x)
    if topk < 1:
        raise ValueError("topk must be positive")
    _scatter(scatter_indx, M * topk, dev)
    out = _like(out, "out", x, (M * topk, H), x.dtype)
    _call("moe_gather_tokens", dev, x.data_ptr(), code, M, H, scatter_indx.data_ptr(), topk, out.data_ptr())
    return out


def gather_tokens_backward(grad_sorted: torch.Tensor, scatter_indx: torch.Tensor, topk: int, out=None) -> torch.Tensor:
    """Gradient of ``gather_tokens``: (M * topk, H) to (M, H), each token the
    sum of its places' rows (moe_gather_tokens_backward)."""
    dev = _rows(grad_sorted, "grad_sorted")
    H, topk = grad_sorted.shape[1], int(topk)
    code = _dtype_code(grad_sorted)
    M = _tokens_of(grad_sorted, topk, "grad_sorted")
    _scatter(scatter_indx, M * topk, dev)
    out = _like(out, "out", grad_sorted, (M, H), grad_sorted.dtype)
    _call("moe_gather_tokens_backward", dev, grad_sorted.data_ptr(), code, M, H, scatter_indx.data_ptr(), topk,
          out.data_ptr())
    return out


def combine_tokens(y: torch.Tensor, scatter_indx: torch.Tensor, topk_weights: torch.Tensor, residual=None,
                   out=None) -> torch.Tensor:
    """The experts' rows (M * k, H) back to their tokens, weighted and summed,
    plus ``residual`` (M, H): (M, H) of y's dtype (moe_combine_tokens)."""
    dev = _rows(y, "y")
    _rows(topk_weights, "topk_weights")
    M, k = topk_weights.shape
    H = y.shape[1]
    code = _dtype_code(y)
    _expect(topk_weights, "topk_weights", (M, k), torch.float32, dev)
    if y.shape[0] != M * k:
        raise ValueError(f"y must have a row for each of the {M * k} places")
    _scatter(scatter_indx, M * k, dev)
    if residual is not None:
        _expect(residual, "residual", (M, H), y.dtype, dev)
    out = _like(out, "out", y, (M, H), y.dtype)
    _call("moe_combine_tokens", dev, y.data_ptr(), code, M, H, scatter_indx.data_ptr(), k, topk_weights.data_ptr(),
          None if residual is None else residual.data_ptr(), out.data_ptr())
    return out


def combine_tokens_backward(grad_out: torch.Tensor, y: torch.Tensor, scatter_indx: torch.Tensor,
                            topk_weights: torch.Tensor, grad_y=None, grad_weights=None):
    """Gradients of ``combine_tokens`` with respect to y and topk_weights:
    (grad_y (M * k, H), grad_weights fp32 (M, k)); the residual's is grad_out
    itself (moe_combine_tokens_backward)."""
    dev = _rows(grad_out, "grad_out")
    _rows(topk_weights, "topk_weights")
    M, k = topk_weights.shape
    H = grad_out.shape[1]
    code = _dtype_code(grad_out)
    if grad_out.shape[0] != M:
        raise ValueError(f"grad_out must have a row for each of the {M} tokens")
    _expect(topk_weights, "topk_weights", (M, k), torch.float32, dev)
    _expect(y, "y", (M * k, H), grad_out.dtype, dev)
    _scatter(scatter_indx, M * k, dev)
    grad_y = _like(grad_y, "grad_y", y, (M * k, H), y.dtype)
    grad_weights = _like(grad_weights, "grad_weights", topk_weights, (M, k), torch.float32)
    _call("moe_combine_tokens_backward", dev, grad_out.data_ptr(), y.data_ptr(), code, M, H, scatter_indx.data_ptr(),
          k, topk_weights.data_ptr(), grad_y.data_ptr(), grad_weights.data_ptr())
    return grad_y, grad_weights


def _experts(rows: torch.Tensor, name: str, expert_offsets: torch.Tensor):
    """Checks of a sorted row array and the offsets; the device's number and
    the number of experts."""
    index = _rows(rows, name)
    if rows.dtype is not torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16")
    if not (expert_offsets.dtype is torch.int32 and expert_offsets.dim() == 1 and expert_offsets.numel() >= 2
            and expert_offsets.is_contiguous() and expert_offsets.get_device() == index):
        raise ValueError(f"expert_offsets must be a contiguous int32 tensor of E + 1 values on cuda:{index}")
    return index, expert_offsets.numel() - 1


def _weight(weight: torch.Tensor, E: int, index: int):
    """(N, K) of a weight."""
    if not (weight.dtype is torch.bfloat16 and weight.dim() == 3 and weight.is_contiguous()
            and weight.get_device() == index and weight.shape[0] == E):
        raise ValueError(f"weight must be a contiguous bfloat16 tensor (E = {E}, N, K) on cuda:{index}")
    return weight.shape[1:]


def expert_matmul(x: torch.Tensor, weight: torch.Tensor, expert_offsets: torch.Tensor, bias=None,
                  activation: str = "none", gated: bool = False, residual=None, return_preact: bool = False,
                  out=None, preact_out=None):
    """Rows (P, K) in expert order times their expert's weight (E, N, K), with
    bias fp32 (E, N), activation ("none", "silu", "gelu") and residual (P, N)
    in the same pass (moe_expert_matmul).  ``gated``: the weight is
    (E, 2 N, K) and the result f(first half) * second half.  Returns out
    (P, N) or, with ``return_preact`` or ``preact_out``, (out, preact): the
    activation's input, for the backward pass.  A plain matrix product is
    E = 1 with offsets [0, P]."""
    dev, E = _experts(x, "x", expert_offsets)
    act, gated = _activation(activation), bool(gated)
    P, K = x.shape
    Nz, Kw = _weight(weight, E, dev)
    if Kw != K or (gated and Nz % 2):
        raise ValueError("weight does not match x's columns, or a gated weight has an odd number of rows")
    N = Nz // 2 if gated else Nz
    if bias is not None:
        _expect(bias, "bias", (E, Nz), torch.float32, dev)
    if residual is not None:
        _expect(residual, "residual", (P, N), torch.bfloat16, dev)
    out = _like(out, "out", x, (P, N), torch.bfloat16)
    kept = return_preact or preact_out is not None
    if kept:
        preact_out = _like(preact_out, "preact_out", x, (P, Nz), torch.bfloat16)
    _call("moe_expert_matmul", dev, x.data_ptr(), weight.data_ptr(), expert_offsets.data_ptr(), P, K, N, E,
          None if bias is None else bias.data_ptr(), act, int(gated),
          None if residual is None else residual.data_ptr(), out.data_ptr(), preact_out.data_ptr() if kept else None)
    return (out, preact_out) if kept else out


def expert_matmul_grad_input(grad_out: torch.Tensor, weight: torch.Tensor, expert_offsets: torch.Tensor, preact=None,
                             activation: str = "none", gated: bool = False, out=None) -> torch.Tensor:
    """Gradient of ``expert_matmul`` (without activation) with respect to its
    rows: grad_out (P, N) times weight (E, N, K), taken on through the
    activation that made those rows if ``preact``, (P, K) or gated (P, 2 K), is
    given: the result then has preact's shape (moe_expert_matmul_grad_input)."""
    dev, E = _experts(grad_out, "grad_out", expert_offsets)
    act, gated = _activation(activation), bool(gated)
    P, N = grad_out.shape
    Nw, K = _weight(weight, E, dev)
    if Nw != N:
        raise ValueError("weight does not match grad_out's columns")
    shape = (P, 2 * K if gated else K)
    if preact is not None:
        _expect(preact, "preact", shape, torch.bfloat16, dev)
    elif act != MOE_ACT_NONE or gated:
        raise ValueError("an activation's gradient needs its preact")
    out = _like(out, "out", grad_out, shape, torch.bfloat16)
    _call("moe_expert_matmul_grad_input", dev, grad_out.data_ptr(), weight.data_ptr(), expert_offsets.data_ptr(), P,
          K, N, E, None if preact is None else preact.data_ptr(), act, int(gated), out.data_ptr())
    return out


def expert_matmul_grad_weight(grad_out: torch.Tensor, x: torch.Tensor, expert_offsets: torch.Tensor,
                              bias_grad: bool = False, dtype: torch.dtype = torch.bfloat16, out=None):
    """Gradient of ``expert_matmul`` (without activation) with respect to its
    weight: (E, N, K) of ``dtype`` (bfloat16 or float32) from grad_out (P, N)
    and x (P, K); with ``bias_grad`` also the bias's, fp32 (E, N).  Experts
    without rows get zeros (moe_expert_matmul_grad_weight)."""
    dev, E = _experts(grad_out, "grad_out", expert_offsets)
    P, N = grad_out.shape
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    K = x.shape[1]
    _expect(x, "x", (P, K), torch.bfloat16, dev)
    out = _like(out, "out", x, (E, N, K), dtype if out is None else out.dtype)
    code = _dtype_code(out)
    db = x.new_empty((E, N), dtype=torch.float32) if bias_grad else None
    _call("moe_expert_matmul_grad_weight", dev, grad_out.data_ptr(), x.data_ptr(), expert_offsets.data_ptr(), P, K, N,
          E, code, out.data_ptr(), None if db is None else db.data_ptr())
    return (out, db) if bias_grad else out


def topk_backward(grad_weights: torch.Tensor, gating_output: torch.Tensor, topk_ids: torch.Tensor, scoring: str,
                  renormalize: bool, routed_scaling_factor: float = 1.0, softcap: float = 0.0,
                  out=None) -> torch.Tensor:
    """Gradient of a routing call's weights with respect to its logits, the
    choice of experts held fixed: (M, E) of the logits' dtype
    (moe_topk_backward).  ``scoring``: "softmax" (``topk_softmax``,
    ``grouped_topk``) or "sigmoid" (``biased_grouped_topk``, fused routers);
    the other arguments as in the routing call."""
    dev = _rows(gating_output, "gating_output")
    M, E = gating_output.shape
    code = _dtype_code(gating_output)
    if scoring not in SCORINGS:
        raise ValueError(f"scoring must be one of {sorted(SCORINGS)}, not {scoring!r}")
    if topk_ids.dim() != 2:
        raise ValueError("topk_ids must be 2-D")
    k = topk_ids.shape[1]
    _expect(topk_ids, "topk_ids", (M, k), torch.int32, dev)
    _expect(grad_weights, "grad_weights", (M, k), torch.float32, dev)
    out = _like(out, "out", gating_output, (M, E), gating_output.dtype)
    _call("moe_topk_backward", dev, grad_weights.data_ptr(), gating_output.data_ptr(), code, topk_ids.data_ptr(), M,
          E, k, SCORINGS[scoring], int(bool(renormalize)), float(routed_scaling_factor), float(softcap),
          out.data_ptr())
    return out
