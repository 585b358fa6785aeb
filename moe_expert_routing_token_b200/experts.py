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
give, and calls the C entry point on the operands' device and current stream
(csrc/binding.cpp: through ctypes, a decode-sized call would spend three times
its kernel's time on that).  Rows behind the last expert's segment are not
written: freshly allocated outputs hold anything there.  Outputs must not
overlap inputs.  The functions record nothing for autograd: the backward calls
are made by name, as above.  A tensor that was made on another stream is the caller's to
order and, where it is freed early, to ``record_stream``.
"""
from __future__ import annotations

import importlib.machinery
import importlib.util
import os

import torch

from .routing import (LIB_PATH, MOE_ACT_GELU, MOE_ACT_NONE, MOE_ACT_SILU, MOE_SCORE_SIGMOID, MOE_SCORE_SOFTMAX, lib)

ACTIVATIONS = {"none": MOE_ACT_NONE, "silu": MOE_ACT_SILU, "gelu": MOE_ACT_GELU}
SCORINGS = {"softmax": MOE_SCORE_SOFTMAX, "sigmoid": MOE_SCORE_SIGMOID}
BINDING_PATH = os.path.join(os.path.dirname(LIB_PATH), "_experts.so")


class _Unloaded:
    """Loads the native binding at the first use (the package can be imported
    before it is built)."""

    def __getattr__(self, name):
        global _native
        if not os.path.exists(BINDING_PATH):
            raise RuntimeError(f"_experts.so not found at {BINDING_PATH}; build it with "
                               "`python -m moe_expert_routing_token_b200.build`")
        lib()
        loader = importlib.machinery.ExtensionFileLoader("_experts", BINDING_PATH)
        module = importlib.util.module_from_spec(importlib.util.spec_from_loader("_experts", loader))
        loader.exec_module(module)
        _native = module
        return getattr(module, name)


_native = _Unloaded()


def _named(table: dict, name: str, what: str) -> int:
    code = table.get(name)
    if code is None:
        raise ValueError(f"{what} must be one of {sorted(table)}, not {name!r}")
    return code


def gather_tokens(x: torch.Tensor, scatter_indx: torch.Tensor, topk: int, out=None) -> torch.Tensor:
    """Token rows (M, H) to their places in expert order: (M * topk, H), by the
    scatter indices of ``expert_permutation`` (moe_gather_tokens)."""
    return _native.gather_tokens(x, scatter_indx, topk, out)


def gather_tokens_backward(grad_sorted: torch.Tensor, scatter_indx: torch.Tensor, topk: int, out=None) -> torch.Tensor:
    """Gradient of ``gather_tokens``: (M * topk, H) to (M, H), each token the
    sum of its places' rows (moe_gather_tokens_backward)."""
    return _native.gather_tokens_backward(grad_sorted, scatter_indx, topk, out)


def combine_tokens(y: torch.Tensor, scatter_indx: torch.Tensor, topk_weights: torch.Tensor, residual=None,
                   out=None) -> torch.Tensor:
    """The experts' rows (M * k, H) back to their tokens, weighted and summed,
    plus ``residual`` (M, H): (M, H) of y's dtype (moe_combine_tokens)."""
    return _native.combine_tokens(y, scatter_indx, topk_weights, residual, out)


def combine_tokens_backward(grad_out: torch.Tensor, y: torch.Tensor, scatter_indx: torch.Tensor,
                            topk_weights: torch.Tensor, grad_y=None, grad_weights=None):
    """Gradients of ``combine_tokens`` with respect to y and topk_weights:
    (grad_y (M * k, H), grad_weights fp32 (M, k)); the residual's is grad_out
    itself (moe_combine_tokens_backward)."""
    return _native.combine_tokens_backward(grad_out, y, scatter_indx, topk_weights, grad_y, grad_weights)


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
    return _native.expert_matmul(x, weight, expert_offsets, bias, _named(ACTIVATIONS, activation, "activation"), gated,
                                 residual, return_preact, out, preact_out)


def expert_matmul_grad_input(grad_out: torch.Tensor, weight: torch.Tensor, expert_offsets: torch.Tensor, preact=None,
                             activation: str = "none", gated: bool = False, out=None) -> torch.Tensor:
    """Gradient of ``expert_matmul`` (without activation) with respect to its
    rows: grad_out (P, N) times weight (E, N, K), taken on through the
    activation that made those rows if ``preact``, (P, K) or gated (P, 2 K), is
    given: the result then has preact's shape (moe_expert_matmul_grad_input)."""
    return _native.expert_matmul_grad_input(grad_out, weight, expert_offsets, preact,
                                            _named(ACTIVATIONS, activation, "activation"), gated, out)


def expert_matmul_grad_weight(grad_out: torch.Tensor, x: torch.Tensor, expert_offsets: torch.Tensor,
                              bias_grad: bool = False, dtype: torch.dtype = torch.bfloat16, out=None):
    """Gradient of ``expert_matmul`` (without activation) with respect to its
    weight: (E, N, K) of ``dtype`` (bfloat16 or float32) from grad_out (P, N)
    and x (P, K); with ``bias_grad`` also the bias's, fp32 (E, N).  Experts
    without rows get zeros (moe_expert_matmul_grad_weight)."""
    if dtype not in (torch.bfloat16, torch.float32):
        raise ValueError(f"unsupported dtype {dtype}; expected float32 or bfloat16")
    return _native.expert_matmul_grad_weight(grad_out, x, expert_offsets, bias_grad, dtype == torch.float32, out)


def topk_backward(grad_weights: torch.Tensor, gating_output: torch.Tensor, topk_ids: torch.Tensor, scoring: str,
                  renormalize: bool, routed_scaling_factor: float = 1.0, softcap: float = 0.0,
                  out=None) -> torch.Tensor:
    """Gradient of a routing call's weights with respect to its logits, the
    choice of experts held fixed: (M, E) of the logits' dtype
    (moe_topk_backward).  ``scoring``: "softmax" for ``topk_softmax``,
    ``grouped_topk`` and ``fused_router_top1``, "sigmoid" for
    ``biased_grouped_topk`` and ``fused_router_topk``; the other arguments as
    in the routing call (``fused_router_top1``: ``renormalize`` False and its
    ``softcap``; the fused routers' logits: ``return_logits``).

    ``topk_ids`` are the ids that the routing call wrote.  Where
    ``fill_shared_expert_slot`` has overwritten the last slot (in place: keep
    the ids from before), the weights' gradient dw goes back through the fill
    first::

        routed = ids.clone()
        moe.fill_shared_expert_slot(w, ids, E, num_shared, pick, factor)
        # ... the layer, forward and backward, with w and ids: dw
        if factor is not None:
            dw[:, :-1] += dw[:, -1:] / factor
            dw[:, -1] = 0
        dlogits = moe.topk_backward(dw, logits, routed, scoring, renormalize, rsf)
    """
    return _native.topk_backward(grad_weights, gating_output, topk_ids, _named(SCORINGS, scoring, "scoring"),
                                 renormalize, routed_scaling_factor, softcap, out)
