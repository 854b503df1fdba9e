"""Global gradient norm over many tensors, and clipping by it, on libpoetx's
kernels: what a training step does with the generator gradients of every
layer (PoetxLinear.backward) and the bias and weight gradients beside them.

Gradients are contiguous float32 or bfloat16 tensors of any sizes on one GPU,
the two types mixed freely; lists of views of one flat buffer, in order, are
taken as one range.
"""
from __future__ import annotations

import torch

from . import poetx as P
from .dense import _here, _on


def _device_of(grads, outs, norm):
    """The one GPU that all of them are on (the current one if there are none)."""
    tensors = [*grads, *(outs or ()), *(() if norm is None else (norm,))]
    if not tensors:
        return torch.device("cuda", torch.cuda.current_device())
    found = set(map(torch.Tensor.get_device, tensors))
    if len(found) != 1 or -1 in found:
        raise ValueError("gradients, outputs and norm must be on one GPU")
    return tensors[0].device


def grad_norm(grads, stream=None):
    """sqrt of the sum of squares of every value of every tensor: a float32
    scalar tensor on their device."""
    grads = list(grads)
    device = _device_of(grads, None, None)
    tensors = P.make_grad_list(grads)
    if _here(device, stream):
        return _measure(tensors, len(grads), device, None)
    with _on(device, stream):
        return _measure(tensors, len(grads), device, None)


def _measure(tensors, count, device, max_norm):
    """The norm of a list of records, which are clipped with a max_norm."""
    norm = torch.empty((), device=device, dtype=torch.float32)
    ws = torch.empty(P.poetx_grad_workspace_size(count), device=device, dtype=torch.uint8)
    if max_norm is None:
        P.poetx_grad_norm(tensors, norm, ws)
    else:
        P.poetx_grad_clip(tensors, max_norm, norm, ws)
    return norm


def clip_grads(grads, max_norm, outs=None, norm=None, stream=None):
    """grad min(1, max_norm / norm) for every tensor, in place or into `outs`,
    and returns the norm before clipping (a float32 scalar tensor). A norm
    that is not finite leaves the values as they are. norm: a float32 scalar
    tensor to clip by, where the caller has the norm already (joined over the
    ranks of a sharded job, say)."""
    grads = list(grads)
    if outs is not None:
        outs = list(outs)
        if len(outs) != len(grads):
            raise ValueError("one output per gradient")
    device = _device_of(grads, outs, norm)
    if norm is not None and (norm.numel() != 1 or norm.dtype != torch.float32):
        raise ValueError("norm must be one float32 value")
    tensors = P.make_grad_list(grads, outs)
    if norm is None and _here(device, stream):
        return _measure(tensors, len(grads), device, max_norm)
    with _on(device, stream):
        if norm is None:
            return _measure(tensors, len(grads), device, max_norm)
        P.poetx_grad_scale(tensors, max_norm, norm)
    return norm
