"""Losses that end a language model, on libpoetx's kernels: a projection onto
the vocabulary, z = x W^T, and a loss of each row's logits, which are formed
and used on the chip and never kept.

  cross_entropy_forward    loss = lse - z[target], lse = log sum_j exp(z_j)
  cross_entropy_backward   g_z = (g_loss + g_lse) exp(z - lse) - g_loss [j = target]
  distill_forward          from a teacher's logits at listed ids of each row, at
                           the temperature T: p = softmax(teacher / T),
                           lse = log sum_j exp(z_j / T),
                           loss = T^2 sum_k p_k (log p_k - z[id_k] / T + lse)
  distill_backward         g_z = g_loss T (exp(z / T - lse) - sum_k p_k [j = id_k])
  both backwards           g_x = g_z W,  g_W = g_z^T x

x [tokens, d] and W [vocab, d] are contiguous device tensors of one type
(float32 or bfloat16), of at least one row, d a multiple of 16 bytes, any
vocabulary. targets [tokens] and ids [tokens, top] are int64; losses, lse and
their gradients are float32 [tokens]: one weight a row, so that a mean or any
other reduction is the caller's (a mean over n rows: g_loss = 1 / n).

A row whose target is negative takes no part: its loss and lse are 0, and it
adds nothing to a gradient, whatever its x holds. Likewise an entry of a
teacher's list with a negative id or a logit of -inf, and a row without any
other. A row whose g_loss (and g_lse) is 0 adds nothing to a gradient, either.
A target or id past the vocabulary makes its row's loss, and the gradients,
NaN.

Outputs and workspaces come from torch's allocator on the stream that the call
runs on, so calls on different streams, and calls captured into different
graphs, share no memory.
"""
from __future__ import annotations

import functools

import torch

from . import poetx as P
from .dense import _ACT, _check, _here, _on, _workspace


def _sizes(x, W):
    """Checks x against W; tokens, d, vocab, the type's code and the device."""
    act = _ACT.get(x.dtype)
    if act is None:
        raise ValueError(f"x is {x.dtype}, expected float32 or bfloat16")
    if not x.is_cuda:
        raise ValueError("x must be on a GPU")
    if len(x.shape) != 2 or len(W.shape) != 2:
        raise ValueError("x and W must have two dimensions")
    (tokens, d), vocab = x.shape, W.shape[0]
    _check("W", W, (vocab, d), x.dtype, x.device)
    return tokens, d, vocab, act, x.device


def _teacher(ids, teacher, tokens, device):
    """Checks a teacher's list; its length a row and its type's code."""
    if len(ids.shape) != 2 or ids.shape[1] < 1:
        raise ValueError(f"ids has shape {tuple(ids.shape)}, expected (tokens, top)")
    top, kind = ids.shape[1], _ACT.get(teacher.dtype)
    if kind is None:
        raise ValueError(f"teacher is {teacher.dtype}, expected float32 or bfloat16")
    _check("ids", ids, (tokens, top), torch.int64, device)
    _check("teacher", teacher, (tokens, top), teacher.dtype, device)
    return top, kind


@functools.lru_cache(maxsize=4096)
def _plan(tokens, d, vocab, act, top, kind, temperature, forward):
    """The descriptor and its workspace bytes (forward: True, backward:
    False): both follow from the sizes alone."""
    desc = P.make_vocab_desc(tokens, d, vocab, act, top, kind, temperature)
    size = P.poetx_vocab_fwd_workspace_size if forward else P.poetx_vocab_bwd_workspace_size
    return desc, size(desc)


def _rows(like, shape):
    return like.new_empty(shape, dtype=torch.float32)


def _gradients(x, W, need_g_x, need_g_W):
    if not (need_g_x or need_g_W):
        raise ValueError("no gradient asked for")
    return x.new_empty(x.shape) if need_g_x else None, W.new_empty(W.shape) if need_g_W else None


def _run(device, stream, call, *args):
    if _here(device, stream):
        return call(*args)
    with _on(device, stream):
        return call(*args)


def cross_entropy_forward(x, W, targets, stream=None):
    """Returns (loss, lse), float32 [tokens]."""
    tokens, d, vocab, act, device = _sizes(x, W)
    _check("targets", targets, (tokens,), torch.int64, device)
    desc, nbytes = _plan(tokens, d, vocab, act, 0, 0, 1.0, True)

    def call():
        loss, lse = _rows(x, tokens), _rows(x, tokens)
        P.poetx_cross_entropy_fwd(desc, x, W, targets, loss, lse, _workspace(nbytes, device))
        return loss, lse
    return _run(device, stream, call)


def cross_entropy_backward(g_loss, x, W, targets, lse, g_lse=None, need_g_x=True, need_g_W=False,
                           stream=None):
    """Returns (g_x, g_W), None in the place of one not asked for, from the
    forward's lse and the gradients to loss and (a penalty on it, say) to lse."""
    tokens, d, vocab, act, device = _sizes(x, W)
    _check("targets", targets, (tokens,), torch.int64, device)
    for name, t in (("g_loss", g_loss), ("lse", lse), ("g_lse", g_lse)):
        if t is not None:
            _check(name, t, (tokens,), torch.float32, device)
    desc, nbytes = _plan(tokens, d, vocab, act, 0, 0, 1.0, False)

    def call():
        g_x, g_W = _gradients(x, W, need_g_x, need_g_W)
        P.poetx_cross_entropy_bwd(desc, g_loss, g_lse, x, W, targets, lse, g_x, g_W,
                                  _workspace(nbytes, device))
        return g_x, g_W
    return _run(device, stream, call)


def distill_forward(x, W, ids, teacher, temperature=1.0, stream=None):
    """Returns (loss, lse, z): loss and lse float32 [tokens], z float32
    [tokens, top], the student's logits at the ids, which the backward takes."""
    tokens, d, vocab, act, device = _sizes(x, W)
    top, kind = _teacher(ids, teacher, tokens, device)
    desc, nbytes = _plan(tokens, d, vocab, act, top, kind, float(temperature), True)

    def call():
        loss, lse, z = _rows(x, tokens), _rows(x, tokens), _rows(x, (tokens, top))
        P.poetx_distill_fwd(desc, x, W, ids, teacher, loss, lse, z, _workspace(nbytes, device))
        return loss, lse, z
    return _run(device, stream, call)


def distill_backward(g_loss, x, W, ids, teacher, lse, z, temperature=1.0, need_g_x=True,
                     need_g_W=False, stream=None):
    """Returns (g_x, g_W), None in the place of one not asked for, from the
    forward's lse and z. The teacher's logits have no gradient."""
    tokens, d, vocab, act, device = _sizes(x, W)
    top, kind = _teacher(ids, teacher, tokens, device)
    for name, t, shape in (("g_loss", g_loss, (tokens,)), ("lse", lse, (tokens,)),
                           ("z", z, (tokens, top))):
        _check(name, t, shape, torch.float32, device)
    desc, nbytes = _plan(tokens, d, vocab, act, top, kind, float(temperature), False)

    def call():
        g_x, g_W = _gradients(x, W, need_g_x, need_g_W)
        P.poetx_distill_bwd(desc, g_loss, x, W, ids, teacher, lse, z, g_x, g_W,
                            _workspace(nbytes, device))
        return g_x, g_W
    return _run(device, stream, call)
