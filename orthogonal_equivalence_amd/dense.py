"""The dense linear with bias, activation and residual in its epilogue, on
libpoetx's kernels: the layer that carries no R and P (a POET-X weight merged
after training, or a weight that was never reparameterised).

    u = x W^T + bias,   y = act(u) + residual

dense_forward and dense_backward take contiguous device tensors x [tokens,
d_in], W [d_out, d_in], residual and u [tokens, d_out] of one type (float32 or
bfloat16) and a float32 bias [d_out], of at least one row, widths that are
multiples of 16 bytes and 16-byte aligned; W may be the int8 codes of
poetx_quantize_weight with their float32 row scales w_scale [d_out].
DenseLinear keeps a weight and its bias. Outputs and workspaces come from
torch's allocator on the stream that the call runs on, so calls on different
streams, and calls captured into different graphs, share no memory.
"""
from __future__ import annotations

import contextlib
import functools

import torch

from . import poetx as P

ACTIVATIONS = {"none": P.POETX_ACT_NONE, "relu": P.POETX_ACT_RELU, "gelu": P.POETX_ACT_GELU,
               "gelu_tanh": P.POETX_ACT_GELU_TANH, "silu": P.POETX_ACT_SILU}
_ACT = {torch.float32: P.POETX_F32, torch.bfloat16: P.POETX_BF16}


@contextlib.contextmanager
def _on(device, stream):
    """The tensors' device, and `stream` (a torch stream, or a hipStream_t
    address) as the current one."""
    if isinstance(stream, int):
        stream = (torch.cuda.ExternalStream(stream, device=device) if stream else
                  torch.cuda.default_stream(device))
    if stream is not None and stream.device != device:
        raise ValueError(f"stream of {stream.device} for tensors on {device}")
    with torch.cuda.device(device), torch.cuda.stream(stream):
        yield


def _check(name, t, shape, dtype, device):
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    if t.dtype != dtype:
        raise ValueError(f"{name} is {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _desc(name, t, W, activation, w_scale, width):
    """Checks the weight against the activations t (their columns are W's
    dimension `width`); the descriptor, the workspace bytes and t's device."""
    code, act = ACTIVATIONS.get(activation), _ACT.get(t.dtype)
    if code is None:
        raise ValueError(f"unknown activation {activation!r}")
    if act is None:
        raise ValueError(f"{name} is {t.dtype}, expected float32 or bfloat16")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a GPU")
    shape, w_shape, device = t.shape, W.shape, t.device
    if len(shape) != 2 or len(w_shape) != 2:
        raise ValueError(f"{name} and W must have two dimensions")
    tokens, (d_out, d_in) = shape[0], w_shape
    if shape[1] != w_shape[width]:
        raise ValueError(f"{name} has {shape[1]} columns, W is {tuple(w_shape)}")
    _check("W", W, w_shape, t.dtype if w_scale is None else torch.int8, device)
    if w_scale is None:
        desc, ws = _plan(tokens, d_in, d_out, act, code, False, width)
    else:
        _check("w_scale", w_scale, (d_out,), torch.float32, device)
        desc, ws = _plan(tokens, d_in, d_out, act, code, True, width)
        desc = P.make_dense_desc(tokens, d_in, d_out, act, code, w_scale)
    return desc, ws, device


@functools.lru_cache(maxsize=4096)
def _plan(tokens, d_in, d_out, act, activation, int8, forward):
    """The descriptor of these sizes (its w_scale, with int8, a placeholder)
    and its workspace bytes (forward: 1, backward: 0): both follow from the
    sizes alone."""
    desc = P.make_dense_desc(tokens, d_in, d_out, act, activation, 16 if int8 else None)
    size = P.poetx_dense_fwd_workspace_size if forward else P.poetx_dense_bwd_workspace_size
    return desc, size(desc)


def _workspace(nbytes, device):
    return torch.empty(nbytes, device=device, dtype=torch.uint8) if nbytes else None


def _here(device, stream):
    """Whether the call runs on the current device's current stream as it is."""
    return stream is None and device.index == torch.cuda.current_device()


def dense_forward(x, W, bias=None, residual=None, activation="none", w_scale=None, save_u=False,
                  stream=None):
    """Returns (y, u): u, the pre-activation that dense_backward takes, with
    save_u, else None."""
    desc, nbytes, device = _desc("x", x, W, activation, w_scale, 1)
    out = (desc.tokens, desc.d_out)
    if bias is not None:
        _check("bias", bias, out[1:], torch.float32, device)
    if residual is not None:
        _check("residual", residual, out, x.dtype, device)
    if _here(device, stream):
        return _forward(desc, x, W, bias, residual, out, save_u, nbytes)
    with _on(device, stream):
        return _forward(desc, x, W, bias, residual, out, save_u, nbytes)


def _forward(desc, x, W, bias, residual, out, save_u, nbytes):
    y = x.new_empty(out)
    u = x.new_empty(out) if save_u else None
    P.poetx_dense_fwd(desc, x, W, bias, residual, y, u, _workspace(nbytes, x.device))
    return y, u


def dense_backward(g_y, W, x=None, u=None, activation="none", w_scale=None, need_g_x=True,
                   need_g_W=False, need_g_bias=False, stream=None):
    """Returns (g_x, g_W, g_bias), None in the place of one not asked for. x is
    needed for g_W, u (dense_forward's, with save_u) for an activation. The
    gradient of the residual is g_y itself. int8 codes have no g_W."""
    desc, nbytes, device = _desc("g_y", g_y, W, activation, w_scale, 0)
    if x is not None:
        _check("x", x, (desc.tokens, desc.d_in), g_y.dtype, device)
    if u is not None:
        _check("u", u, g_y.shape, g_y.dtype, device)
    if need_g_W and x is None:
        raise ValueError("g_W needs x")
    if need_g_W and w_scale is not None:
        raise ValueError("int8 codes have no gradient")
    if activation != "none" and u is None:
        raise ValueError("the backward of an activation needs u")
    if not (need_g_x or need_g_W or need_g_bias):
        raise ValueError("no gradient asked for")
    if _here(device, stream):
        return _backward(desc, g_y, W, x, u, need_g_x, need_g_W, need_g_bias, nbytes)
    with _on(device, stream):
        return _backward(desc, g_y, W, x, u, need_g_x, need_g_W, need_g_bias, nbytes)


def _backward(desc, g_y, W, x, u, need_g_x, need_g_W, need_g_bias, nbytes):
    g_x = g_y.new_empty((desc.tokens, desc.d_in)) if need_g_x else None
    g_W = g_y.new_empty((desc.d_out, desc.d_in)) if need_g_W else None
    g_b = g_y.new_empty(desc.d_out, dtype=torch.float32) if need_g_bias else None
    P.poetx_dense_bwd(desc, g_y, x, W, u, g_x, g_W, g_b, _workspace(nbytes, g_y.device))
    return g_x, g_W, g_b


class DenseLinear:
    """y = act(x W^T + bias) + residual with W [d_out, d_in] kept on the device
    in the activation type `act` ("f32", "bf16"), or with int8=True as INT8
    codes with per-row scales (poetx_quantize_weight), formed from W as it is
    given, float32 or the activation type."""

    def __init__(self, W: torch.Tensor, act: str, bias=None, activation="none", device="cuda",
                 int8: bool = False):
        if activation not in ACTIVATIONS:
            raise ValueError(f"unknown activation {activation!r}")
        self.torch_dtype = {"f32": torch.float32, "bf16": torch.bfloat16}[act]
        self.device = torch.device(device)
        self.activation = activation
        kept = torch.float32 if int8 and W.dtype != self.torch_dtype else self.torch_dtype
        self.W = W.to(self.device, kept).contiguous()
        self.d_out, self.d_in = self.W.shape
        self.bias = None
        if bias is not None:
            self.bias = torch.as_tensor(bias).to(self.device, torch.float32).contiguous()
        self.w_scale = None
        if int8:
            with torch.cuda.device(self.W.device):
                q = torch.empty(self.W.shape, device=self.device, dtype=torch.int8)
                self.w_scale = torch.empty(self.d_out, device=self.device, dtype=torch.float32)
                P.poetx_quantize_weight(self.W, self.d_out, self.d_in, _ACT[kept], q, self.w_scale)
            self.W = q

    def forward(self, x, residual=None, save_u=False, stream=None):
        return dense_forward(x, self.W, self.bias, residual, self.activation, self.w_scale, save_u,
                             stream)

    def backward(self, g_y, x=None, u=None, need_g_x=True, need_g_W=False, need_g_bias=None,
                 stream=None):
        """(g_x, g_W, g_bias); g_bias by default where the layer has a bias."""
        if need_g_bias is None:
            need_g_bias = self.bias is not None
        return dense_backward(g_y, self.W, x, u, self.activation, self.w_scale, need_g_x, need_g_W,
                              need_g_bias, stream)
