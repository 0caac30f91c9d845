"""Queries and keys normed per head and rotated by position in one pass, with its backward.

    q, k = qk_norm_rope(q, k, gamma_q, gamma_k, inv_freq, positions)

``q`` [B, T, Hq, D] and ``k`` [B, T, Hk, D] (or [T, H, D] both) may be views of a packed projection
or of a [B, H, T, D] array: any strides of the first dimensions that are multiples of 16 bytes, the
last dimension dense.  The write-ups' model norms queries and keys per head and rotates them
(QK-norm, RoPE, 24 query heads over 8 key heads); include/flce_train.h states the formulas.
"""
from __future__ import annotations

import contextlib

import torch
from torch.autograd.function import once_differentiable

from . import _abi

_DTYPES = {torch.float32: _abi.DTYPE_F32, torch.bfloat16: _abi.DTYPE_BF16}


def on_stream(stream, device):
    """A context in which the device's current stream is the caller's: launches, outputs and
    workspaces go to it.  None leaves the current one."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    if stream.device != device:
        raise ValueError(f"stream is on {stream.device}, the tensors on {device}")
    return torch.cuda.stream(stream)


def _rows(t, name, like=None):
    """The shape [B, T, H, D] of a tensor of rows; checks type, device, rank and the dense last
    dimension."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in _DTYPES:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    shape, strides = tuple(t.shape), t.stride()
    n = len(shape)
    if n != 4 and n != 3:
        raise ValueError(f"{name} must be [T, H, D] or [B, T, H, D], got {shape}")
    if like is not None:
        if t.device != like.device:
            raise ValueError(f"{name} must be on {like.device}")
        if t.dtype != like.dtype:
            raise TypeError(f"{name} must be {like.dtype}, got {t.dtype}")
        if n != len(like.shape):
            raise ValueError(f"{name} must have as many dimensions as q")
    if strides[-1] != 1 and shape[-1] > 1:
        raise ValueError(f"the last dimension of {name} must be dense")
    return shape if n == 4 else (1, *shape)


def _say_inputs(q, k, gamma_q, gamma_k, inv_freq, positions, eps, interleaved):
    """Raises what is wrong with the inputs."""
    (B, T, Hq, D), dev = _rows(q, "q"), q.device
    if k is not None:
        kB, kT, _, kD = _rows(k, "k", q)
        if kB != B or kT != T or kD != D:
            raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)} differ in more than "
                             "their heads")
    elif gamma_k is not None:
        raise ValueError("gamma_k given without k")
    gamma_dtype = None
    for name, g in (("gamma_q", gamma_q), ("gamma_k", gamma_k)):
        if g is None:
            continue
        if g.dtype not in _DTYPES or (gamma_dtype is not None and g.dtype != gamma_dtype):
            raise TypeError(f"{name}: gamma_q and gamma_k must both be float32 or bfloat16")
        gamma_dtype = g.dtype
        _abi._check_buffer(g, name, gamma_dtype, (D,), dev)
    if inv_freq is not None:
        _abi._check_buffer(inv_freq, "inv_freq", torch.float32, (inv_freq.numel(),), dev)
    if positions is not None:
        shape = tuple(positions.shape)
        if not positions.is_cuda or positions.device != dev:
            raise ValueError(f"positions must be a CUDA tensor on {dev}")
        if positions.dtype != torch.int64:
            raise TypeError(f"positions must be int64, got {positions.dtype}")
        if shape != (B, T) and shape != (T,):
            raise ValueError(f"positions must be [T] or [B, T], got {shape}")
        if T > 1 and positions.stride(-1) != 1:
            raise ValueError("the last dimension of positions must be dense")


def _say(inputs, rows, vectors=(), accumulate=False):
    """Raises what is wrong with arguments that the compiled helper has refused.  ``rows``: (name,
    tensor, the input it is like, whether it must be given); ``vectors``: (name, tensor, gamma)."""
    _say_inputs(*inputs)
    q = inputs[0]
    for name, t, like, needed in rows:
        if t is None and (like is None or not needed):
            continue
        if t is None or like is None:
            raise ValueError(f"{name} must be given exactly when its input is" if needed else
                             f"{name} given without its input")
        _rows(t, name, like)
        if tuple(t.shape) != tuple(like.shape):
            raise ValueError(f"{name} must have shape {tuple(like.shape)}, got {tuple(t.shape)}")
    for name, t, gamma in vectors:
        if gamma is None and t is not None:
            raise ValueError(f"{name} given without its gamma")
        if gamma is not None and t is None and accumulate:
            raise ValueError(f"accumulate_dgamma needs {name}")
        _abi._check_buffer(t, name, torch.float32, (q.shape[-1],), q.device)
    raise TypeError("q, k and all that goes with them must be dense CUDA tensors of torch with memory "
                    "of their own")


def qk_norm_rope_forward(q, k, gamma_q, gamma_k, inv_freq, positions=None, eps: float = 1e-6,
                         interleaved: bool = False, q_out=None, k_out=None, stream=None):
    """Norm of every head's row of q and k, then the rotation by position.  Returns (q, k) of the
    inputs' shapes (dense unless ``q_out`` / ``k_out`` are given; these may be q and k themselves, and
    must not overlap each other or the inputs in another way).

    ``gamma_q`` / ``gamma_k`` [D]: None for a norm without weights.  ``inv_freq`` [rot/2] float32:
    the rotated elements are the first ``rot``; None for no rotation.  ``positions`` int64 [T] or
    [B, T]; None numbers the tokens 0 .. T-1.  ``k`` may be None (queries only)."""
    inputs = (q, k, gamma_q, gamma_k, inv_freq, positions, eps, interleaved)
    if stream is None:
        made = _abi.marshal().qk_forward(*inputs, q_out, k_out)
    else:
        with on_stream(stream, q.device):
            made = _abi.marshal().qk_forward(*inputs, q_out, k_out)
    if made is None:
        _say(inputs, (("q_out", q_out, q, False), ("k_out", k_out, k, False)))
    if made[0] != _abi.FLCE_OK:
        raise _abi.FlceError(made[0], "flce_qk_norm_rope_forward")
    return made[1:]


def qk_norm_rope_backward(dq_out, dk_out, q, k, gamma_q, gamma_k, inv_freq, positions=None,
                          eps: float = 1e-6, interleaved: bool = False, dq=None, dk=None,
                          dgamma_q=None, dgamma_k=None, accumulate_dgamma: bool = False,
                          stream=None):
    """Chain rule of qk_norm_rope_forward for the gradients of its outputs.  Returns
    (dq, dk, dgamma_q, dgamma_k); the gammas' gradients are float32, written or (with
    ``accumulate_dgamma``) added to, and None where there is no gamma.  ``dgamma_q`` and ``dgamma_k``
    may not be one buffer, even where gamma_q and gamma_k are: add the two."""
    inputs = (q, k, gamma_q, gamma_k, inv_freq, positions, eps, interleaved)
    with on_stream(stream, q.device):
        made = _abi.marshal().qk_backward(*inputs, dq_out, dk_out, dq, dk, dgamma_q, dgamma_k,
                                          accumulate_dgamma)
    if made is None:
        _say(inputs, (("dq_out", dq_out, q, True), ("dk_out", dk_out, k, True),
                      ("dq", dq, q, False), ("dk", dk, k, False)),
             (("dgamma_q", dgamma_q, gamma_q), ("dgamma_k", dgamma_k, gamma_k)),
             accumulate_dgamma)
    if made[0] != _abi.FLCE_OK:
        raise _abi.FlceError(made[0], "flce_qk_norm_rope_backward")
    return made[1:]


def _dense_last(t):
    """The gradient as autograd hands it, copied only when its layout cannot be read."""
    if t is None:
        return None
    unit = 16 // t.element_size()
    ok = (t.shape[-1] <= 1 or t.stride(-1) == 1) and t.data_ptr() % 16 == 0 and all(
        n <= 1 or s % unit == 0 for n, s in zip(t.shape[:-1], t.stride()[:-1]))
    return t if ok else t.contiguous()


class QKNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, gamma_q, gamma_k, inv_freq, positions, eps, interleaved):
        qo, ko = qk_norm_rope_forward(q, k, gamma_q, gamma_k, inv_freq, positions, eps,
                                      interleaved)
        ctx.save_for_backward(q, k, gamma_q, gamma_k, inv_freq, positions)
        ctx.meta = (eps, interleaved)
        return qo, ko

    @staticmethod
    @once_differentiable
    def backward(ctx, dqo, dko):
        q, k, gamma_q, gamma_k, inv_freq, positions = ctx.saved_tensors
        dq, dk, dgq, dgk = qk_norm_rope_backward(
            _dense_last(dqo), _dense_last(dko), q, k, gamma_q, gamma_k, inv_freq, positions,
            *ctx.meta)
        wants = ctx.needs_input_grad
        return (dq if wants[0] else None, dk if wants[1] else None, dgq if wants[2] else None,
                dgk if wants[3] else None, None, None, None, None)


def qk_norm_rope(q, k, gamma_q, gamma_k, inv_freq, positions=None, eps: float = 1e-6,
                 interleaved: bool = False):
    """qk_norm_rope_forward with gradients into q, k, gamma_q and gamma_k (the gammas' are formed
    in float32 and cast to their dtype by autograd).  As with torch's own operators, a backward pass
    is captured into a CUDA graph only while no graph built outside the capture holds the same
    leaves."""
    return QKNormRope.apply(q, k, gamma_q, gamma_k, inv_freq, positions, eps, interleaved)
