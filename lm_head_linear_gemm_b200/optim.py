"""AdamW over many tensors in one launch, with states in 32 or in 8 bits, and the global gradient
norm: what a training loop does with the gradients the head, the norms and the rest of the model
leave behind.

    opt = AdamW([dict(params=[W], lr=0.002828, betas=(0.8, 0.96), eps=1e-10, weight_decay=0.01),
                 dict(params=[gamma], lr=1e-3, weight_decay=0.0)], state_bits=8)
    norm, factor = grad_norm(opt.grads(), max_norm=1.0)
    opt.step(grad_scale=factor)            # clipped on the device, nothing waits for the host

include/flce_train.h states the formulas and the 8-bit format.
"""
from __future__ import annotations

import contextlib
from array import array
from ctypes import c_float
from types import MappingProxyType

import torch

from . import _abi
from .qk_norm import _DTYPES, on_stream

__all__ = ["AdamW", "grad_norm"]


def on_device(device):
    """A context in which the device is the current one."""
    same = device.index == torch._C._cuda_getDevice()
    return contextlib.nullcontext() if same else torch.cuda.device(device)


def device_scalar(t, name, device):
    """The address of a one-element float32 tensor on the device; None for None."""
    if t is None:
        return None
    _abi._check_scalar(t, name, torch.float32, device)
    _abi._check_memory(t, name)
    return t.data_ptr()


def grad_norm(grads, max_norm: float | None = None, stream=None):
    """(norm, factor) of a list of gradients (None entries are left out) as one-element float32
    device tensors: the L2 norm over all of them and ``min(1, max_norm / (norm + 1e-6))``, NaN when
    the norm is not finite; factor is None without ``max_norm``.  Nothing waits for the host."""
    grads = list(grads)
    dev = None if stream is None else next((g.device for g in grads if g is not None), None)
    with on_stream(stream, dev):
        made = _abi.marshal().grad_norm(grads, max_norm)
    if made is None:
        raise ValueError("grad_norm needs at least one gradient")
    rc, norm, factor = made
    if rc != _abi.FLCE_OK:
        raise _abi.FlceError(rc, "flce_grad_norm")
    return norm, factor


class AdamW:
    """AdamW (decoupled weight decay) over many tensors, one launch for every 384 of them.

    ``params``: tensors, or groups ``dict(params=[...], lr=, betas=, eps=, weight_decay=,
    states=)`` that override the arguments (at most 16 groups).  Parameters are contiguous float32
    or bfloat16 CUDA tensors on one device; gradients may be float32 or bfloat16 whatever the
    parameter's type.  The groups stand in ``param_groups`` and their numbers may be changed between
    steps; ``lr`` may be a one-element float32 device tensor, which a captured step reads anew.
    It is no ``torch.optim.Optimizer``: it has no ``zero_grad`` (set the gradients to None), and torch's
    learning-rate schedulers do not take it (write the rate into the group, or into its tensor).

    ``state_bits`` = 32: ``m`` and ``v`` in float32.  8: e4m3 codes of m and of r = sqrt(v) with a
    float32 scale for every 256 elements, for tensors of at least ``min_8bit_size`` elements (a
    small tensor's states stay in 32 bits; 0 puts all in 8 bits, which is faster: a launch with one
    tensor of fp32 states keeps fewer tiles in flight).  A tensor with an array off its alignment
    (fp32 at 32 bytes, others at 16) is stepped element by element, two to four times slower.
    ``master_weights``: bf16 parameters get a float32 copy that takes the update; the parameter is
    its rounding. ``states`` of a group adopts the caller's tensors instead of zeros: for each
    parameter a dict with ``m`` and ``v``, or ``m``, ``r``, ``m_scale`` and ``r_scale``, and
    ``master`` where there is one.

    ``state`` has a read-only dict of tensors for each parameter: their values may be written, the
    tensors not replaced.  ``step_count`` [1] int64 on the device counts the steps done (``step=``
    adopts the caller's).  Every parameter shares it: one without a gradient in a step is left as it
    is.  With ``skip_nonfinite`` a step whose ``grad_scale`` is not finite (grad_norm's factor after an
    overflow) changes nothing and is not counted.  An optimizer's steps follow one another: they must
    not overlap on the GPU (on two streams, or in two graphs replayed at once)."""

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.95), eps: float = 1e-8,
                 weight_decay: float = 0.01, state_bits: int = 32, min_8bit_size: int = 4096,
                 master_weights: bool = False, step=None, skip_nonfinite: bool = True):
        if state_bits not in (8, 32):
            raise ValueError(f"state_bits must be 8 or 32, got {state_bits}")
        if isinstance(params, torch.Tensor):
            raise TypeError("params must be a list of tensors or of groups, got a tensor")
        groups = list(params)
        if not groups:
            raise ValueError("AdamW needs at least one parameter")
        if not isinstance(groups[0], dict):
            groups = [dict(params=groups)]
        if len(groups) > _abi.ADAMW_MAX_GROUPS:
            raise ValueError(f"at most {_abi.ADAMW_MAX_GROUPS} groups, got {len(groups)}")
        self.param_groups, self.params, self.state = [], [], []
        self.skip_nonfinite = bool(skip_nonfinite)
        self._group_of = []
        defaults = dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay)
        for k, group in enumerate(groups):
            unknown = set(group) - set(defaults) - {"params", "states"}
            if unknown:
                raise TypeError(f"unknown group entries {sorted(unknown)}")
            g = {**defaults, **group}
            one = isinstance(g["params"], torch.Tensor)
            g["params"] = [g["params"]] if one else list(g["params"])
            states = g.pop("states", None)
            if states is not None and len(states) != len(g["params"]):
                raise ValueError("states must have one entry for each parameter of its group")
            self.param_groups.append(g)
            for i, p in enumerate(g["params"]):
                self._check_param(p)
                self.params.append(p)
                self._group_of.append(k)
                # read-only: the library is given these tensors' addresses once
                self.state.append(MappingProxyType(
                    dict(states[i]) if states is not None else
                    self._new_state(p, state_bits == 8 and p.numel() >= min_8bit_size,
                                    master_weights)))
        if not self.params:
            raise ValueError("AdamW needs at least one parameter")
        dev = self.device = self.params[0].device
        if step is None:
            step = torch.zeros(1, dtype=torch.int64, device=dev)
        _abi._check_buffer(step, "step", torch.int64, (1,), dev)
        _abi._check_memory(step, "step")
        self.step_count = step
        self._scratch = torch.zeros(4, dtype=torch.int32, device=dev)
        n = len(self.params)
        self._tensors = (_abi.flce_adamw_tensor * n)()
        self._grad_types = bytes(array("i", [_DTYPES[torch.float32]]) * n)
        self._describe()

    # ------------------------------------------------------------------ parameters and states
    @staticmethod
    def _check_param(p):
        if not p.is_cuda:
            raise ValueError("parameters must be CUDA tensors")
        if p.dtype not in _DTYPES:
            raise TypeError(f"parameters must be float32 or bfloat16, got {p.dtype}")
        if not p.is_contiguous():
            raise ValueError("parameters must be contiguous")
        _abi._check_memory(p, "every parameter")

    @staticmethod
    def _new_state(p, eight, master):
        n, dev = p.numel(), p.device
        if eight:
            blocks = -(-n // _abi.STATE_BLOCK)
            s = {name: torch.zeros(n, dtype=torch.uint8, device=dev).view(torch.float8_e4m3fn)
                 for name in ("m", "r")}
            for name in ("m_scale", "r_scale"):
                s[name] = torch.zeros(blocks, dtype=torch.float32, device=dev)
        else:
            s = {name: torch.zeros(n, dtype=torch.float32, device=dev) for name in ("m", "v")}
        if master and p.dtype == torch.bfloat16:
            s["master"] = p.detach().float().reshape(-1)
        return s

    def _describe(self):
        """The library's descriptors of all tensors, checked."""
        for i, (p, s) in enumerate(zip(self.params, self.state)):
            self._tensors[i] = self._descriptor(p, s, array("i", self._grad_types)[i],
                                                self._group_of[i])
        self._check_overlap()
        none = [None] * len(self.params)
        self._places = _abi.marshal().gradients(none, self.params, 0, self._grad_types)[2]

    def _descriptor(self, p, s, grad_code, group):
        self._check_param(p)
        dev, n, eight = self.device, p.numel(), "r" in s
        if p.device != dev:
            raise ValueError(f"every parameter must be on {dev}")
        names = {"m", "r", "m_scale", "r_scale"} if eight else {"m", "v"}
        if set(s) - {"master"} != names:
            raise ValueError("a state holds m and v, or m, r, m_scale and r_scale, and may hold "
                             f"master; got {sorted(s)}")
        code = torch.float8_e4m3fn if eight else torch.float32
        for name, t in s.items():
            size = -(-n // _abi.STATE_BLOCK) if name.endswith("_scale") else n
            if t.numel() != size:
                raise ValueError(f"{name} must have {size} elements, got {t.numel()}")
            _abi._check_buffer(t, name, code if name in ("m", "v", "r") else torch.float32,
                               tuple(t.shape), dev)
            _abi._check_memory(t, name)
        if "master" in s and p.dtype != torch.bfloat16:
            raise ValueError("only a bfloat16 parameter takes a master copy")
        ptr = {name: t.data_ptr() for name, t in s.items()}
        return _abi.flce_adamw_tensor(
            p.data_ptr(), ptr["m"], ptr["r" if eight else "v"], ptr.get("m_scale"),
            ptr.get("r_scale"), ptr.get("master"), n, _DTYPES[p.dtype], grad_code,
            _abi.STATE_E4M3 if eight else _abi.STATE_F32, group)

    def _check_overlap(self):
        """A step writes its tensors in any order: none may share memory with another."""
        spans = sorted((t.data_ptr(), t.numel() * t.element_size())
                       for p, s in zip(self.params, self.state) for t in (p, *s.values())
                       if t.numel())
        for (a, size), (b, _) in zip(spans, spans[1:]):
            if a + size > b:
                raise ValueError("parameters and states must not overlap (a parameter listed "
                                 "twice, or views of the same memory)")

    def grads(self):
        """Every parameter's gradient as ``step`` takes it: ``main_grad`` where the parameter has
        one (the float32 buffer the fused loss accumulates into), else ``grad``; may be None."""
        return [g if (g := getattr(p, "main_grad", None)) is not None else p.grad
                for p in self.params]

    # ------------------------------------------------------------------ the step
    def _groups(self):
        out = (_abi.flce_adamw_group * len(self.param_groups))()
        for o, g in zip(out, self.param_groups):
            lr = g["lr"]
            if isinstance(lr, torch.Tensor):
                o.lr_device = device_scalar(lr, "lr", self.device)
            else:
                o.lr = float(lr)
            o.beta1, o.beta2 = g["betas"]
            o.eps, o.weight_decay = float(g["eps"]), float(g["weight_decay"])
        return out

    def step(self, grads=None, grad_scale=None, stream=None):
        """One step.  ``grads``: a list in the order of ``params`` (all groups' parameters one after
        the other) with None for a parameter to leave alone; default ``self.grads()``.
        ``grad_scale`` multiplies every gradient: a float (in a captured step its value stays) or a
        one-element float32 device tensor."""
        grads = self.grads() if grads is None else list(grads)
        n, dev = len(self.params), self.device
        pointers, types, places = _abi.marshal().gradients(grads, self.params, dev.index,
                                                           self._grad_types)
        if places != self._places:                       # p.data was replaced
            self._describe()
        if types != self._grad_types:
            for tensor, code in zip(self._tensors, array("i", types)):
                tensor.grad_dtype = code
            self._grad_types = types
        with on_stream(stream, dev), on_device(dev):
            handle = torch._C._cuda_getCurrentRawStream(dev.index)
            if grad_scale is not None and not isinstance(grad_scale, torch.Tensor):
                # a fill, not a copy from the host: nothing waits, and a capture may hold it
                grad_scale = torch.full((), c_float(grad_scale).value, dtype=torch.float32,
                                        device=dev)
            rc = _abi.lib().flce_adamw_step(
                self._tensors, pointers, n, self._groups(), len(self.param_groups),
                device_scalar(grad_scale, "grad_scale", dev), self.step_count.data_ptr(),
                int(self.skip_nonfinite), self._scratch.data_ptr(), handle)
        if rc != _abi.FLCE_OK:
            raise _abi.FlceError(rc, "flce_adamw_step")
        _abi.marshal().stepped(grads, self.params)

    def status(self) -> int:
        """Device status bits of the steps so far (DEV_TIMEOUT: a wait inside a kernel ran out and
        its step is incomplete); waits for the steps issued on the current stream."""
        return int(self._scratch[1])

    # ------------------------------------------------------------------ checkpoints
    def state_dict(self):
        """Group numbers, states and the step count (references, as torch's optimizers give)."""
        return {"step": self.step_count,
                "groups": [{k: v for k, v in g.items() if k != "params"}
                           for g in self.param_groups],
                "state": [dict(s) for s in self.state]}

    def load_state_dict(self, saved):
        """Copies a state_dict's values into this optimizer's tensors; the layout (bits, master
        copies, sizes) has to be this optimizer's.  Where this optimizer's learning rate is on the
        device, the saved one, a tensor or a number, is written into it, so that a captured step
        follows."""
        if len(saved["state"]) != len(self.state) or len(saved["groups"]) != len(self.param_groups):
            raise ValueError("the saved optimizer has other parameters or groups")
        for mine, theirs in zip(self.state, saved["state"]):
            if set(mine) != set(theirs) or any(
                    mine[k].numel() != theirs[k].numel() or mine[k].dtype != theirs[k].dtype
                    for k in mine):
                raise ValueError("a saved state has another layout than this optimizer's")
        for mine, theirs in zip(self.state, saved["state"]):
            for k in mine:
                mine[k].copy_(theirs[k].reshape(mine[k].shape))
        for mine, theirs in zip(self.param_groups, saved["groups"]):
            for k, v in theirs.items():
                own, given = mine.get(k), isinstance(v, torch.Tensor)
                if isinstance(own, torch.Tensor):        # a rate on the device: its own tensor stays
                    own.copy_(v.reshape(own.shape)) if given else own.fill_(v)
                else:
                    mine[k] = v.to(self.device, copy=True) if given else v
        self.step_count.copy_(saved["step"])
