"""Entry points of the gated linear recurrence (include/kda.h).  Argument marshalling only, as in ``_gdn``."""
from __future__ import annotations

import torch

from . import _binding as _b
from ._gdn import _call, _call_with_workspace, _check, _contiguous, _first, _new, _p, _sequences, _stream

_GATE_KINDS = {"log_decay": 0, "sigmoid": _b.KDA_GLR_SIGMOID}
_F32 = torch.float32


def _gate(gate, x, code, dev, gate_kind, complement):
    """(dtype code, flags) of the gates of x, whose code is given: in the type of x or fp32."""
    flags = _GATE_KINDS.get(gate_kind)
    if flags is None:
        raise ValueError(f"gate_kind must be 'log_decay' or 'sigmoid', got {gate_kind!r}")
    if isinstance(gate, torch.Tensor) and gate.dtype is _F32:
        _check(gate, "gate", _F32, x.shape, dev)
        code = _b.KDA_DTYPE_F32
    else:
        _check(gate, "gate", x.dtype, x.shape, dev)
    return code, flags | _b.KDA_GLR_COMPLEMENT if complement else flags


def _like(x, stream, dev):
    """An output of the shape and type of x."""
    return torch.empty_like(x) if stream is None else _new(stream, dev, torch.empty_like, x)


def _f32(shape, stream, dev):
    if stream is None:
        return torch.empty(shape, dtype=_F32, device=dev)
    return _new(stream, dev, torch.empty, shape, dtype=_F32, device=dev)


def _checkpoint_shape(T, dim):
    return -(-T // _b.KDA_GLR_CHECKPOINT), dim


def kda_glr_prefill(x, gate, cu_seqlens, h0=None, *, gate_kind="log_decay", complement=False, h=None, h_final=None,
                    return_final=True, checkpoints=None, return_checkpoints=False, device_status=None, stream=None):
    """h_t = a_t h_{t-1} + s_t x_t over packed sequences, channel by channel (see include/kda.h).

    x: [T, dim] (bf16 or fp32); gate: [T, dim] in that type or fp32, a = exp(gate) ("log_decay") or
    sigmoid(gate) ("sigmoid"); kda.h bounds log decays above 0; s = 1, or 1 - a with complement; cu_seqlens: int32
    [N+1] on the device; h0: fp32 [N, dim] or None.  Returns (h, h_final, checkpoints): h [T, dim] in the type of x,
    h_final fp32 [N, dim], or None when return_final is False and none was given; checkpoints fp32 [ceil(T / 64), dim]
    for kda_glr_prefill_backward, or None unless asked for or given.
    """
    lib = _b.load_library()
    dev, code = _first(x, "x", 2)
    T, dim = x.shape
    _contiguous(x, "x")
    gate_code, flags = _gate(gate, x, code, dev, gate_kind, complement)
    N = _sequences(cu_seqlens, dev)
    if h0 is not None:
        _check(h0, "h0", _F32, (N, dim), dev)
    handle = _stream(stream, dev)
    if h is None:
        h = _like(x, stream, dev)
    else:
        _check(h, "h", x.dtype, (T, dim), dev)
    if h_final is not None:
        _check(h_final, "h_final", _F32, (N, dim), dev)
    elif return_final:
        h_final = _f32((N, dim), stream, dev)
    if checkpoints is not None:
        _check(checkpoints, "checkpoints", _F32, _checkpoint_shape(T, dim), dev)
    elif return_checkpoints:
        checkpoints = _f32(_checkpoint_shape(T, dim), stream, dev)
    if device_status is not None:
        _b._check(device_status, "device_status", torch.int32, dev)
    _call(lib.kda_glr_prefill, dev,
          x.data_ptr(), code, gate.data_ptr(), gate_code, flags, _p(h0), cu_seqlens.data_ptr(), N, T, dim, h.data_ptr(),
          _p(h_final), _p(checkpoints), _p(device_status), handle)
    return h, h_final, checkpoints


def kda_glr_prefill_backward_workspace_bytes(total_tokens: int, dim: int) -> int:
    return int(_b.load_library().held.kda_glr_prefill_backward_workspace_bytes(int(total_tokens), int(dim)))


def kda_glr_prefill_backward(x, gate, cu_seqlens, grad_h, h0=None, grad_h_final=None, *, gate_kind="log_decay",
                             complement=False, checkpoints=None, need_grad_h0=True, grads=None, workspace=None,
                             device_status=None, stream=None):
    """Gradient of kda_glr_prefill for L = <h, grad_h> + <h_final, grad_h_final> (see include/kda.h).

    grad_h: [T, dim] in the type of x; grad_h_final: fp32 [N, dim] or None (zeros); checkpoints: those of the
    forward on these inputs, or None (the call runs it again for them).  Returns (grad_x, grad_gate, grad_h0)
    in the types of x, gate and fp32; grad_h0 is None when need_grad_h0 is False.  `grads` may pass those three
    tensors in.
    """
    lib = _b.load_library()
    dev, code = _first(x, "x", 2)
    T, dim = x.shape
    _contiguous(x, "x")
    gate_code, flags = _gate(gate, x, code, dev, gate_kind, complement)
    _check(grad_h, "grad_h", x.dtype, (T, dim), dev)
    N = _sequences(cu_seqlens, dev)
    for t, name in ((h0, "h0"), (grad_h_final, "grad_h_final")):
        if t is not None:
            _check(t, name, _F32, (N, dim), dev)
    if checkpoints is not None:
        _check(checkpoints, "checkpoints", _F32, _checkpoint_shape(T, dim), dev)
    handle = _stream(stream, dev)
    if grads is None:
        grads = (_like(x, stream, dev), _like(gate, stream, dev), _f32((N, dim), stream, dev) if need_grad_h0 else None)
    elif len(grads) != 3:
        raise ValueError("grads must hold 3 tensors")
    else:
        for t, name, dtype, shape in zip(grads, ("grad_x", "grad_gate", "grad_h0"), (x.dtype, gate.dtype, _F32),
                                         ((T, dim), (T, dim), (N, dim))):
            if t is not None or name != "grad_h0":
                _check(t, name, dtype, shape, dev)
    if workspace is not None:
        _b._check(workspace, "workspace", torch.uint8, dev)
    if device_status is not None:
        _b._check(device_status, "device_status", torch.int32, dev)
    args = (x.data_ptr(), code, gate.data_ptr(), gate_code, flags, _p(h0), cu_seqlens.data_ptr(), N, T, dim,
            grad_h.data_ptr(), _p(grad_h_final), _p(checkpoints), *(_p(t) for t in grads))
    rest = (_p(device_status), handle)
    if checkpoints is not None and workspace is None:
        _call(lib.kda_glr_prefill_backward, dev, *args, None, 0, *rest)
    else:
        need = lib.held.kda_glr_prefill_backward_workspace_bytes(T, dim) if workspace is None else 0
        _call_with_workspace(lib.kda_glr_prefill_backward, dev, workspace, need, args, rest)
    return tuple(grads)


def kda_glr_decode_step(x, gate, state, state_indices=None, *, gate_kind="log_decay", complement=False, h=None,
                        device_status=None, stream=None):
    """One token of the gated linear recurrence; state [slots, dim] fp32 is updated in place (see include/kda.h).

    x: [N, dim] (bf16 or fp32); gate: [N, dim] in that type or fp32; state_indices: int32 [N] or None (slot n
    for sequence n).  Returns h [N, dim] in the type of x.
    """
    lib = _b.load_library()
    dev, code = _first(x, "x", 2)
    N, dim = x.shape
    _contiguous(x, "x")
    gate_code, flags = _gate(gate, x, code, dev, gate_kind, complement)
    slots = state.shape[0] if isinstance(state, torch.Tensor) and state.dim() else 0
    _check(state, "state", _F32, (slots, dim), dev)
    if state_indices is not None:
        _check(state_indices, "state_indices", torch.int32, (N,), dev)
    handle = _stream(stream, dev)
    if h is None:
        h = _like(x, stream, dev)
    else:
        _check(h, "h", x.dtype, (N, dim), dev)
    if device_status is not None:
        _b._check(device_status, "device_status", torch.int32, dev)
    _call(lib.kda_glr_decode_step, dev,
          x.data_ptr(), code, gate.data_ptr(), gate_code, flags, state.data_ptr(), slots, _p(state_indices), N, dim,
          h.data_ptr(), _p(device_status), handle)
    return h
