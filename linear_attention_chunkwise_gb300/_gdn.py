"""Entry points of the gated delta rule and of the RMS norm (include/kda.h).  Argument marshalling only.

As in ``_binding``: tensors are checked, outputs allocated when the caller passes none, and raw pointers
handed to libkda.so, on the current stream of the tensors' own device or on ``stream``.
"""
from __future__ import annotations

import torch

from . import _binding as _b

_NORM_OUT = {None: (_b.KDA_NORM_OUT_SAME, None), "e4m3": (_b.KDA_NORM_OUT_E4M3, torch.float8_e4m3fn),
             "int8": (_b.KDA_NORM_OUT_INT8, torch.int8)}
# the current stream's handle without the Stream object that torch.cuda.current_stream makes of it (2 us)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
# the current device without torch.cuda.current_device's look whether CUDA is up: a call's tensors are there
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device

# PyTorch's allocator on the current device, (bytes, stream handle) -> address; torch.cuda.caching_allocator_alloc less
# its device switch
_allocate = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc", None) or (
    lambda size, stream: torch.cuda.caching_allocator_alloc(size, stream=stream))
_free = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_delete", None) or torch.cuda.caching_allocator_delete


def _check(t, name, dtype, shape, dev):
    """t: a contiguous CUDA tensor of this type, shape and device."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.device == dev
            and t.is_contiguous()):
        _refuse(t, name, dtype, shape, dev)


def _refuse(t, name, dtype, shape, dev):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    raise ValueError(f"{name} must be contiguous")


def _first(t, name, dims):
    """(device, dtype code) that the call goes by; t has `dims` dimensions."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {t.dim()}")
    return t.device, _b._dtype_code(t.dtype)


def _contiguous(t, name):
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _p(t):
    return None if t is None else t.data_ptr()


def _call(function, dev, *args):
    """The call with its tensors' device current: launches go to it whatever device the caller has current."""
    if _current_device() == dev.index:
        st = function(*args)
    else:
        with torch.cuda.device(dev):
            st = function(*args)
    if st != _b.KDA_OK:
        raise _b.KdaError(function.__name__, st, _b.kda_status_string(st))


def _call_with_workspace(function, dev, workspace, need, args, rest):
    """_call(args, workspace and its bytes, rest), with the caller's workspace, or one of `need` bytes for this call.

    That one comes from PyTorch's allocator without a tensor around it (4 us), for the stream that the call
    goes to, rest[-1], and is back with the allocator once the launches are queued on it.
    """
    if workspace is not None:
        return _call(function, dev, *args, workspace.data_ptr(), workspace.numel(), *rest)
    if _current_device() != dev.index:
        with torch.cuda.device(dev):
            return _call_with_workspace(function, dev, None, need, args, rest)
    need = max(need, 256)
    memory = _allocate(need, rest[-1])
    try:
        _call(function, dev, *args, memory, need, *rest)
    finally:
        _free(memory)


def _stream(stream, dev):
    """The handle of the stream that the call goes to."""
    if stream is None:
        return _current_stream(dev.index)
    if stream.device != dev:
        raise ValueError(f"stream is on {stream.device}, expected {dev}")
    return stream.cuda_stream


def _new(stream, dev, make, *args, **kwargs):
    """An output of this call, make(...), in memory of the stream that writes it.

    A block of the current stream's may still be in use there, by work queued before the block was freed, which the
    caller's `stream` does not wait for.  Where the caller drops the output, it is free once the current stream is done with it too.
    """
    if stream is None:
        return make(*args, **kwargs)
    current = torch.cuda.current_stream(dev)
    with torch.cuda.stream(stream):
        t = make(*args, **kwargs)
    t.record_stream(current)
    return t


def _heads(q, v, name):
    """Hk, Hv, dk, dv of q [.., Hk, dk] and v [.., Hv, dv]."""
    if not isinstance(v, torch.Tensor) or v.dim() != q.dim():
        raise ValueError(f"v must be {name}")
    return q.shape[-2], v.shape[-2], q.shape[-1], v.shape[-1]


def _sequences(cu_seqlens, dev):
    """Their number."""
    N = cu_seqlens.numel() - 1 if isinstance(cu_seqlens, torch.Tensor) else 0
    if N < 0:
        raise ValueError("cu_seqlens must have at least one entry")
    _check(cu_seqlens, "cu_seqlens", torch.int32, (N + 1,), dev)
    return N


def kda_gdn_prefill_workspace_bytes(qkv_dtype, num_seqs: int, total_tokens: int, Hk: int, Hv: int, dk: int = 128,
                                    dv: int = 128) -> int:
    code = qkv_dtype if isinstance(qkv_dtype, int) else _b._dtype_code(qkv_dtype)
    return int(_b.load_library().held.kda_gdn_prefill_workspace_bytes(
        code, int(num_seqs), int(total_tokens), int(Hk), int(Hv), int(dk), int(dv)))


def kda_gdn_prefill(q, k, v, log_decay, beta, cu_seqlens, S0=None, *, o=None, S_final=None, return_final=True,
                    workspace=None, device_status=None, stream=None):
    """Prefill of the gated delta rule over packed sequences (see include/kda.h).

    q, k: [T, Hk, 128]; v: [T, Hv, 128] (bf16 or fp32), Hv a multiple of Hk; log_decay, beta: [T, Hv] fp32;
    cu_seqlens: int32 [N+1] on the device; S0: fp32 [N, Hv, 128, 128] or None.  Returns (o, S_final) --
    S_final is None when return_final is False and none was given.
    """
    lib = _b.load_library()
    dev, code = _first(q, "q", 3)
    T = q.shape[0]
    Hk, Hv, dk, dv = _heads(q, v, "[T, Hv, 128]")
    _contiguous(q, "q")
    _check(k, "k", q.dtype, (T, Hk, dk), dev)
    _check(v, "v", q.dtype, (T, Hv, dv), dev)
    _check(log_decay, "log_decay", torch.float32, (T, Hv), dev)
    _check(beta, "beta", torch.float32, (T, Hv), dev)
    N = _sequences(cu_seqlens, dev)
    if S0 is not None:
        _check(S0, "S0", torch.float32, (N, Hv, dk, dv), dev)
    handle = _stream(stream, dev)
    if o is None:
        o = _new(stream, dev, torch.empty_like, v)
    else:
        _check(o, "o", q.dtype, (T, Hv, dv), dev)
    if S_final is not None:
        _check(S_final, "S_final", torch.float32, (N, Hv, dk, dv), dev)
    elif return_final:
        S_final = _new(stream, dev, torch.empty, (N, Hv, dk, dv), dtype=torch.float32, device=dev)
    need = 0
    if workspace is None:
        need = lib.held.kda_gdn_prefill_workspace_bytes(code, N, T, Hk, Hv, dk, dv)
    else:
        _b._check(workspace, "workspace", torch.uint8, dev)
    _b._check(device_status, "device_status", torch.int32, dev)
    _call_with_workspace(
        lib.kda_gdn_prefill, dev, workspace, need,
        (q.data_ptr(), k.data_ptr(), v.data_ptr(), code, log_decay.data_ptr(), beta.data_ptr(), _p(S0),
         cu_seqlens.data_ptr(), N, T, Hk, Hv, dk, dv, o.data_ptr(), _p(S_final)),
        (_p(device_status), handle))
    return o, S_final


def kda_gdn_prefill_backward_workspace_bytes(qkv_dtype, num_seqs: int, total_tokens: int, Hk: int, Hv: int,
                                             dk: int = 128, dv: int = 128) -> int:
    code = qkv_dtype if isinstance(qkv_dtype, int) else _b._dtype_code(qkv_dtype)
    return int(_b.load_library().held.kda_gdn_prefill_backward_workspace_bytes(
        code, int(num_seqs), int(total_tokens), int(Hk), int(Hv), int(dk), int(dv)))


def kda_gdn_prefill_backward(q, k, v, log_decay, beta, cu_seqlens, grad_o, S0=None, grad_S_final=None, *,
                             need_grad_S0=True, grads=None, workspace=None, device_status=None, stream=None):
    """Gradient of kda_gdn_prefill for L = <o, grad_o> + <S_final, grad_S_final> (see include/kda.h; bf16).

    grad_o: [T, Hv, 128] in the dtype of q; grad_S_final: fp32 [N, Hv, 128, 128] or None (zeros).
    Returns (grad_q, grad_k, grad_v, grad_log_decay, grad_beta, grad_S0): the first three in the dtype of q,
    the others fp32; grad_S0 is None when need_grad_S0 is False.  `grads` may pass those six tensors in.
    """
    lib = _b.load_library()
    dev, code = _first(q, "q", 3)
    T = q.shape[0]
    Hk, Hv, dk, dv = _heads(q, v, "[T, Hv, 128]")
    f32 = torch.float32
    _contiguous(q, "q")
    _check(k, "k", q.dtype, (T, Hk, dk), dev)
    _check(v, "v", q.dtype, (T, Hv, dv), dev)
    _check(grad_o, "grad_o", q.dtype, (T, Hv, dv), dev)
    _check(log_decay, "log_decay", f32, (T, Hv), dev)
    _check(beta, "beta", f32, (T, Hv), dev)
    N = _sequences(cu_seqlens, dev)
    state = (N, Hv, dk, dv)
    for x, name in ((S0, "S0"), (grad_S_final, "grad_S_final")):
        if x is not None:
            _check(x, name, f32, state, dev)
    specs = (("grad_q", q.dtype, (T, Hk, dk)), ("grad_k", q.dtype, (T, Hk, dk)), ("grad_v", q.dtype, (T, Hv, dv)),
             ("grad_log_decay", f32, (T, Hv)), ("grad_beta", f32, (T, Hv)), ("grad_S0", f32, state))
    handle = _stream(stream, dev)
    if grads is None:
        grads = tuple(_new(stream, dev, torch.empty_like, t) for t in (q, k, v, log_decay, beta)) + (
            _new(stream, dev, torch.empty, state, dtype=f32, device=dev) if need_grad_S0 else None,)
    elif len(grads) != 6:
        raise ValueError("grads must hold 6 tensors")
    else:
        for x, (n, dt, shape) in zip(grads, specs):
            if x is not None or n != "grad_S0":
                _check(x, n, dt, shape, dev)
    need = 0
    if workspace is None:
        need = lib.held.kda_gdn_prefill_backward_workspace_bytes(code, N, T, Hk, Hv, dk, dv)
    else:
        _b._check(workspace, "workspace", torch.uint8, dev)
    _b._check(device_status, "device_status", torch.int32, dev)
    _call_with_workspace(
        lib.kda_gdn_prefill_backward, dev, workspace, need,
        (q.data_ptr(), k.data_ptr(), v.data_ptr(), code, log_decay.data_ptr(), beta.data_ptr(), _p(S0),
         cu_seqlens.data_ptr(), N, T, Hk, Hv, dk, dv, grad_o.data_ptr(), _p(grad_S_final), *(_p(x) for x in grads)),
        (_p(device_status), handle))
    return tuple(grads)


def kda_gdn_decode_step(q, k, v, log_decay, beta, S, state_indices=None, *, o=None, device_status=None,
                        stream=None):
    """One token of the gated delta rule; S [slots, Hv, 128, 128] fp32 is updated in place.

    q, k: [N, Hk, 128]; v: [N, Hv, 128] (bf16 or fp32); log_decay, beta: [N, Hv] fp32; state_indices:
    int32 [N] or None (slot n for sequence n).  Returns o [N, Hv, 128].
    """
    lib = _b.load_library()
    dev, code = _first(q, "q", 3)
    N = q.shape[0]
    Hk, Hv, dk, dv = _heads(q, v, "[N, Hv, 128]")
    _contiguous(q, "q")
    _check(k, "k", q.dtype, (N, Hk, dk), dev)
    _check(v, "v", q.dtype, (N, Hv, dv), dev)
    _check(log_decay, "log_decay", torch.float32, (N, Hv), dev)
    _check(beta, "beta", torch.float32, (N, Hv), dev)
    slots = S.shape[0] if isinstance(S, torch.Tensor) and S.dim() else 0
    _check(S, "S", torch.float32, (slots, Hv, dk, dv), dev)
    if state_indices is not None:
        _check(state_indices, "state_indices", torch.int32, (N,), dev)
    handle = _stream(stream, dev)
    if o is None:
        o = _new(stream, dev, torch.empty_like, v)
    else:
        _check(o, "o", q.dtype, (N, Hv, dv), dev)
    _b._check(device_status, "device_status", torch.int32, dev)
    _call(lib.kda_gdn_decode_step, dev,
          q.data_ptr(), k.data_ptr(), v.data_ptr(), code, log_decay.data_ptr(), beta.data_ptr(), S.data_ptr(),
          slots, _p(state_indices), N, Hk, Hv, dk, dv, o.data_ptr(), _p(device_status),
          handle)
    return o


def kda_rms_norm(x, weight=None, residual=None, *, eps=1e-6, quant=None, group=0, y=None, scales=None,
                 residual_out=None, stream=None):
    """h = x + residual, y = h / sqrt(mean h^2 + eps) * weight over the last dimension (see include/kda.h).

    x, residual: [rows, dim] (bf16 or fp32); weight: fp32 [dim] or None (ones).  quant: None (y in the
    type of x), "e4m3" or "int8", with one fp32 scale for each row (group=0) or for every 128 columns
    (group=128).  Returns (y, scales, residual_out): scales [rows, scales in a row] is None without quant,
    residual_out (h in the type of x) None without a residual.
    """
    lib = _b.load_library()
    dev, code = _first(x, "x", 2)
    rows, dim = x.shape
    _contiguous(x, "x")
    if weight is not None:
        _check(weight, "weight", torch.float32, (dim,), dev)
    if quant not in _NORM_OUT:
        raise ValueError(f"quant must be None, 'e4m3' or 'int8', got {quant!r}")
    out_type, out_dtype = _NORM_OUT[quant]
    if group not in ((0, 128) if quant else (0,)) or (group and dim % group):
        raise ValueError(f"group must be 0, or 128 with an 8-bit output and dim a multiple of it, got {group}")
    handle = _stream(stream, dev)
    if residual is not None:
        _check(residual, "residual", x.dtype, (rows, dim), dev)
    if residual_out is not None:
        _check(residual_out, "residual_out", x.dtype, (rows, dim), dev)
    elif residual is not None:
        residual_out = _new(stream, dev, torch.empty_like, x)
    if y is None:
        y = _new(stream, dev, torch.empty_like, x, dtype=out_dtype)
    else:
        _check(y, "y", out_dtype or x.dtype, (rows, dim), dev)
    if quant:
        shape = (rows, dim // group if group else 1)
        if scales is None:
            scales = _new(stream, dev, torch.empty, shape, dtype=torch.float32, device=dev)
        else:
            _check(scales, "scales", torch.float32, shape, dev)
    elif scales is not None:
        raise ValueError("scales are written with an 8-bit output only")
    _call(lib.kda_rms_norm, dev,
          x.data_ptr(), _p(residual), code, _p(weight), eps, rows, dim, out_type, group, y.data_ptr(), _p(scales),
          _p(residual_out), handle)
    return y, scales, residual_out


def kda_rms_norm_backward_workspace_bytes(rows: int, dim: int) -> int:
    return int(_b.load_library().held.kda_rms_norm_backward_workspace_bytes(int(rows), int(dim)))


def kda_rms_norm_backward(grad_y, h, weight=None, *, grad_h=None, eps=1e-6, need_grad_weight=True, grad_x=None,
                          grad_weight=None, workspace=None, stream=None):
    """Gradient of kda_rms_norm for L = <y, grad_y> + <h, grad_h> (see include/kda.h).

    grad_y, h, grad_h: [rows, dim] of one type (bf16 or fp32), h the normed row (residual_out, or x);
    weight: fp32 [dim] or None (ones).  Returns (grad_x, grad_weight): grad_x, in that type, is the
    gradient of x and of residual alike; grad_weight fp32 [dim], or None when not asked for.
    """
    lib = _b.load_library()
    dev, code = _first(h, "h", 2)
    rows, dim = h.shape
    _contiguous(h, "h")
    _check(grad_y, "grad_y", h.dtype, (rows, dim), dev)
    if grad_h is not None:
        _check(grad_h, "grad_h", h.dtype, (rows, dim), dev)
    if weight is not None:
        _check(weight, "weight", torch.float32, (dim,), dev)
    handle = _stream(stream, dev)
    if grad_x is None:
        grad_x = _new(stream, dev, torch.empty_like, h)
    else:
        _check(grad_x, "grad_x", h.dtype, (rows, dim), dev)
    if grad_weight is not None:
        _check(grad_weight, "grad_weight", torch.float32, (dim,), dev)
    elif need_grad_weight:
        grad_weight = _new(stream, dev, torch.empty, (dim,), dtype=torch.float32, device=dev)
    need = 0
    if workspace is not None:
        _b._check(workspace, "workspace", torch.uint8, dev)
    elif grad_weight is not None:
        need = lib.held.kda_rms_norm_backward_workspace_bytes(rows, dim)
    args = (grad_y.data_ptr(), h.data_ptr(), _p(grad_h), code, _p(weight), eps, rows, dim, grad_x.data_ptr(),
            _p(grad_weight))
    if grad_weight is None and workspace is None:
        _call(lib.kda_rms_norm_backward, dev, *args, None, 0, handle)
    else:
        _call_with_workspace(lib.kda_rms_norm_backward, dev, workspace, need, args, (handle,))
    return grad_x, grad_weight
