"""Entry points of the products in 8-bit floats (include/kda.h).  Argument marshalling only, as in ``_gdn``."""
from __future__ import annotations

import torch

from . import _binding as _b
from ._gdn import _call, _check, _contiguous, _new, _p, _stream

_E4M3, _F32 = torch.float8_e4m3fn, torch.float32
_FORMS = {"blocks": _b.KDA_FP8_BLOCKS, "rows": _b.KDA_FP8_ROWS, "columns": _b.KDA_FP8_COLUMNS}


def _blocks(n):
    return -(-n // 128)


def _empty(shape, dtype, stream, dev):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    return _new(stream, dev, torch.empty, shape, dtype=dtype, device=dev)


def _codes(t, name, dims):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, got {t.dim()}")
    if t.dtype is not _E4M3:
        raise TypeError(f"{name} must be {_E4M3}, got {t.dtype}")
    _contiguous(t, name)


def _product(function, x, x_scales, w, w_scales, offsets, out_dtype, out, device_status, stream):
    _codes(x, "x", 2)
    dev = x.device
    M, K = x.shape
    _codes(w, "w", 2 if offsets is None else 3)
    N = w.shape[-2]
    _check(w, "w", _E4M3, (*w.shape[:-1], K), dev)
    _check(x_scales, "x_scales", _F32, (M, _blocks(K)), dev)
    # one scale for a row of w where there are as many as rows, else for a block of 128 x 128
    form = "rows" if isinstance(w_scales, torch.Tensor) and w_scales.dim() == w.dim() and w_scales.shape[-2] == N else "blocks"
    _check(w_scales, "w_scales", _F32, (*w.shape[:-2], N if form == "rows" else _blocks(N), _blocks(K)), dev)
    if offsets is not None:
        _check(offsets, "offsets", torch.int32, (w.shape[0] + 1,), dev)
    handle = _stream(stream, dev)
    if out is None:
        code = _b._dtype_code(out_dtype)
        out = _empty((M, N), out_dtype, stream, dev)
    else:
        code = _b._dtype_code(out.dtype if isinstance(out, torch.Tensor) else out_dtype)
        _check(out, "out", out.dtype if isinstance(out, torch.Tensor) else out_dtype, (M, N), dev)
    if device_status is not None:
        _b._check(device_status, "device_status", torch.int32, dev)
    group = () if offsets is None else (offsets.data_ptr(), w.shape[0])
    _call(function, dev, x.data_ptr(), x_scales.data_ptr(), w.data_ptr(), w_scales.data_ptr(), _FORMS[form], *group, M, N, K,
          code, out.data_ptr(), _p(device_status), handle)
    return out


def kda_fp8_matmul(x, x_scales, w, w_scales, *, out_dtype=torch.bfloat16, out=None, device_status=None, stream=None):
    """x w^T of e4m3 codes with an fp32 scale for every 128 of them along K (see include/kda.h).

    x: [M, K], x_scales: [M, ceil(K / 128)] (as kda_rms_norm gives them with quant="e4m3", group=128); w: [N, K],
    w_scales: [ceil(N / 128), ceil(K / 128)], or [N, ceil(K / 128)] for a scale a row; K a multiple of 16.
    Returns out [M, N] in out_dtype (bf16 or fp32), or in the type of the `out` that is given.
    """
    return _product(_b.load_library().kda_fp8_matmul, x, x_scales, w, w_scales, None, out_dtype, out, device_status, stream)


def kda_fp8_matmul_grouped(x, x_scales, w, w_scales, offsets, *, out_dtype=torch.bfloat16, out=None, device_status=None,
                           stream=None):
    """kda_fp8_matmul for rows packed by expert: rows offsets[e] to offsets[e + 1] times w[e]^T (see include/kda.h).

    x: [rows, K], x_scales: [rows, ceil(K / 128)]; w: [experts, N, K], w_scales: [experts, ceil(N / 128) or N,
    ceil(K / 128)]; offsets: int32 [experts + 1] on the device.  Returns out [rows, N]; rows from the last offset on
    are left as they are (in an `out` made here: not set).
    """
    if not isinstance(offsets, torch.Tensor):
        raise TypeError("offsets must be a torch.Tensor")
    return _product(_b.load_library().kda_fp8_matmul_grouped, x, x_scales, w, w_scales, offsets, out_dtype, out,
                    device_status, stream)


def kda_fp8_quantize(x, *, form="rows", codes=None, scales=None, stream=None):
    """x in e4m3 with fp32 scales (see include/kda.h): (codes, scales).

    x: [rows, cols] (bf16 or fp32).  form "rows": a scale for 128 of a row, codes [rows, cols], scales [rows,
    ceil(cols / 128)]; "blocks": for 128 x 128, scales [ceil(rows / 128), ceil(cols / 128)]; "columns": the rows form of
    the transposed x, codes [cols, rows], scales [cols, ceil(rows / 128)].  A product over those codes takes a multiple
    of 16 rows of x: fill others up with rows of zeros, which change no scale and no code.
    """
    lib = _b.load_library()
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    if x.dim() != 2:
        raise ValueError(f"x must have 2 dimensions, got {x.dim()}")
    if form not in _FORMS:
        raise ValueError(f"form must be 'rows', 'blocks' or 'columns', got {form!r}")
    _contiguous(x, "x")
    dev, code = x.device, _b._dtype_code(x.dtype)
    rows, cols = x.shape
    shape = (cols, rows) if form == "columns" else (rows, cols)
    scale_shape = (_blocks(rows) if form == "blocks" else shape[0], _blocks(shape[1]))
    handle = _stream(stream, dev)
    if codes is None:
        codes = _empty(shape, _E4M3, stream, dev)
    else:
        _check(codes, "codes", _E4M3, shape, dev)
    if scales is None:
        scales = _empty(scale_shape, _F32, stream, dev)
    else:
        _check(scales, "scales", _F32, scale_shape, dev)
    _call(lib.kda_fp8_quantize, dev, x.data_ptr(), code, rows, cols, _FORMS[form], codes.data_ptr(), scales.data_ptr(), handle)
    return codes, scales
