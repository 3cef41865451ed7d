"""The RMS norm on the GPU against its formula in 64 bits.

Tolerances.  One rounding to the type of y or h: half a step, eps / 2.  Before it, fp32: the sum of dim
squares in blocks (dim / threads + log2 steps of 2^-24 at most; 64 x 2^-24 for every dim here), its root
and four products: MATH = 80 x 2^-24 of the value.  8 bits: the code is that of y / scale, so it is
half a step off at most -- e4m3 2^-4 of the value (2^-10 of the scale's unit below its normal range),
int8 half a unit -- and MATH more.
"""
import numpy as np
import pytest
import torch

import linear_attention_chunkwise_gb300 as kda
from tests.conftest import cuda_ok

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

MATH = 80 * 2.0 ** -24
QMAX = {"e4m3": 448.0, "int8": 127.0}


def randn(*shape, seed, dtype=torch.float32):
    return torch.randn(shape, device="cuda", generator=torch.Generator("cuda").manual_seed(seed)).to(dtype)


def formula(x, w, res, eps):
    h = x.double() if res is None else x.double() + res.double()
    h = h.to(x.dtype).double()
    y = h / (h.square().sum(-1, keepdim=True) / x.shape[1] + eps).sqrt()
    return (y if w is None else y * w.double()), h


def close(got, ref, rel, floor=0.0):
    assert bool(((got.double() - ref).abs() <= rel * ref.abs() + floor).all())


def check_norm(x, w, res, eps, got, quant, group):
    y, scales, h = got
    ref, rh = formula(x, w, res, eps)
    if res is not None:
        assert torch.equal(h.double(), rh)
    if not quant:
        return close(y, ref, torch.finfo(x.dtype).eps / 2 + MATH)
    ref = ref.view(x.shape[0], -1, group or x.shape[1])
    scale = (ref.abs().amax(-1) / QMAX[quant]).clamp_min(2.0 ** -126)
    close(scales, scale, MATH)
    value = y.float().view(ref.shape).double() * scales.double()[..., None]
    if quant == "e4m3":
        close(value, ref, 2.0 ** -4 + MATH, (scale * 2.0 ** -10 * (1 + MATH))[..., None])
    else:
        close(value, ref, MATH, (scale * (0.5 + 127 * MATH))[..., None])


ROWS_DIMS = [(1, 1), (3, 7), (1, 64), (9, 65), (5, 100), (17, 128), (8, 256), (2, 1000), (33, 1024), (3, 1025), (7, 2310),
             (4, 4096), (2, 8192), (3, 8200), (2, 12345), (2, 16384), (1, 32768), (2, 40000), (1, 65537)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,dim", ROWS_DIMS)
def test_norm(rows, dim, dtype):
    x, res, w = randn(rows, dim, seed=1, dtype=dtype), randn(rows, dim, seed=2, dtype=dtype), 1 + 0.3 * randn(dim, seed=3)
    check_norm(x, w, res, 1e-6, kda.kda_rms_norm(x, w, res), None, 0)
    check_norm(x, None, None, 1e-3, kda.kda_rms_norm(x, eps=1e-3), None, 0)


@pytest.mark.parametrize("quant", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,dim", ROWS_DIMS)
def test_norm_in_8_bits(rows, dim, dtype, quant):
    x, res, w = randn(rows, dim, seed=4, dtype=dtype), randn(rows, dim, seed=5, dtype=dtype), 1 + 0.3 * randn(dim, seed=6)
    check_norm(x, w, res, 1e-6, kda.kda_rms_norm(x, w, res, quant=quant), quant, 0)
    if dim % 128 == 0:
        x = x * torch.exp(2 * randn(1, dim, seed=7)).to(dtype)
        check_norm(x, w, None, 1e-6, kda.kda_rms_norm(x, w, quant=quant, group=128), quant, 128)


@pytest.mark.parametrize("dim", [96, 2048, 40000])
def test_norm_in_place(dim):
    x, res, w = randn(5, dim, seed=8, dtype=torch.bfloat16), randn(5, dim, seed=9, dtype=torch.bfloat16), randn(dim, seed=10)
    y, _, h = kda.kda_rms_norm(x, w, res)
    res2 = res.clone()
    assert torch.equal(kda.kda_rms_norm(x, w, res2, residual_out=res2)[0], y) and torch.equal(res2, h)
    x2 = x.clone()
    assert torch.equal(kda.kda_rms_norm(x2, w, res, residual_out=x2)[0], y) and torch.equal(x2, h)
    x3 = x.clone()
    kda.kda_rms_norm(x3, w, res, y=x3, residual_out=res2)
    assert torch.equal(x3, y)


@pytest.mark.parametrize("quant", [None, "e4m3", "int8"])
@pytest.mark.parametrize("dim", [128, 4096, 66048])
def test_norm_of_odd_rows(dim, quant):
    """Zeros, tiny and huge rows; NaN and infinity spoil their own row (or group) only."""
    x = randn(6, dim, seed=11)
    x[0] = 0
    x[1] *= 1e-18
    x[2] *= 1e17
    x[3, 5] = float("nan")
    x[4, 9] = float("inf")
    y, scales, _ = kda.kda_rms_norm(x, eps=1e-30, quant=quant)
    v = y.float() if quant is None else y.float() * scales
    assert bool((v[0] == 0).all()) and bool(torch.isfinite(v[[0, 1, 2, 5]]).all())
    close(v[[1, 2, 5]], formula(x[[1, 2, 5]], None, None, 1e-30)[0], 2.0 ** -4 + MATH, 6.0 / 127)
    assert bool(v[3].isnan().all()) and bool(v[4].isnan().any())
    if quant:
        assert bool(scales[3:5].isnan().all()) and bool(v[4].isnan().all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,dim", ROWS_DIMS + [(700, 72), (5000, 128), (1300, 1536), (613, 9000)])
def test_backward(rows, dim, dtype):
    h, dy, dh = (randn(rows, dim, seed=s, dtype=dtype) for s in (20, 21, 22))
    w = 1 + 0.3 * randn(dim, seed=23)
    for gh, ww in ((dh, w), (None, None)):
        dx, dw = kda.kda_rms_norm_backward(dy, h, ww, grad_h=gh)
        h64, dy64 = h.double(), dy.double()
        w64 = torch.ones(dim, device="cuda", dtype=torch.float64) if ww is None else w.double()
        r = (h64.square().sum(-1, keepdim=True) / dim + 1e-6).rsqrt()
        terms = (r * w64 * dy64, -h64 * r ** 3 / dim * (h64 * w64 * dy64).sum(-1, keepdim=True),
                 torch.zeros_like(h64) if gh is None else gh.double())
        size = terms[0].abs() + h64.abs() * r ** 3 / dim * (h64 * w64 * dy64).abs().sum(-1, keepdim=True) + terms[2].abs()
        ref = sum(terms)
        assert bool(((dx.double() - ref).abs() <= torch.finfo(dtype).eps / 2 * ref.abs() + MATH * size).all())
        # the rows are added in blocks of rows / 304 and then 10 + 32 shares
        each = dy64 * h64 * r
        steps = (rows // 304 + 64) * 2.0 ** -24
        assert bool(((dw.double() - each.sum(0)).abs() <= (MATH + steps) * each.abs().sum(0)).all())
    dx2, none = kda.kda_rms_norm_backward(dy, h, need_grad_weight=False)
    assert none is None and torch.equal(dx, dx2)
    assert torch.equal(dw, kda.kda_rms_norm_backward(dy, h)[1])


def test_backward_is_the_forwards_slope():
    """Central differences of the forward in fp32, for x and the weight."""
    x, w, dy, dh = randn(2, 24, seed=30), 1 + 0.3 * randn(24, seed=31), randn(2, 24, seed=32), randn(2, 24, seed=33)
    zero = torch.zeros_like(x)
    dx, dw = kda.kda_rms_norm_backward(dy, x, w, grad_h=dh)

    def loss(x, w):
        y, _, h = kda.kda_rms_norm(x, w, zero)
        return float((y.double() * dy.double()).sum() + (h.double() * dh.double()).sum())

    # step 2^-7: truncation ~ step^2, rounding of the 48 terms ~ 48 x 2^-24 x 3 / 2^-6: below 2e-3 both
    step = 2.0 ** -7
    for i in range(0, 48, 5):
        d = torch.zeros(48, device="cuda")
        d[i] = step
        d = d.view(2, 24)
        assert abs((loss(x + d, w) - loss(x - d, w)) / (2 * step) - float(dx.view(-1)[i])) < 2e-3
    for i in range(0, 24, 5):
        d = torch.zeros(24, device="cuda")
        d[i] = step
        assert abs((loss(x, w + d) - loss(x, w - d)) / (2 * step) - float(dw[i])) < 2e-3


def test_no_rows():
    x = torch.empty(0, 64, device="cuda", dtype=torch.bfloat16)
    assert kda.kda_rms_norm(x)[0].shape == (0, 64)
    dx, dw = kda.kda_rms_norm_backward(x, x)
    assert dx.shape == (0, 64) and bool((dw == 0).all())


def test_rows_behind_stay(rows=5, dim=2310):
    x = randn(rows, dim, seed=40, dtype=torch.bfloat16)
    y = torch.full((rows + 2, dim), 9.0, dtype=torch.bfloat16, device="cuda")
    kda.kda_rms_norm(x, y=y[:rows])
    assert bool((y[rows:] == 9.0).all())


def test_captured_with_its_gradient():
    x, res, dy = (randn(64, 1024, seed=s, dtype=torch.bfloat16) for s in (50, 51, 52))
    w = randn(1024, seed=53)
    want = kda.kda_rms_norm(x, w, res)
    dwant = kda.kda_rms_norm_backward(dy, want[2], w, grad_h=dy)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = kda.kda_rms_norm(x, w, res)
        dgot = kda.kda_rms_norm_backward(dy, got[2], w, grad_h=dy)
    graph.replay()
    for a, b in zip((want[0], want[2]) + dwant, (got[0], got[2]) + dgot):
        assert torch.equal(a, b)
    assert np.isfinite(float(dgot[1].sum()))
