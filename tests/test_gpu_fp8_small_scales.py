"""The quantiser where its scales are small, at quotients that lie on the border between two codes or a step beside it.

code = x / scale is an fp32 quotient rounded once, and then rounded to e4m3: as the quotient in 64 bits rounded to 32 gives it, equal (zeros of
either sign are).
"""
import math

import pytest
import torch

import linear_attention_chunkwise_gb300 as kda
from tests.conftest import cuda_ok
from tests.test_gpu_fp8 import BF, E4M3, F32, gen, plain_quantize

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]


def borders():
    """The values halfway between two codes of e4m3 that lie beside each other, in 64 bits."""
    codes = torch.arange(0x7F, dtype=torch.uint8).view(E4M3).double()
    return (codes[1:] + codes[:-1]) / 2


def rows_at_borders(exponent, rows, dtype, seed, form):
    """Rows of 128: the largest of 2^exponent to 2^(exponent + 1), which sets the scale (of 128 rows in blocks), and the values of that type
    that its borders are nearest to, or up to two steps beside them."""
    g = gen(seed)
    most = (torch.rand(rows, 1, device="cuda", generator=g).double() + 1).mul(2.0 ** exponent).to(dtype)
    if form == "blocks":
        most = most[::128].repeat_interleave(128, 0)
    scale = (most.double() / 448).float().clamp_min(2.0 ** -126)
    at = borders().cuda()
    pick = at[torch.randint(0, len(at), (rows, 127), device="cuda", generator=g)]
    x = (pick * scale.double()).to(dtype)
    step = torch.randint(-2, 3, x.shape, device="cuda", generator=g)
    bits = x.view(torch.int32 if dtype is F32 else torch.int16)
    x = torch.where(bits > 2, bits + step.to(bits.dtype), bits).view(dtype)
    sign = torch.randint(0, 2, x.shape, device="cuda", generator=g) * 2 - 1
    return torch.cat([most, x * sign.to(dtype)], 1)


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("form", ["rows", "columns", "blocks"])
@pytest.mark.parametrize("exponent", [-140, -126, -118, -110, -100, -93, -84, -80, -60, 0, 100, 126])
def test_codes_at_their_borders(exponent, form, dtype):
    x = rows_at_borders(exponent, 8192, dtype, seed=200 + exponent, form=form)
    if form == "columns":
        x = x.T.contiguous()
    want, want_s = plain_quantize(x, form)
    codes, scales = kda.kda_fp8_quantize(x, form=form)
    assert torch.equal(scales, want_s)
    assert torch.equal(codes.float(), want.float()), int((codes.float() != want.float()).sum())


@pytest.mark.parametrize("form", ["rows", "columns", "blocks"])
def test_one_quotient_by_hand(form):
    """x / scale lies a quarter step under 0.484375, the border between 0.46875 and 0.5, and rounds to it."""
    scale, value = 1.7829773e-37, 8.636296e-38
    x = torch.zeros(128, 128, device="cuda")
    x[0, 0], x[0, 1] = 448 * torch.tensor(scale), value
    if form == "columns":
        x = x.T.contiguous()
    codes, scales = kda.kda_fp8_quantize(x, form=form)
    want, want_s = plain_quantize(x, form)
    assert torch.equal(scales, want_s) and torch.equal(codes.float(), want.float())
    assert math.isclose(float(scales[0, 0]), scale, rel_tol=1e-6)
