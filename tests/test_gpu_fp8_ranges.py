"""What kda.h asks of a layer's products in 8-bit floats: lengths that are multiples of 16 (zeros fill up the others), and scales whose products
fp32 holds."""
import pytest
import torch

import linear_attention_chunkwise_gb300 as kda
from tests.conftest import cuda_ok
from tests.test_gpu_fp8 import BF, E4M3, F32, check, randn, wide, whole

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]


def filled(x, rows):
    return torch.nn.functional.pad(x, (0, 0, 0, rows - len(x)))


def turned(codes, scales):
    return codes.view(torch.uint8).T.contiguous().view(E4M3), scales.T.contiguous()


def refused(call):
    with pytest.raises(kda.KdaError) as told:
        call()
    assert told.value.status == kda.KDA_ERR_UNSUPPORTED


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("T", [1, 15, 129, 777, 1037])
def test_a_weights_gradient_over_any_number_of_tokens(T, dtype):
    """dW = dy^T x: its K is the tokens.  Rows of zeros behind them leave every scale and code as it is."""
    N, K, whole_T = 144, 260, -(-T // 16) * 16
    dy, x = randn(T, N, seed=1, dtype=dtype), randn(T, K, seed=2, dtype=dtype)
    (dc, ds), (xc, xs) = (kda.kda_fp8_quantize(t, form="columns") for t in (dy, x))
    refused(lambda: kda.kda_fp8_matmul(dc, ds, xc, xs, out_dtype=F32))
    (dz, dzs), (xz, xzs) = (kda.kda_fp8_quantize(filled(t, whole_T), form="columns") for t in (dy, x))
    assert torch.equal(dz[:, :T].float(), dc.float()) and not bool(dz[:, T:].float().any()) and torch.equal(dzs, ds)
    assert torch.equal(xz[:, :T].float(), xc.float()) and not bool(xz[:, T:].float().any()) and torch.equal(xzs, xs)
    check(kda.kda_fp8_matmul(dz, dzs, xz, xzs, out_dtype=F32), wide(dc, ds, "rows"), wide(xc, xs, "rows"), T)


@pytest.mark.parametrize("N", [1, 100, 257])
def test_an_inputs_gradient_with_any_number_of_outputs(N):
    """dx = dy W: its K is the weights' rows, and dy's columns."""
    T, K, whole_N = 75, 272, -(-N // 16) * 16
    dy, w = randn(T, N, seed=1, dtype=BF), randn(N, K, seed=2, dtype=BF)
    (dc, ds), (wc, ws) = kda.kda_fp8_quantize(dy), kda.kda_fp8_quantize(w, form="blocks")
    refused(lambda: kda.kda_fp8_matmul(dc, ds, *turned(wc, ws)))
    (dz, dzs), (wz, wzs) = kda.kda_fp8_quantize(filled(dy.T, whole_N).T.contiguous()), kda.kda_fp8_quantize(filled(w, whole_N), form="blocks")
    assert torch.equal(dz[:, :N].float(), dc.float()) and torch.equal(dzs, ds) and torch.equal(wz[:N].float(), wc.float()) and torch.equal(wzs, ws)
    check(kda.kda_fp8_matmul(dz, dzs, *turned(wz, wzs)), wide(dc, ds, "rows"), wide(wc, ws, "blocks").T, N)


@pytest.mark.parametrize("form", ["blocks", "rows"])
@pytest.mark.parametrize("M", [5, 100, 600])
def test_scales_of_any_size_whose_product_is_normal(M, form):
    """x's scales from 2^-120 to 2^120, w's so that the products are 2^-100 to 2^100: sums of whole codes, exact."""
    x, _ = whole((M, 256), "rows", 1)
    w, ws = whole((256, 256), form, 3)
    for of_x, of_w in ((120, -20), (120, -120), (-120, 20), (-20, -80), (60, 40), (0, 100)):
        xs, each = torch.full((M, 2), 2.0 ** of_x, device="cuda"), torch.full_like(ws, 2.0 ** of_w)
        got = kda.kda_fp8_matmul(x, xs, w, each, out_dtype=F32)
        assert torch.equal(got, (wide(x, xs, "rows") @ wide(w, each, form).T).to(F32))
