"""Products in 8-bit floats where a block goes through several tiles: what it carries from one to the next (the walk over the experts, turns of
the operands' and the scales' rings and of the accumulators), in each form that the launch chooses.

K = 656 and 1168 are 6 and 10 blocks: no multiple of the 4 whose scales come together, nor of the 4 or 5 stages of the ring.
"""
import pytest
import torch

import linear_attention_chunkwise_gb300 as kda
from tests.conftest import cuda_ok
from tests.test_gpu_fp8 import BF, E4M3, F32, check, ordinary, wide, whole

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

# rows of each expert: on average up to 8, 32, 80 and more; some without rows, runs of those longer than a warp looks at at once
GAP = [0] * 40
GROUPS = {"tiles of 16": [3, 0, 8, 20, 1, 5, 7, 9, 4, 2] * 4 + GAP + [33, 1, 6] * 4,
          "tiles of 32": [20, 0, 70, 31, 1, 33] * 8 + GAP + [64, 90, 5, 250] * 3,
          "tiles of 64": [60, 130, 0, 64, 1, 200] * 8 + GAP + [300, 65, 90] * 3,
          "pairs": [700, 0, 129, 1, 256, 257] + GAP + [2000, 300, 511, 400, 0, 900]}


def average(lengths):
    return -(-sum(lengths) // len(lengths))


def tiles(lengths, rows, along):
    return sum(-(-n // rows) for n in lengths) * along


def test_the_groups_are_what_they_say():
    """By the launch's rule, with two tiles or more for each place of 152 SMs (two blocks an SM, or pairs)."""
    g = GROUPS
    assert average(g["tiles of 16"]) <= 8 < average(g["tiles of 32"]) <= 32 < average(g["tiles of 64"]) <= 80 < average(g["pairs"])
    assert all(tiles(g[f"tiles of {n}"], n, -(-2050 // 128)) > 2 * 304 for n in (16, 32, 64)) and tiles(g["pairs"], 256, -(-2602 // 256)) > 2 * 76


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("form", ["blocks", "rows"])
@pytest.mark.parametrize("K", [656, 1168])
@pytest.mark.parametrize("name", GROUPS)
def test_grouped(name, K, form, dtype):
    lengths, N = GROUPS[name], 2602 if name == "pairs" else 2050
    T, E = sum(lengths), len(lengths)
    offsets = torch.tensor([sum(lengths[:i]) for i in range(E + 1)], dtype=torch.int32, device="cuda")
    for make in (whole, ordinary):
        x, xs = make((T, K), "rows", 11)
        w, ws = make((E, N, K), form, 13)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = torch.full((T + 3, N), 7.0, dtype=dtype, device="cuda")
        kda.kda_fp8_matmul_grouped(x, xs, w, ws, offsets, out=out[:T], device_status=status)
        at = 0
        for e, n in enumerate(lengths):
            if not n:
                continue
            px, pw = wide(x[at:at + n], xs[at:at + n], "rows"), wide(w[e], ws[e], form)
            if make is whole:
                assert torch.equal(out[at:at + n], (px @ pw.T).to(dtype)), e
            else:
                check(out[at:at + n], px, pw, K)
            at += n
        assert bool((out[T:] == 7.0).all()) and int(status) == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("form", ["blocks", "rows"])
@pytest.mark.parametrize("M,N,K", [(2500, 2602, 656), (2500, 2602, 1168), (24, 60000, 656), (24, 60000, 1168)])
def test_matmul(M, N, K, form, dtype):
    """110 tiles for 76 pairs, 469 or more for 304 places."""
    x, xs = whole((M, K), "rows", 1)
    w, ws = whole((N, K), form, 3)
    assert torch.equal(kda.kda_fp8_matmul(x, xs, w, ws, out_dtype=dtype), (wide(x, xs, "rows") @ wide(w, ws, form).T).to(dtype))
    x, xs = ordinary((M, K), "rows", 5)
    w, ws = ordinary((N, K), form, 7)
    got = kda.kda_fp8_matmul(x, xs, w, ws, out_dtype=dtype)
    check(got, wide(x, xs, "rows"), wide(w, ws, form), K)
    assert torch.equal(got, kda.kda_fp8_matmul(x, xs, w, ws, out_dtype=dtype))


@pytest.mark.parametrize("lengths", [[5, 0, 3, 9], [300, 0, 77, 500]])
def test_gradient_of_the_experts_rows(lengths):
    """dx = dy W of each expert: the grouped product with its codes and block scales turned over."""
    T, E, N, K = sum(lengths), len(lengths), 400, 528
    offsets = torch.tensor([sum(lengths[:i]) for i in range(E + 1)], dtype=torch.int32, device="cuda")
    dy, ds = ordinary((T, N), "rows", 1)
    w, ws = ordinary((E, N, K), "blocks", 3)
    wt, wts = w.view(torch.uint8).transpose(1, 2).contiguous().view(E4M3), ws.transpose(1, 2).contiguous()
    dx = kda.kda_fp8_matmul_grouped(dy, ds, wt, wts, offsets)
    assert dx.shape == (T, K)
    for e, (d, s, got) in enumerate(zip(dy.split(lengths), ds.split(lengths), dx.split(lengths))):
        check(got, wide(d, s, "rows"), wide(w[e], ws[e], "blocks").T, N)
