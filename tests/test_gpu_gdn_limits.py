"""The gated delta rule's kernels with every pipeline wait expired, and with their ranges checked.

As for the prefill and its gradient of the channel-wise rule: a copy of the library whose pipeline waits
expire when they are not over at the first look (KDA_PIPE_WAIT_CYCLES=0; what is waited for completes as
usual) has to come back with KDA_DEV_TIMEOUT, and one that checks every range it derives (KDA_DEBUG_BOUNDS)
has to give the same bits and find nothing.
"""
import os

import pytest
import torch

import linear_attention_chunkwise_gb300 as kda
from linear_attention_chunkwise_gb300 import _binding, _build
from tests.conftest import cuda_ok
from tests.test_gpu_debug_bounds import DBG_DIR, _both, _using
from tests.test_gpu_gdn import check, inputs
from tests.test_gpu_gdn_backward import check as check_grads
from tests.test_gpu_gdn_backward import with_grads
from tests.test_gpu_wait_limit import WAIT_DIR

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

# few and many (sequence, value head) pairs, more chunks than a pipeline has stages; the last in clusters
LAYOUTS = [([300, 77, 130], 1, 3), ([700, 0, 65], 16, 32), ([64] * 45, 2, 4), ([130, 64], 2, 4)]


@pytest.fixture(scope="module")
def wait_lib():
    return _binding.load_library(_build.build(extra_flags=["-DKDA_PIPE_WAIT_CYCLES=0"], build_dir=WAIT_DIR,
                                              lib_path=os.path.join(WAIT_DIR, "libkda_pipe_wait_0.so")))


@pytest.fixture(scope="module")
def libs():
    path = _build.build(extra_flags=["-DKDA_DEBUG_BOUNDS"], lib_path=os.path.join(DBG_DIR, "libkda_debug_bounds.so"),
                        build_dir=DBG_DIR)
    return _binding.load_library(), _binding.load_library(path)


@pytest.mark.parametrize("lengths,Hk,Hv", LAYOUTS)
def test_expired_waits_in_the_prefill(wait_lib, lengths, Hk, Hv):
    x = inputs(lengths, Hk, Hv, seed=101)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    with _using(wait_lib):
        kda.kda_gdn_prefill(**x, device_status=status)
        torch.cuda.synchronize()
    assert int(status.item()) & kda.KDA_DEV_TIMEOUT
    check(x, *kda.kda_gdn_prefill(**x))


@pytest.mark.parametrize("lengths,Hk,Hv", LAYOUTS)
def test_expired_waits_in_the_gradient(wait_lib, lengths, Hk, Hv):
    x = with_grads(inputs(lengths, Hk, Hv, seed=102))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    with _using(wait_lib):
        kda.kda_gdn_prefill_backward(**x, device_status=status)
        torch.cuda.synchronize()
    assert int(status.item()) & kda.KDA_DEV_TIMEOUT
    check_grads(x, kda.kda_gdn_prefill_backward(**x))


@pytest.mark.parametrize("lengths,Hk,Hv", LAYOUTS + [([1, 2], 1, 2), ([333], 40, 80)])
def test_ranges(libs, lengths, Hk, Hv):
    x = inputs(lengths, Hk, Hv, seed=103)
    y = with_grads(x)
    assert _both(libs, lambda s: kda.kda_gdn_prefill(**x, device_status=s)) == 0
    assert _both(libs, lambda s: kda.kda_gdn_prefill_backward(**y, device_status=s)) == 0


@pytest.mark.parametrize("Hv", [2, 32])
@pytest.mark.parametrize("cu", [[0, 50, 40, 100], [1, 30, 60, 100], [0, 30, 200, 100]])
def test_ranges_of_malformed_cu_seqlens(libs, cu, Hv):
    x = with_grads(inputs([30, 30, 40], Hv, Hv, seed=104))
    x["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    y = {n: t for n, t in x.items() if n not in ("grad_o", "grad_S_final")}

    def forward(s):
        o = torch.zeros_like(x["v"])
        kda.kda_gdn_prefill(**y, o=o, return_final=False, device_status=s)
        return (o,)

    def back(s):
        like = [x[n] for n in ("q", "k", "v", "log_decay", "beta", "S0")]
        return kda.kda_gdn_prefill_backward(**x, grads=tuple(torch.zeros_like(t) for t in like), device_status=s)

    assert _both(libs, forward) == kda.KDA_DEV_BAD_CU_SEQLENS
    assert _both(libs, back) == kda.KDA_DEV_BAD_CU_SEQLENS
