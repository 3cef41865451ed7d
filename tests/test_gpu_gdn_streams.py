"""Outputs that a call makes for another stream than the current one."""
import pytest
import torch

import linear_attention_chunkwise_gb300 as kda
from tests.conftest import cuda_ok
from tests.test_gpu_gdn import inputs
from tests.test_gpu_gdn_backward import with_grads

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

SPIN = 100_000_000  # cycles, some 50 ms: far longer than the calls


def _jobs():
    x = inputs([300, 77], 2, 4, seed=201)
    g = with_grads(x)
    rows = torch.randn(700, 1024, device="cuda", generator=torch.Generator("cuda").manual_seed(202)).bfloat16()
    S = x["S0"][:1].expand(377, -1, -1, -1).contiguous()
    step = [x[n] for n in ("q", "k", "v", "log_decay", "beta")]
    return {"prefill": lambda s: kda.kda_gdn_prefill(**x, stream=s),
            "backward": lambda s: kda.kda_gdn_prefill_backward(**g, stream=s),
            "decode": lambda s: (kda.kda_gdn_decode_step(*step, S.clone() if s is None else S, stream=s),),
            "norm": lambda s: kda.kda_rms_norm(rows, None, rows, quant="int8", stream=s),
            "norm_backward": lambda s: kda.kda_rms_norm_backward(rows, rows, stream=s)}


@pytest.mark.parametrize("name", ["prefill", "backward", "decode", "norm", "norm_backward"])
def test_outputs_are_not_in_memory_that_the_current_stream_still_writes(name):
    """Blocks of the outputs' sizes, freed while the current stream has yet to write them."""
    call = _jobs()[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for _ in range(2):  # the second time the side stream has blocks of its own
        torch.cuda._sleep(SPIN)
        old = [torch.empty_like(t) for t in want]
        for t in old:
            t.view(torch.uint8).fill_(77)
        del old, t
        got = call(side)
        side.synchronize()
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want)), name
        if name == "decode":
            break  # its state moves on
        del got


def test_dropped_outputs_wait_for_the_current_stream():
    """An output dropped while the current stream has yet to read it is not handed to the side stream's next call."""
    x, y = inputs([300], 2, 4, seed=203), inputs([300], 2, 4, seed=204)
    want, _ = kda.kda_gdn_prefill(**x)
    kda.kda_gdn_prefill(**y)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        o, _ = kda.kda_gdn_prefill(**x, stream=side, return_final=False)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(SPIN)
        kept = o.clone()
        del o
        other, _ = kda.kda_gdn_prefill(**y, stream=side, return_final=False)
        torch.cuda.synchronize()
        assert torch.equal(kept, want)
        del other
