"""Outputs that a call makes for another stream than the current one."""
import pytest
import torch

import linear_attention_chunkwise_gb300 as kda
from linear_attention_chunkwise_gb300 import synth
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


# ------------------------------------------------- the channel-wise siblings ----
def _sibling_jobs():
    p = synth.prefill_inputs([300, 77], 4, s0_std=0.1, seed=205)
    x = (p.q, p.k, p.v, p.log_alpha, p.beta, p.cu_seqlens)
    dO = torch.randn(p.v.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(206)).bfloat16()
    at = torch.tensor([0, 1], dtype=torch.int32, device="cuda"), torch.tensor([64, 77], dtype=torch.int32, device="cuda")
    norm = kda.Fusion(l2norm_qk=True)
    S = p.S0[:1].expand(377, -1, -1, -1).contiguous()
    step = (p.q, p.k, p.v, p.log_alpha, p.beta)
    many = tuple(t.unsqueeze(1) for t in step)
    return {"prefill": lambda s: kda.kda_prefill(*x, p.S0, stream=s),
            "snapshots": lambda s: kda.kda_prefill_snapshots(*x, *at, p.S0, stream=s),
            "ex": lambda s: kda.kda_prefill_ex(*x, p.S0, fusion=norm, stream=s),
            "backward": lambda s: kda.kda_prefill_backward(*x, dO, p.S0, stream=s),
            "decode": lambda s: (kda.kda_decode_step(*step, S.clone() if s is None else S, stream=s),),
            "multi": lambda s: (kda.kda_decode_multi(*many, S.clone() if s is None else S, stream=s),)}


@pytest.mark.parametrize("name", ["prefill", "snapshots", "ex", "backward", "decode", "multi"])
def test_sibling_outputs_are_not_in_memory_that_the_current_stream_still_writes(name):
    call = _sibling_jobs()[name]
    flat = lambda r: [t for t in (r[0] if isinstance(r[0], tuple) else r) if t is not None]  # noqa: E731
    want = [t.clone() for t in flat(call(None))]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda._sleep(SPIN)
    old = [torch.empty_like(t) for t in want]
    for t in old:
        t.view(torch.uint8).fill_(77)
    del old, t
    got = flat(call(side))
    side.synchronize()
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(got, want)), name


def test_a_siblings_workspace_is_not_handed_on_while_its_kernels_run():
    """The call's own workspace goes back to the allocator when it returns; the current stream must not get it then."""
    p = synth.prefill_inputs([2000, 700], 8, s0_std=0.1, seed=207)
    args = (p.q, p.k, p.v, p.log_alpha, p.beta, p.cu_seqlens, p.S0)
    want = [t.clone() for t in kda.kda_prefill(*args)]
    need = kda.kda_prefill_workspace_bytes(torch.bfloat16, 2, 2700, 8)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    for _ in range(3):
        with torch.cuda.stream(side):
            torch.cuda._sleep(SPIN // 10)
        got = kda.kda_prefill(*args, stream=side)
        scratch = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        del scratch
