"""The gated delta rule on the GPU against the fp64 oracle (the KDA recurrence with its decay broadcast).

Tolerances.  o is rounded once to its type: half a step, eps / 2 of the type, of the value (bf16 2^-8);
every other error is held to STATE, relative to the largest value of the row or state.  STATE = 5 x 2^-17:
at most five products of a chunk have an operand that is held as two bf16 terms, each off by at most
2^-17 of the value (for 2^e <= |x| < 2^(e+1) the first term leaves at most 2^(e-8), and the second, rounding
that, at most 2^(e-17)); fp32 rounding, 2^-24 a step over contractive steps, is far below it.
"""
import numpy as np
import pytest
import torch

import linear_attention_chunkwise_gb300 as kda
import oracle
from linear_attention_chunkwise_gb300 import synth
from tests.conftest import cuda_ok
from tests.gpu_util import host

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

STATE = 5 * 2.0 ** -17
# The chunkwise prefill (bf16) rounds four things to bf16 on the way to o: the state and U as the output
# products take them, P, and o itself.  A rounding is spread over +- half a step (2^-8 of the value), so
# in the 2-norm it is at most 2^-8 / sqrt(3) of what it rounds, and the four add up in squares at worst
# with equal weight on all of o: 2 x 2^-8 / sqrt(3) = 4.6e-3; twice that where Q S and P U cancel in o.
CHUNKED_O = 4 * 2.0 ** -8 / 3 ** 0.5


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def inputs(lengths, Hk, Hv, dtype=torch.bfloat16, seed=0, lo=-0.5, start=True):
    p = synth.prefill_inputs(lengths, Hv, dtype=dtype, lo=lo, s0_std=0.1 if start else None, seed=seed)
    return dict(q=p.q[:, :Hk].contiguous(), k=p.k[:, :Hk].contiguous(), v=p.v, log_decay=p.log_alpha[:, :, 0].contiguous(),
                beta=p.beta, cu_seqlens=p.cu_seqlens, S0=p.S0)


def reference(x):
    m = x["v"].shape[1] // x["q"].shape[1]
    rep = lambda t: host(t.repeat_interleave(m, 1))  # noqa: E731
    la = np.repeat(host(x["log_decay"])[:, :, None], 128, 2)
    return oracle.kda_prefill(rep(x["q"]), rep(x["k"]), host(x["v"]), la, host(x["beta"]),
                              x["cu_seqlens"].cpu().numpy(), host(x["S0"]))


def check_o(o, ref):
    o64, top = host(o).astype(np.float64), np.abs(ref).max(initial=1e-30)
    assert np.all(np.abs(o64 - ref) <= half_step(o.dtype) * np.abs(ref) * (1 + STATE) + STATE * top)


def check_chunked_o(o, ref):
    assert np.linalg.norm(host(o).astype(np.float64) - ref) <= CHUNKED_O * np.linalg.norm(ref)


def check_state(S, ref):
    d = np.abs(host(S).astype(np.float64) - ref)
    assert np.all(d <= STATE * np.abs(ref).max(axis=(-1, -2), initial=1e-30, keepdims=True))


def check(x, o, S):
    ro, rs = reference(x)
    if o.dtype == torch.bfloat16:
        check_chunked_o(o, ro)
    else:
        check_o(o, ro)
    check_state(S, rs)


CASES = [([1], 1, 1), ([2], 2, 4), ([63], 1, 3), ([64], 2, 2), ([65], 1, 2), ([16, 17, 15], 2, 2), ([128, 0, 1, 200], 2, 4),
         ([300, 77, 0, 0, 640, 129], 3, 6), ([1500], 2, 2), ([2111, 64, 1], 1, 4)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("lengths,Hk,Hv", CASES)
def test_prefill(lengths, Hk, Hv, dtype):
    x = inputs(lengths, Hk, Hv, dtype, seed=31 + sum(lengths))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, S = kda.kda_gdn_prefill(**x, device_status=status)
    assert int(status.item()) == 0
    check(x, o, S)


@pytest.mark.parametrize("lengths", [[5], [700]])
def test_prefill_without_start_or_final_state(lengths):
    x = inputs(lengths, 2, 2, start=False, seed=5)
    o, S = kda.kda_gdn_prefill(**x)
    o2, none = kda.kda_gdn_prefill(**x, return_final=False)
    assert none is None and torch.equal(o, o2)
    check(x, o, S)


@pytest.mark.parametrize("lengths", [[40], [900]])
def test_prefill_state_in_place_and_repeatable(lengths):
    x = inputs(lengths, 1, 2, seed=6)
    o, S = kda.kda_gdn_prefill(**x)
    y = dict(x, S0=x["S0"].clone())
    o2, S2 = kda.kda_gdn_prefill(**y, S_final=y["S0"])
    assert S2.data_ptr() == y["S0"].data_ptr() and torch.equal(S, S2) and torch.equal(o, o2)


@pytest.mark.parametrize("lengths", [[20, 9], [1000, 130]])
def test_prefill_extreme_decays(lengths):
    """Decays of 0 (log -inf, the lowest fp32 value, -1000) and of 1 among ordinary ones; beta 0 and 1."""
    x = inputs(lengths, 2, 2, seed=7)
    ld, T = x["log_decay"], sum(lengths)
    ld[3, 0], ld[7, 1], ld[8, 0] = -np.inf, torch.finfo(torch.float32).min, -1000.0
    ld[10:14] = 0.0
    ld[T // 2:, 1] = -30.0
    x["beta"][5], x["beta"][6] = 0.0, 1.0
    check(x, *kda.kda_gdn_prefill(**x))


def test_prefill_slow_decay_over_many_chunks():
    x = inputs([4096], 1, 1, lo=-1e-4, seed=8)
    check(x, *kda.kda_gdn_prefill(**x))


def test_prefill_similar_keys():
    """Keys that point the same way: the chunk's triangular system is far from the identity."""
    x = inputs([640], 1, 2, seed=9, lo=-0.02)
    k = x["k"].float() + 0.5 / 128 ** 0.5 * 4
    x["k"] = (k / k.norm(dim=-1, keepdim=True)).to(torch.bfloat16)
    check(x, *kda.kda_gdn_prefill(**x))


@pytest.mark.parametrize("cut", [1, 64, 100])
def test_prefill_in_parts_and_decode_agree(cut):
    """A prompt, the rest of it from the state, and a token: all as one walk."""
    x = inputs([200], 2, 4, seed=10)
    part = lambda a, b: {n: (t[a:b] if n not in ("S0", "cu_seqlens") else t) for n, t in x.items()}  # noqa: E731
    cu = lambda n: torch.tensor([0, n], dtype=torch.int32, device="cuda")  # noqa: E731
    _, S = kda.kda_gdn_prefill(**dict(part(0, cut), cu_seqlens=cu(cut)))
    o2, S = kda.kda_gdn_prefill(**dict(part(cut, 199), cu_seqlens=cu(199 - cut), S0=S))
    y = part(199, 200)
    o3 = kda.kda_gdn_decode_step(y["q"], y["k"], y["v"], y["log_decay"], y["beta"], S)
    ro, rs = reference(x)
    check_chunked_o(torch.cat([o2, o3]), ro[cut:])
    check_state(S, rs)


def test_prefill_no_tokens():
    x = inputs([0, 0], 1, 2, seed=11)
    o, S = kda.kda_gdn_prefill(**x)
    assert o.shape[0] == 0 and torch.equal(S, x["S0"])


@pytest.mark.parametrize("cu", [[0, 50, 40, 100], [0, 30, 60, 99], [1, 30, 60, 100], [0, -5, 60, 100], [0, 30, 200, 100]])
def test_prefill_bad_cu_seqlens(cu):
    x = inputs([30, 30, 40], 1, 2, seed=12)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    guard = torch.full((120, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    x["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    kda.kda_gdn_prefill(**x, o=guard[:100], device_status=status)
    assert int(status.item()) == kda.KDA_DEV_BAD_CU_SEQLENS
    assert bool((guard[100:] == 7.0).all())


def test_prefill_under_a_graph_and_on_a_stream():
    x = inputs([300, 100], 2, 4, seed=13)
    o, S = kda.kda_gdn_prefill(**x)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o1, S1 = kda.kda_gdn_prefill(**x, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(o, o1) and torch.equal(S, S1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2, S2 = kda.kda_gdn_prefill(**x)
    x["v"].mul_(-0.5)
    graph.replay()
    check(x, o2, S2)


# ------------------------------------------------------------------ decode ----
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,slots,Hk,Hv", [(1, 1, 1, 1), (3, 9, 2, 6), (16, 16, 4, 4), (65, 70, 1, 2)])
def test_decode(N, slots, Hk, Hv, dtype):
    x = inputs([1] * N, Hk, Hv, dtype, seed=40 + N, start=False)
    S = torch.randn(slots, Hv, 128, 128, device="cuda", generator=torch.Generator("cuda").manual_seed(N)) * 0.1
    idx = torch.randperm(slots, generator=torch.Generator().manual_seed(N))[:N].to(torch.int32).cuda()
    before = S.clone()
    o = kda.kda_gdn_decode_step(x["q"], x["k"], x["v"], x["log_decay"], x["beta"], S, idx)
    ro, rs = reference(dict(x, S0=before[idx.long()]))
    check_o(o, ro)
    check_state(S[idx.long()], rs)
    rest = torch.ones(slots, dtype=torch.bool, device="cuda")
    rest[idx.long()] = False
    assert torch.equal(S[rest], before[rest])


def test_decode_bad_slots_are_left_out():
    x = inputs([1] * 4, 1, 2, seed=50, start=False)
    S = torch.randn(4, 2, 128, 128, device="cuda")
    before, o = S.clone(), torch.full((4, 2, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    idx = torch.tensor([-1, 2, 4, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    kda.kda_gdn_decode_step(x["q"], x["k"], x["v"], x["log_decay"], x["beta"], S, idx, o=o, device_status=status)
    assert int(status.item()) == kda.KDA_DEV_BAD_SLOT
    assert torch.equal(S[[0, 1, 3]], before[[0, 1, 3]]) and not torch.equal(S[2], before[2])
    assert bool((o[[0, 2, 3]] == 3.0).all())


def test_decode_replayed_steps_match_the_prefill():
    x = inputs([24], 2, 4, seed=51)
    _, rs = reference(x)
    S = x["S0"].clone()
    cur = {n: x[n][:1].clone() for n in ("q", "k", "v", "log_decay", "beta")}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_gdn_decode_step(cur["q"], cur["k"], cur["v"], cur["log_decay"], cur["beta"], S)
    for t in range(24):
        for n, c in cur.items():
            c.copy_(x[n][t:t + 1])
        graph.replay()
    check_state(S, rs)


# ------------------------------------------- one CTA for a pair's 128 columns ----
# More than half as many (sequence, value head) pairs as a GPU has SMs take the wide scan (80 on 152 SMs).
WIDE = [([1 + (37 * i) % 131 for i in range(20)], 2, 4), ([64] * 40, 1, 2), ([0, 200, 65, 0, 1, 0, 129, 63, 0, 448], 4, 12),
        ([700], 40, 80), ([257, 40], 24, 48), ([900, 0, 330], 16, 32)]


@pytest.mark.parametrize("lengths,Hk,Hv", WIDE)
def test_prefill_many_pairs(lengths, Hk, Hv):
    x = inputs(lengths, Hk, Hv, seed=81 + sum(lengths))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, S = kda.kda_gdn_prefill(**x, device_status=status)
    assert int(status.item()) == 0
    check(x, o, S)
    y = dict(x, S0=x["S0"].clone())
    o2, S2 = kda.kda_gdn_prefill(**y, S_final=y["S0"])
    assert torch.equal(S, S2) and torch.equal(o, o2)
    o3, S3 = kda.kda_gdn_prefill(**dict(x, S0=None))
    check(dict(x, S0=torch.zeros_like(x["S0"])), o3, S3)


def test_prefill_many_pairs_extreme_decays():
    x = inputs([700, 1, 130], 16, 32, seed=82)
    ld = x["log_decay"]
    ld[3, 0], ld[7, 1], ld[8, 0] = -np.inf, torch.finfo(torch.float32).min, -1000.0
    ld[10:14] = 0.0
    ld[400:, 1] = -30.0
    x["beta"][5], x["beta"][6] = 0.0, 1.0
    check(x, *kda.kda_gdn_prefill(**x))


@pytest.mark.parametrize("Hk,Hv", [(1, 2), (16, 32)])
def test_prefill_keeps_a_bad_sequence_to_itself(Hk, Hv):
    """A sequence of NaNs leaves its neighbours' outputs and states as they are without it."""
    x = inputs([70, 100, 61, 33], Hk, Hv, seed=83)
    o, S = kda.kda_gdn_prefill(**x)
    for n in ("q", "k", "v", "log_decay", "beta"):
        x[n][70:170] = float("nan")
    o2, S2 = kda.kda_gdn_prefill(**x)
    keep = [0, 2, 3]
    assert torch.equal(S[keep], S2[keep]) and torch.equal(o[:70], o2[:70]) and torch.equal(o[170:], o2[170:])
    assert bool(S2[1].isnan().any()) and bool(o2[70:170].isnan().any())


@pytest.mark.parametrize("cu", [[0, 50, 40, 100], [0, 30, 60, 99], [1, 30, 60, 100], [0, -5, 60, 100], [0, 30, 200, 100]])
def test_prefill_many_pairs_bad_cu_seqlens(cu):
    x = inputs([30, 30, 40], 16, 32, seed=84)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    guard = torch.full((120, 32, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    x["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    kda.kda_gdn_prefill(**x, o=guard[:100], device_status=status)
    assert int(status.item()) == kda.KDA_DEV_BAD_CU_SEQLENS
    assert bool((guard[100:] == 7.0).all())


@pytest.mark.parametrize("Hv", [2, 80])
@pytest.mark.parametrize("cu", [[0, 99], [1, 100], [0, 101], [0, -1], [-1, 100]])
def test_prefill_one_sequence_bad_cu_seqlens(cu, Hv):
    x = inputs([100], Hv, Hv, seed=85)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    guard = torch.full((120, Hv, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    x["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    kda.kda_gdn_prefill(**x, o=guard[:100], device_status=status)
    assert int(status.item()) == kda.KDA_DEV_BAD_CU_SEQLENS
    assert bool((guard[100:] == 7.0).all())


def test_prefill_many_pairs_on_two_streams():
    a, b = inputs([300, 100], 24, 48, seed=86), inputs([130, 64, 77], 16, 32, seed=87)
    ra, rb = kda.kda_gdn_prefill(**a), kda.kda_gdn_prefill(**b)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        got.append((kda.kda_gdn_prefill(**a, stream=one), kda.kda_gdn_prefill(**b, stream=two)))
    torch.cuda.synchronize()
    for ga, gb in got:
        assert torch.equal(ga[0], ra[0]) and torch.equal(ga[1], ra[1]) and torch.equal(gb[0], rb[0]) and torch.equal(gb[1], rb[1])


# ---------------------------------------------------------------- refusals ----
def wrong(t):
    """What a tensor argument must not be: another type, shape, place or layout, or no tensor."""
    spread = torch.empty(tuple(t.shape) + (2,), dtype=t.dtype, device="cuda")[..., 0]
    return [(t.to(torch.float64), TypeError), (t[..., :-1].contiguous(), ValueError), (t.cpu(), ValueError),
            (spread, ValueError), (t.tolist(), TypeError)]


def test_prefill_refuses_tensors():
    x = inputs([40, 24], 2, 4, seed=71)
    for name in x:
        for bad, error in wrong(x[name]):
            if name == "q" and error is ValueError and bad.is_cuda and bad.is_contiguous():
                continue  # a q of another shape: the others are the wrong ones then
            if name == "cu_seqlens" and error is ValueError and bad.is_cuda and bad.is_contiguous():
                continue  # one sequence fewer: S0 is the wrong one
            with pytest.raises((error, ValueError) if name in ("v", "q") else error):
                kda.kda_gdn_prefill(**dict(x, **{name: bad}))
    for name, like in (("o", x["v"]), ("S_final", x["S0"])):
        for bad, error in wrong(like):
            with pytest.raises(error):
                kda.kda_gdn_prefill(**x, **{name: bad})
    with pytest.raises(kda.KdaError):
        kda.kda_gdn_prefill(**x, workspace=torch.empty(100, dtype=torch.uint8, device="cuda"))
    with pytest.raises(kda.KdaError):
        kda.kda_gdn_prefill(**x, o=x["v"])


def test_decode_refuses_tensors():
    x = inputs([1] * 3, 2, 4, seed=72)
    args = dict({n: x[n] for n in ("q", "k", "v", "log_decay", "beta")}, S=x["S0"],
                state_indices=torch.tensor([2, 0, 1], dtype=torch.int32, device="cuda"), o=torch.empty_like(x["v"]))
    for name in args:
        for bad, error in wrong(args[name]):
            if name == "q" and error is ValueError and bad.is_cuda and bad.is_contiguous():
                continue
            with pytest.raises((error, ValueError) if name in ("v", "q") else error):
                kda.kda_gdn_decode_step(**dict(args, **{name: bad}))
    with pytest.raises(kda.KdaError):  # more sequences than slots
        kda.kda_gdn_decode_step(**dict(args, S=x["S0"][:2], state_indices=None))


# ------------------------------------------------- the choice of the path ----
@pytest.mark.parametrize("lengths", [[16], [17], [8] * 5, [8] * 4 + [9], [1] * 40 + [300], [1] * 63 + [441], [0] * 9 + [64, 3]])
def test_prefill_around_the_choice_of_the_path(lengths):
    x = inputs(lengths, 2, 4, seed=74 + len(lengths))
    check(x, *kda.kda_gdn_prefill(**x))


def test_prefill_many_pairs_under_a_graph():
    x = with_same(inputs([300, 0, 65], 16, 32, seed=88))
    o, S = kda.kda_gdn_prefill(**x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2, S2 = kda.kda_gdn_prefill(**x)
        o3, S3 = kda.kda_gdn_prefill(**dict(x, S0=S2))  # one after the other, in the workspace that the first gave back
    o2.zero_()
    S2.zero_()
    for _ in range(3):
        graph.replay()
    assert torch.equal(o, o2) and torch.equal(S, S2)
    o4, S4 = kda.kda_gdn_prefill(**dict(x, S0=S))
    assert torch.equal(o4, o3) and torch.equal(S4, S3)


def with_same(x):
    return {n: t.clone() for n, t in x.items()}


def test_prefill_many_pairs_slow_decay_over_many_chunks():
    x = inputs([2048], 40, 80, lo=-1e-4, seed=89)
    check(x, *kda.kda_gdn_prefill(**x))


def test_prefill_many_pairs_similar_keys():
    x = inputs([320, 130], 20, 40, seed=90, lo=-0.02)
    k = x["k"].float() + 0.5 / 128 ** 0.5 * 4
    x["k"] = (k / k.norm(dim=-1, keepdim=True)).to(torch.bfloat16)
    check(x, *kda.kda_gdn_prefill(**x))


@pytest.mark.parametrize("lengths,Hk,Hv", [([70, 100, 200], 1, 2), ([70, 100, 200], 16, 32), ([70], 1, 2), ([5, 6], 1, 2)])
def test_prefill_with_a_workspace_of_nans(lengths, Hk, Hv):
    """Nothing that the call has not written itself reaches a result."""
    x = inputs(lengths, Hk, Hv, seed=98)
    need = kda.kda_gdn_prefill_workspace_bytes(torch.bfloat16, len(lengths), sum(lengths), Hk, Hv)
    o, S = kda.kda_gdn_prefill(**x, workspace=torch.full((need,), 255, dtype=torch.uint8, device="cuda"))
    o2, S2 = kda.kda_gdn_prefill(**x, workspace=torch.zeros(need, dtype=torch.uint8, device="cuda"))
    assert torch.equal(o, o2) and torch.equal(S, S2)
    check(x, o, S)


@pytest.mark.parametrize("lengths,Hk,Hv", [([0] * 40 + [257] + [0] * 30, 1, 2), ([0] * 40 + [258] + [0] * 30, 1, 2), ([4] * 60, 2, 4),
                                           ([1] * 255 + [250], 2, 4), ([1] * 29 + [211], 16, 32), ([1] * 29 + [212], 16, 32)])
def test_prefill_around_the_most_tokens_of_short_sequences(lengths, Hk, Hv):
    x = inputs(lengths, Hk, Hv, seed=106 + sum(lengths))
    check(x, *kda.kda_gdn_prefill(**x))


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("name", ["q", "k", "v", "log_decay", "beta"])
@pytest.mark.parametrize("lengths,Hk,Hv,exact", [([30, 130, 40], 1, 2, False), ([30, 130, 40], 16, 32, False), ([3, 2, 2], 1, 2, True)])
def test_prefill_how_far_back_a_bad_token_reaches(lengths, Hk, Hv, exact, name, value):
    """Not before the 16 tokens of its sequence that it is among (before itself where the call goes token by token)."""
    x = inputs(lengths, Hk, Hv, seed=108)
    o, S = kda.kda_gdn_prefill(**x)
    start, end = lengths[0], lengths[0] + lengths[1]
    bad = start + (1 if exact else 64 + 37)
    first = bad if exact else start + 64 + 32
    y = {n: t.clone() for n, t in x.items()}
    y[name][bad] = value
    o2, S2 = kda.kda_gdn_prefill(**y)
    assert torch.equal(o[:first], o2[:first]) and torch.equal(o[end:], o2[end:])
    assert torch.equal(S[[0, 2]], S2[[0, 2]])
    assert not bool(o2[bad].isfinite().all())
