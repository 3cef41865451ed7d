"""Gradient of the gated delta rule on the GPU against the fp64 oracle's (the KDA gradient with the decay
broadcast: its log_alpha gradient summed over channels, q and k gradients summed over a group's heads).

Tolerances.  A product has at most two operands in two bf16 terms, each off by at most 2^-17 of the value; ten
products at most lie between an input and a gradient (K S, T R, K^T U, K X, T^T dU, Q^T dO, K^T W and the three
of the last step): 20 x 2^-17, spread evenly to F32 = 20 x 2^-17 / sqrt(3) of the 2-norm of what they make, the
states S and their adjoints G among it.  grad_S0 is held to that.  grad_log_decay = <G, S> and grad_beta =
(G^T k) . e are inner products whose terms cancel: an error of F32 |G| in G has no preferred direction among its
128 x 128, and is felt in them as F32 |G| |S| / 128 (F32 |G| |e| / 128, F32 |S| |G^T k| / 128) in the mean; 8 times
that is allowed.  bf16 gradients are rounded once (2^-8 of the value) and take M and E, rounded once too, into q's
and k's: 2 x 2^-8 / sqrt(3) of the 2-norm, twice that where terms cancel.
"""
import numpy as np
import pytest
import torch

import linear_attention_chunkwise_gb300 as kda
import oracle
from tests.conftest import cuda_ok
from tests.gpu_util import host
from tests.test_gpu_gdn import inputs, wrong

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

F32 = 20 * 2.0 ** -17 / 3 ** 0.5
BF16 = 4 * 2.0 ** -8 / 3 ** 0.5
NAMES = ("q", "k", "v", "log_decay", "beta", "S0")


def with_grads(x, seed=0, final=True):
    g = torch.Generator("cuda").manual_seed(1000 + seed)
    dO = torch.randn(x["v"].shape, generator=g, device="cuda").to(x["v"].dtype)
    N = x["cu_seqlens"].numel() - 1
    dS = torch.randn(N, x["v"].shape[1], 128, 128, generator=g, device="cuda") * 0.1 if final else None
    return dict(x, grad_o=dO, grad_S_final=dS)


def reference(x):
    Hk, Hv = x["q"].shape[1], x["v"].shape[1]
    m = Hv // Hk
    rep = lambda t: host(t.repeat_interleave(m, 1))  # noqa: E731
    la = np.repeat(host(x["log_decay"])[:, :, None], 128, 2)
    dq, dk, dv, dla, db, dS0 = oracle.kda_prefill_backward(rep(x["q"]), rep(x["k"]), host(x["v"]), la, host(x["beta"]),
                                                           x["cu_seqlens"].cpu().numpy(), host(x["S0"]),
                                                           host(x["grad_o"]), host(x["grad_S_final"]))
    shared = lambda a: a.reshape(a.shape[0], Hk, m, 128).sum(2)  # noqa: E731
    return shared(dq), shared(dk), dv, dla.sum(-1), db, dS0


def sizes(x):
    """|G| |S| / 128 and (|G| |e| + |S| |G^T k|) / 128 of every token and head, in a walk of its own (64 bits)."""
    m = x["v"].shape[1] // x["q"].shape[1]
    q, k = (x[n].double().repeat_interleave(m, 1) for n in ("q", "k"))
    v, dO, beta, a = x["v"].double(), x["grad_o"].double(), x["beta"].double(), x["log_decay"].double().exp()
    cu = x["cu_seqlens"].tolist()
    ld, db = torch.zeros_like(beta), torch.zeros_like(beta)
    for n in range(len(cu) - 1):
        S = torch.zeros(v.shape[1], 128, 128, dtype=torch.float64, device="cuda") if x["S0"] is None else x["S0"][n].double()
        G = torch.zeros_like(S) if x["grad_S_final"] is None else x["grad_S_final"][n].double()
        before = []
        for t in range(cu[n], cu[n + 1]):
            S = S * a[t][:, None, None]
            before.append(S)
            e = v[t] - (k[t][:, None] @ S)[:, 0]
            S = S + k[t][:, :, None] * (beta[t][:, None] * e)[:, None]
        for t in reversed(range(cu[n], cu[n + 1])):
            S = before[t - cu[n]]
            G = G + q[t][:, :, None] * dO[t][:, None]
            gk, e = (k[t][:, None] @ G)[:, 0], v[t] - (k[t][:, None] @ S)[:, 0]
            db[t] = G.norm(dim=(1, 2)) * e.norm(dim=1) + S.norm(dim=(1, 2)) * gk.norm(dim=1)
            G = G - k[t][:, :, None] * (beta[t][:, None] * gk)[:, None]
            ld[t] = G.norm(dim=(1, 2)) * S.norm(dim=(1, 2))
            G = G * a[t][:, None, None]
    return dict(log_decay=ld.cpu().numpy() / 128, beta=db.cpu().numpy() / 128)


def check(x, grads, ref=None):
    size = sizes(x)
    for name, got, want in zip(NAMES, grads, ref or reference(x)):
        if got is None:
            continue
        far = host(got).astype(np.float64) - want
        if name in size:
            assert np.all(np.abs(far) <= F32 * (8 * size[name] + np.abs(want)) + 1e-30), (name, np.abs(far).max())
        else:
            bound = (F32 if got.dtype == torch.float32 else BF16) * np.linalg.norm(want)
            assert np.linalg.norm(far) <= bound, (name, np.linalg.norm(far) / max(np.linalg.norm(want), 1e-300))


CASES = [([1], 1, 1), ([2], 2, 4), ([63], 1, 3), ([64], 2, 2), ([65], 1, 2), ([16, 17, 15], 2, 2), ([128, 0, 1, 200], 2, 4),
         ([300, 77, 0, 0, 640, 129], 3, 6), ([1500], 2, 2), ([700, 64, 1], 1, 4), ([130] * 12, 8, 8)]


@pytest.mark.parametrize("lengths,Hk,Hv", CASES)
def test_backward(lengths, Hk, Hv):
    x = with_grads(inputs(lengths, Hk, Hv, seed=61 + sum(lengths)))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    grads = kda.kda_gdn_prefill_backward(**x, device_status=status)
    assert int(status.item()) == 0
    check(x, grads)


@pytest.mark.parametrize("lengths", [[5], [400]])
def test_backward_without_states(lengths):
    x = with_grads(inputs(lengths, 2, 4, start=False, seed=62), final=False)
    grads = kda.kda_gdn_prefill_backward(**x)
    check(x, grads)
    again = kda.kda_gdn_prefill_backward(**x, need_grad_S0=False)
    assert again[5] is None and all(torch.equal(a, b) for a, b in zip(grads[:5], again[:5]))


def test_backward_extreme_decays_and_betas():
    x = inputs([150, 40], 2, 2, seed=63)
    ld = x["log_decay"]
    ld[3, 0], ld[7, 1], ld[8, 0], ld[70, 1] = -np.inf, torch.finfo(torch.float32).min, -1000.0, -np.inf
    ld[10:14] = 0.0
    x["beta"][5], x["beta"][6], x["beta"][66], x["beta"][67] = 0.0, 1.0, 1e-30, -0.5
    x = with_grads(x)
    grads = kda.kda_gdn_prefill_backward(**x)
    y = dict(x, log_decay=ld.clamp_min(-1000.0))  # a decay of 0 in fp64 as well
    check(x, grads, reference(y))


def test_backward_similar_keys_and_slow_decay():
    x = inputs([640], 1, 2, seed=64, lo=-0.02)
    k = x["k"].float() + 2.0 / 128 ** 0.5
    x["k"] = (k / k.norm(dim=-1, keepdim=True)).to(torch.bfloat16)
    x = with_grads(x)
    check(x, kda.kda_gdn_prefill_backward(**x))


def test_backward_rows_of_other_sequences_do_not_matter():
    """NaN in one sequence stays there; rows behind the gradients' end are left as they were."""
    x = with_grads(inputs([70, 90, 33], 1, 2, seed=65))
    clean = kda.kda_gdn_prefill_backward(**x)
    y = {n: t.clone() for n, t in x.items()}
    for n in ("q", "k", "v", "grad_o"):
        y[n][70:160] = float("nan")
    bufs = [torch.full((200,) + tuple(t.shape[1:]), 5.0, dtype=t.dtype, device="cuda") for t in clean[:5]]
    grads = kda.kda_gdn_prefill_backward(**y, grads=tuple(b[:193] for b in bufs) + (torch.empty_like(clean[5]),))
    for a, b in zip(clean[:5], grads[:5]):
        assert torch.equal(a[:70], b[:70]) and torch.equal(a[160:], b[160:])
    assert torch.equal(clean[5][[0, 2]], grads[5][[0, 2]])
    assert all(bool((b[193:] == 5.0).all()) for b in bufs)


def test_backward_no_tokens():
    x = with_grads(inputs([0, 0], 1, 2, seed=66))
    grads = kda.kda_gdn_prefill_backward(**x)
    assert torch.equal(grads[5], x["grad_S_final"])


def test_backward_captured_and_repeatable():
    x = with_grads(inputs([200, 90], 2, 4, seed=67))
    want = kda.kda_gdn_prefill_backward(**x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = kda.kda_gdn_prefill_backward(**x)
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(want, got))


def test_backward_is_the_forwards_slope():
    """Differences of the forward's fp32 final state along a direction of log_decay, beta and S0 together."""
    x = inputs([90], 1, 1, seed=68)
    g = torch.Generator("cuda").manual_seed(3)
    dS = torch.randn(1, 1, 128, 128, generator=g, device="cuda")
    dirs = {n: torch.randn(x[n].shape, generator=g, device="cuda") * s for n, s in (("log_decay", 0.05), ("beta", 0.05), ("S0", 0.1))}
    grads = dict(zip(NAMES, kda.kda_gdn_prefill_backward(**x, grad_o=torch.zeros_like(x["v"]), grad_S_final=dS)))
    slope = sum(float((grads[n].double() * d.double()).sum()) for n, d in dirs.items())
    size = sum(float((grads[n].double() * d.double()).abs().sum()) for n, d in dirs.items())

    def loss(step):
        _, S = kda.kda_gdn_prefill(**{n: t + step * dirs[n] if n in dirs else t for n, t in x.items()})
        return float((S.double() * dS.double()).sum())

    # step 2^-6: truncation step^2 / 6 of the third derivative (log-decays and betas of 0.05 a step: below
    # 1e-4 of the terms' size), rounding 2^-17 of |S||dS| over 2^-5
    step = 2.0 ** -6
    noise = 2.0 ** -12 * float(dS.double().norm()) * float(kda.kda_gdn_prefill(**x)[1].double().norm())
    assert abs((loss(step) - loss(-step)) / (2 * step) - slope) <= 1e-3 * size + noise
    assert abs(slope) > 10 * (1e-3 * size + noise)


@pytest.mark.parametrize("lengths,Hk,Hv", [([1 + (37 * i) % 131 for i in range(40)], 4, 8), ([0, 65, 1, 200, 0, 64, 640, 90], 12, 36)])
def test_backward_more_chunks_than_sms(lengths, Hk, Hv):
    """A thread block goes over several chunks of several sequences, full ones and others, with two or three heads each."""
    x = with_grads(inputs(lengths, Hk, Hv, seed=91 + Hk))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    grads = kda.kda_gdn_prefill_backward(**x, device_status=status)
    assert int(status.item()) == 0
    check(x, grads)


def test_backward_refuses_tensors():
    x = with_grads(inputs([40, 24], 2, 4, seed=73))
    for name in ("k", "v", "log_decay", "beta", "grad_o", "S0", "grad_S_final"):
        for bad, error in wrong(x[name]):
            with pytest.raises((error, ValueError) if name == "v" else error):
                kda.kda_gdn_prefill_backward(**dict(x, **{name: bad}))
    y = with_grads(inputs([40, 24], 2, 4, dtype=torch.float32, seed=73))
    with pytest.raises(kda.KdaError):
        kda.kda_gdn_prefill_backward(**y)
    with pytest.raises(ValueError):
        kda.kda_gdn_prefill_backward(**x, grads=(None,) * 5)
    with pytest.raises(TypeError):
        kda.kda_gdn_prefill_backward(**x, grads=(None,) * 6)
    with pytest.raises(kda.KdaError):
        kda.kda_gdn_prefill_backward(**x, workspace=torch.empty(4096, dtype=torch.uint8, device="cuda"))
    like = [torch.empty_like(x[n]) for n in ("q", "k", "v", "log_decay", "beta", "S0")]
    with pytest.raises(kda.KdaError):  # a gradient over an input
        kda.kda_gdn_prefill_backward(**x, grads=(x["q"], *like[1:]))


@pytest.mark.parametrize("lengths,Hk,Hv", [([130, 0, 64], 1, 8), ([200], 2, 16), ([65, 3], 4, 16), ([90], 9, 18), ([64] * 9, 4, 8)])
def test_backward_groups_on_few_sms(lengths, Hk, Hv):
    """Groups of two, four and eight value heads with an SM for each, and (the last) without."""
    x = with_grads(inputs(lengths, Hk, Hv, seed=92 + Hv))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    grads = kda.kda_gdn_prefill_backward(**x, device_status=status)
    assert int(status.item()) == 0
    check(x, grads)
    again = kda.kda_gdn_prefill_backward(**x)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


# Up to two tokens a sequence and six more go token by token in fp32.  An error of a value here is some roundings, 2^-24 of what it adds up, of
# which `sizes` bounds the largest part; bf16 gradients are rounded once.
SHORT = 64 * 2.0 ** -24


@pytest.mark.parametrize("lengths,Hk,Hv", [([1], 1, 1), ([1], 2, 8), ([0, 1, 0], 1, 1), ([16], 1, 3), ([3, 0, 4, 5], 2, 4), ([1] * 40, 2, 2),
                                           ([2, 5], 4, 16)])
def test_backward_of_few_tokens(lengths, Hk, Hv):
    x = with_grads(inputs(lengths, Hk, Hv, seed=93 + len(lengths)))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    grads = kda.kda_gdn_prefill_backward(**x, device_status=status)
    assert int(status.item()) == 0
    size, ref = sizes(x), reference(x)
    few = sum(lengths) <= 2 * len(lengths) + 6  # more go in chunks, with their tolerances
    for name, got, want in zip(NAMES, grads, ref) if few else ():
        far = np.abs(host(got).astype(np.float64) - want)
        top = np.abs(want).max(initial=0.0)
        if name in size:
            assert np.all(far <= SHORT * (128 * size[name] + np.abs(want)) + 1e-30), (name, far.max())
        elif got.dtype == torch.float32:
            assert np.all(far <= SHORT * top + 1e-30), name
        else:
            assert np.all(far <= 2.0 ** -8 * np.abs(want) * (1 + SHORT) + 16 * SHORT * top + 1e-30), name
    check(x, grads, ref)
    again = kda.kda_gdn_prefill_backward(**x)
    assert all(torch.equal(a, b) for a, b in zip(grads, again))


def test_backward_of_few_tokens_extreme_decays():
    x = with_grads(inputs([10], 2, 4, seed=94))
    x["log_decay"][3, 0], x["log_decay"][7, 1], x["log_decay"][5, 2] = -np.inf, torch.finfo(torch.float32).min, 0.0
    x["beta"][5], x["beta"][6] = 0.0, 1.0
    grads = kda.kda_gdn_prefill_backward(**x)
    check(x, grads)
    assert float(grads[3][3, 0]) == 0.0 and float(grads[3][7, 1]) == 0.0


@pytest.mark.parametrize("cu", [[0, 2, 1, 5], [0, 1, 2, 4], [1, 2, 3, 5], [0, -5, 3, 5], [0, 3, 20, 5]])
def test_backward_of_few_tokens_bad_cu_seqlens(cu):
    x = with_grads(inputs([2, 1, 2], 1, 2, seed=95))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    x["cu_seqlens"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    guard = torch.full((40, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    like = [torch.empty_like(x[n]) for n in ("q", "k", "v", "log_decay", "beta", "S0")]
    kda.kda_gdn_prefill_backward(**x, grads=(*like[:2], guard[:5], *like[3:]), device_status=status)
    assert int(status.item()) == kda.KDA_DEV_BAD_CU_SEQLENS
    assert bool((guard[5:] == 7.0).all())


@pytest.mark.parametrize("lengths,Hk,Hv", [([3, 2], 2, 4), ([70, 40], 2, 4)])
def test_backward_replayed_and_on_streams(lengths, Hk, Hv):
    x, y = (with_grads(inputs(lengths, Hk, Hv, seed=s)) for s in (96, 97))
    want, other = kda.kda_gdn_prefill_backward(**x), kda.kda_gdn_prefill_backward(**y)
    one, two = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [(kda.kda_gdn_prefill_backward(**x, stream=one), kda.kda_gdn_prefill_backward(**y, stream=two)) for _ in range(5)]
    torch.cuda.synchronize()
    for a, b in got:
        assert all(torch.equal(g, w) for g, w in zip(a, want)) and all(torch.equal(g, w) for g, w in zip(b, other))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first = kda.kda_gdn_prefill_backward(**x)
        second = kda.kda_gdn_prefill_backward(**y)
    for t in (*first, *second):
        t.zero_()
    for _ in range(3):
        graph.replay()
    assert all(torch.equal(g, w) for g, w in zip(first, want)) and all(torch.equal(g, w) for g, w in zip(second, other))


@pytest.mark.parametrize("lengths,Hk,Hv", [([3, 2], 2, 4), ([70, 100], 2, 4), ([70, 100, 65], 16, 32)])
def test_backward_with_a_workspace_of_nans(lengths, Hk, Hv):
    x = with_grads(inputs(lengths, Hk, Hv, seed=99))
    need = kda.kda_gdn_prefill_backward_workspace_bytes(torch.bfloat16, len(lengths), sum(lengths), Hk, Hv)
    got = kda.kda_gdn_prefill_backward(**x, workspace=torch.full((need,), 255, dtype=torch.uint8, device="cuda"))
    check(x, got)
    again = kda.kda_gdn_prefill_backward(**x, workspace=torch.zeros(need, dtype=torch.uint8, device="cuda"))
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("lengths,Hk,Hv", [([1] * 64 + [65], 2, 4), ([0] * 40 + [70] + [0] * 20, 2, 4), ([0] * 49 + [66], 1, 1),
                                           ([0] * 49 + [67], 1, 1), ([1] * 71, 2, 2), ([1] * 72, 2, 2), ([1] * 50 + [2] * 10, 16, 32)])
def test_backward_around_the_choice_of_the_path(lengths, Hk, Hv):
    x = with_grads(inputs(lengths, Hk, Hv, seed=105 + len(lengths)))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    grads = kda.kda_gdn_prefill_backward(**x, device_status=status)
    assert int(status.item()) == 0
    check(x, grads)


def test_one_workspace_for_smaller_calls():
    Hk, Hv = 2, 4
    fwd = torch.empty(kda.kda_gdn_prefill_workspace_bytes(torch.bfloat16, 40, 64, Hk, Hv), dtype=torch.uint8, device="cuda")
    back = torch.empty(kda.kda_gdn_prefill_backward_workspace_bytes(torch.bfloat16, 40, 64, Hk, Hv), dtype=torch.uint8, device="cuda")
    for lengths in ([1] * 40, [64], [7], [8], [1, 63], [0] * 30 + [34], [2] * 8, [0, 0]):
        x = inputs(lengths, Hk, Hv, seed=107 + len(lengths))
        g = with_grads(x)
        for a, b in ((kda.kda_gdn_prefill(**x), kda.kda_gdn_prefill(**x, workspace=fwd)),
                     (kda.kda_gdn_prefill_backward(**g), kda.kda_gdn_prefill_backward(**g, workspace=back))):
            assert all(torch.equal(s, t) for s, t in zip(a, b))
