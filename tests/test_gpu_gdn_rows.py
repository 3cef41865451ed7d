"""The chunkwise gated delta rule value by value: o and the bf16 gradients, each element against a bound of its own.

Tolerances.  h = 2^-8 is half a step of bf16, the most that a rounding takes a value from itself, relative to it.
With a chunk's start state S, U, P, W, X, M and E of the formulas (those of kda_gdn_prefill.cu and kda_gdn_backward.cu):
  o = e^g q S + P U takes S, P and U rounded to bf16 and is rounded: h e^g |q| |S| + (2 h + h^2) |P| |U|, and h |o|.
      P's products q . k are sums of 128 in fp32, off by 128 x 2^-24 |q| . |k|, whatever is left of them.
  dq = e^g dO S^T + M K,  dk = -e^g b W S^T + e^(gC - g) U X^T + M^T Q + (E + E^T) K take M and E rounded, and are
      rounded: h |M| |K|, h (|M|^T |Q| + (|E| + |E|^T) |K|), and h of the value; dv = b W is rounded only.
Everything else is fp32 or in two bf16 terms: for o at most STATE of the largest entry of S and of U (as the states are
held to it), for the gradients at most F32 of the norms of S, X, U and W (as the gradients of the gates are).
"""
import numpy as np
import pytest
import torch

import linear_attention_chunkwise_gb300 as kda
from tests.conftest import cuda_ok
from tests.gpu_util import host
from tests.test_gpu_gdn import STATE, inputs, reference
from tests.test_gpu_gdn_backward import F32, with_grads
from tests.test_gpu_gdn_backward import reference as reference_grads

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

H = 2.0 ** -8


def _heads(x):
    m = x["v"].shape[1] // x["q"].shape[1]
    q, k = (x[n].double().repeat_interleave(m, 1) for n in ("q", "k"))
    return m, q, k, x["v"].double(), x["beta"].double(), x["log_decay"].double()


def _chunks(x):
    cu = x["cu_seqlens"].tolist()
    for n in range(len(cu) - 1):
        S = torch.zeros(x["v"].shape[1], 128, 128, dtype=torch.float64, device="cuda") if x["S0"] is None else x["S0"][n].double()
        yield n, [(t, min(t + 64, cu[n + 1])) for t in range(cu[n], cu[n + 1], 64)], S


def _decays(ld):  # [L, Hv] -> e^g, e^(gC - g), and e^(g_i - g_j) for i >= j [Hv, L, L]
    g = ld.cumsum(0)
    d = (g.T[:, :, None] - g.T[:, None, :]).tril()
    return g.exp(), (g[-1] - g).exp(), d.exp().tril()


def bound_o(x, ref):
    _, q, k, v, b, ld = _heads(x)
    out = torch.zeros_like(v)
    for _, chunks, S in _chunks(x):
        for lo, hi in chunks:
            s = slice(lo, hi)
            start, u = S, []
            for t in range(lo, hi):
                S = S * ld[t].exp()[:, None, None]
                u.append(b[t][:, None] * (v[t] - (k[t][:, None] @ S)[:, 0]))
                S = S + k[t][:, :, None] * u[-1][:, None]
            u = torch.stack(u)
            eg, _, G = _decays(ld[s])
            P = G * torch.einsum("ihc,jhc->hij", q[s], k[s])
            qs = eg[:, :, None] * torch.einsum("ihc,hcv->ihv", q[s].abs(), start.abs())
            pu = torch.einsum("hij,jhv->ihv", P.abs(), u.abs())
            gram = torch.einsum("hij,jhv->ihv", G * torch.einsum("ihc,jhc->hij", q[s].abs(), k[s].abs()), u.abs())
            rest = eg * q[s].abs().sum(-1) * start.abs().amax((1, 2)) + P.abs().sum(-1).T * u.abs().amax((0, 2))
            out[s] = (1 + H) * (H * qs + (2 * H + H * H) * pu + 2.0 ** -17 * gram + STATE * rest[:, :, None])
    return out.cpu().numpy() + H * np.abs(ref)


def bounds_grad(x, refs):
    m, q, k, v, b, ld = _heads(x)
    dO = x["grad_o"].double()
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    norm = lambda t: t.flatten(-2).norm(dim=-1) if t.dim() == 3 and t.shape[-2] == 128 else t.norm(dim=-1)  # noqa: E731
    for n, chunks, S in _chunks(x):
        states, us, starts = {}, {}, []
        for lo, hi in chunks:
            starts.append(S)
            for t in range(lo, hi):
                S = S * ld[t].exp()[:, None, None]
                us[t] = b[t][:, None] * (v[t] - (k[t][:, None] @ S)[:, 0])
                S = S + k[t][:, :, None] * us[t][:, None]
        X = torch.zeros_like(S) if x["grad_S_final"] is None else x["grad_S_final"][n].double()
        for (lo, hi), S in zip(reversed(chunks), reversed(starts)):
            s, end, w = slice(lo, hi), X, {}
            for t in reversed(range(lo, hi)):
                X = X + q[t][:, :, None] * dO[t][:, None]
                w[t] = (k[t][:, None] @ X)[:, 0]
                X = (X - k[t][:, :, None] * (b[t][:, None] * w[t])[:, None]) * ld[t].exp()[:, None, None]
            U, W = torch.stack([us[t] for t in range(lo, hi)]), torch.stack([w[t] for t in range(lo, hi)])
            eg, eo, G = _decays(ld[s])
            M = (G * torch.einsum("ihv,jhv->hij", dO[s], U)).abs()
            E = (b[s].T[:, :, None] * (G * torch.einsum("ihv,jhv->hij", W, U)).tril(-1)).abs()
            nS, nX, nU, nW, nO = norm(S), norm(end), U.norm(dim=-1).amax(0), W.norm(dim=-1).amax(0), dO[s].norm(dim=-1)
            M = H * M + F32 * G * (nO * nU).T[:, :, None]
            E = H * E + 2 * F32 * b[s].T.abs()[:, :, None] * G.tril(-1) * (nW * nU)[:, None, None]
            aq, ak = q[s].abs(), k[s].abs()
            dq[s] = torch.einsum("hij,jhc->ihc", M, ak) + F32 * (eg * nO * nS)[:, :, None]
            dk[s] = (torch.einsum("hij,ihc->jhc", M, aq) + torch.einsum("hij,jhc->ihc", E, ak) + torch.einsum("hij,ihc->jhc", E, ak)
                     + 2 * F32 * (eg * b[s].abs() * nW * nS + eo * nU * nX)[:, :, None])
            dv[s] = F32 * (b[s].abs() * nW)[:, :, None]
    shared = lambda t: t.view(t.shape[0], -1, m, 128).sum(2)  # noqa: E731
    return [(1 + H) * t.cpu().numpy() + H * np.abs(r) for t, r in zip((shared(dq), shared(dk), dv), refs)]


def within(got, ref, bound):
    far = np.abs(host(got).astype(np.float64) - ref)
    assert np.all(far <= bound), (np.argwhere(far > bound)[:5].tolist(), (far / bound).max())


def refused(got, ref, bound_of):
    """What a mistake in one row would look like: the check has to tell it from the right one."""
    T, heads, _ = ref.shape
    rows = [(0, 0), (T - 1, heads - 1), (T // 2, heads // 2)]
    for t, h in rows:
        other = (t + 1) % T if T > 1 else None
        for wrong in (np.zeros(128), 0.7 * ref[t, h], *([ref[other, h]] if other is not None else [])):
            bad = ref.copy()
            bad[t, h] = wrong
            with pytest.raises(AssertionError):
                within(got, bad, bound_of(bad))


CASES = [([17], 1, 2), ([63, 65], 2, 4), ([300, 77, 0, 0, 330, 129], 3, 6), ([257, 40], 24, 48), ([1 + (37 * i) % 131 for i in range(20)], 2, 4),
         ([64] * 20, 4, 4), ([200, 0, 130], 16, 32)]


@pytest.mark.parametrize("lengths,Hk,Hv", CASES)
def test_every_output(lengths, Hk, Hv):
    x = inputs(lengths, Hk, Hv, seed=301 + sum(lengths))
    o, _ = kda.kda_gdn_prefill(**x)
    ref, _ = reference(x)
    rest = bound_o(x, ref) - H * np.abs(ref)
    within(o, ref, rest + H * np.abs(ref))
    refused(o, ref, lambda r: rest + H * np.abs(r))


@pytest.mark.parametrize("lengths,Hk,Hv", CASES[:3] + [([90, 65, 1], 12, 36), ([130] * 5, 8, 8), ([200], 2, 16), ([64, 1, 63, 66], 1, 2)])
def test_every_gradient_of_q_k_and_v(lengths, Hk, Hv):
    x = with_grads(inputs(lengths, Hk, Hv, seed=302 + sum(lengths)))
    got = kda.kda_gdn_prefill_backward(**x)[:3]
    refs = reference_grads(x)[:3]
    for g, r, bound in zip(got, refs, bounds_grad(x, refs)):
        rest = bound - H * np.abs(r)
        within(g, r, bound)
        refused(g, r, lambda bad: rest + H * np.abs(bad))
