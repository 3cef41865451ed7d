"""The norm, the gated delta rule and its decode step as one layer runs them, forward and backward.

x + residual -> norm -> projections -> prefill -> output norm in 8 bits; the prompt's last tokens again by
decode steps; and the gradient from the output back to x and the norm's weight.  The oracle is the layer in
fp64 with autograd, which rounds nothing.

Tolerance.  Between its inputs and any result the layer rounds to bf16 at most ROUNDINGS times in a row: the
normed row, a projection, the unit keys and queries, four times in the prefill (the state and U as the output
takes them, P, o) and as often in its gradient, the projections' gradients, grad_y and grad_x.  Each is off by
at most half a step, 2^-8, of what it rounds and spread over it evenly, so that in the 2-norm it adds at
most 2^-8 / sqrt(3), and where it enters through a second path (q and k, v and the gates) twice that.  e4m3
adds half its step, 2^-4, to the values it stands for.
"""
import pytest
import torch

import linear_attention_chunkwise_gb300 as kda
from tests.conftest import cuda_ok

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

ROUNDINGS = 14
TOL = 2 * ROUNDINGS ** 0.5 * 2.0 ** -8 / 3 ** 0.5
DIM, HK, HV, D, EPS = 512, 2, 4, 128, 1e-6


def weights(seed):
    g = torch.Generator("cuda").manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    return dict(norm=1 + 0.2 * n(DIM), q=n(DIM, HK * D).bfloat16() / DIM ** 0.5, k=n(DIM, HK * D).bfloat16() / DIM ** 0.5,
                v=n(DIM, HV * D).bfloat16() / DIM ** 0.5, a=n(DIM, HV).bfloat16() / DIM ** 0.5, b=n(DIM, HV).bfloat16() / DIM ** 0.5)


def project(y, w):
    """q, k, v, log_decay, beta of normed rows y, in the type of y (the gates fp32 or wider)."""
    wide = torch.float64 if y.dtype == torch.float64 else torch.float32
    heads = lambda name, H: (y @ w[name].to(y.dtype)).view(-1, H, D)  # noqa: E731
    unit = lambda t: (t.to(wide) / t.to(wide).norm(dim=-1, keepdim=True)).to(y.dtype)  # noqa: E731
    gate = lambda name: torch.sigmoid((y @ w[name].to(y.dtype)).to(wide))  # noqa: E731
    return unit(heads("q", HK)), unit(heads("k", HK)), heads("v", HV), -0.2 * gate("a"), gate("b")


def oracle_layer(x, residual, w, lengths):
    h = x.double() + residual.double()
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * w["norm"].double()
    q, k, v, ld, be = project(y, w)
    q, k = q.repeat_interleave(HV // HK, 1), k.repeat_interleave(HV // HK, 1)
    o, states, at = [], [], 0
    for n in lengths:
        S = torch.zeros(HV, D, D, dtype=torch.float64, device="cuda")
        for t in range(at, at + n):
            S = S * ld[t].exp()[:, None, None]
            e = be[t][:, None] * (v[t] - torch.einsum("hk,hkv->hv", k[t], S))
            S = S + k[t][:, :, None] * e[:, None]
            o.append(torch.einsum("hk,hkv->hv", q[t], S))
        states.append(S)
        at += n
    return h, torch.stack(o), torch.stack(states)


def close(got, want, tol=TOL):
    far = float((got.detach().double() - want.detach()).norm() / want.detach().norm())
    assert far <= tol, (far, tol)


@pytest.mark.parametrize("lengths,steps", [([70], 3), ([130, 33, 64], 2)])
def test_a_layer(lengths, steps):
    w, T = weights(7), sum(lengths)
    g = torch.Generator("cuda").manual_seed(8 + T)
    x, residual = (torch.randn(T, DIM, generator=g, device="cuda").bfloat16() for _ in range(2))
    cu = torch.tensor([0] + list(torch.tensor(lengths).cumsum(0)), dtype=torch.int32, device="cuda")

    # the prompt, and the output as the next product would take it
    y, _, h = kda.kda_rms_norm(x, w["norm"], residual, eps=EPS)
    y.requires_grad_()
    ins = project(y, w)
    o, S = kda.kda_gdn_prefill(*(t.detach().contiguous() for t in ins), cu)
    rows = o.view(T, HV * D)
    codes, scales, _ = kda.kda_rms_norm(rows, eps=EPS, quant="e4m3", group=128)

    xr, wn = x.double().requires_grad_(), w["norm"].double().requires_grad_()
    h_ref, o_ref, S_ref = oracle_layer(xr, residual, dict(w, norm=wn), lengths)
    close(h, h_ref)
    close(o, o_ref)
    close(S, S_ref)
    flat = o_ref.detach().reshape(T, HV * D)
    normed = flat * torch.rsqrt(flat.square().mean(-1, keepdim=True) + EPS)
    close(codes.double().view(T, -1, 128) * scales.double()[:, :, None], normed.view(T, -1, 128), TOL + 2.0 ** -4)

    # the last tokens of every sequence again, one at a time, from the state of the rest
    keep = torch.cat([torch.arange(a, b - steps) for a, b in zip(cu.tolist(), cu.tolist()[1:])]).cuda()
    short = torch.tensor([0] + list((torch.tensor(lengths) - steps).cumsum(0)), dtype=torch.int32, device="cuda")
    _, S1 = kda.kda_gdn_prefill(*(t.detach()[keep].contiguous() for t in ins), short)
    for i in range(steps):
        at = cu[1:].long() - steps + i
        o1 = kda.kda_gdn_decode_step(*(t.detach()[at].contiguous() for t in ins), S1)
        close(o1, o_ref.detach()[at])
    close(S1, S_ref)

    # the gradient
    dO = torch.randn(T, HV, D, generator=g, device="cuda").bfloat16()
    dh = torch.randn(T, DIM, generator=g, device="cuda").bfloat16()
    dS = 0.1 * torch.randn(S.shape, generator=g, device="cuda")
    *grads, dS0 = kda.kda_gdn_prefill_backward(*(t.detach().contiguous() for t in ins), cu, dO, None, dS, need_grad_S0=False)
    assert dS0 is None
    dy, = torch.autograd.grad(ins, y, grads)
    dx, dw = kda.kda_rms_norm_backward(dy, h, w["norm"], grad_h=dh, eps=EPS)
    loss = (o_ref * dO.double()).sum() + (S_ref * dS.double()).sum() + (h_ref * dh.double()).sum()
    dx_ref, dw_ref = torch.autograd.grad(loss, (xr, wn))
    close(dx, dx_ref)
    close(dw, dw_ref)
