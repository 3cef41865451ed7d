"""Gates of the gated linear recurrence far from 0, element by element relative to their own values.

u = 2^-24.  e^g is good to 5 u (ex2.approx 4 u, the remainder's product 1 u), so c = 1 / (1 + e^g) to 5 + 1 + 2 = 8 u (the sum's
rounding, rcp.approx's 2^-23) and a (1 - a) = e^g c^2 to 5 + 2 * 8 + 2 = 23 u, whatever g.  Gates end where c or its slope leaves fp32's
normal range (87.3).
"""
import pytest
import torch

import linear_attention_chunkwise_gb300 as kda
from tests.conftest import cuda_ok
from tests.test_gpu_glr import BF, F32, U, close, cu_of, randn

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]

SIGMOID = dict(gate_kind="sigmoid", complement=True)


def spread(lo, hi, dim):
    """One gate a channel, evenly from lo to hi, and magnitudes from 1 to 2 to go with them."""
    gate = torch.linspace(lo, hi, dim, device="cuda", dtype=torch.float64).float()[None]
    return gate, (1 + torch.rand(1, dim, device="cuda", generator=torch.Generator("cuda").manual_seed(1))) * randn(1, dim, seed=2).sign()


def near(got, ref, steps):
    """Within `steps` u of the value and one rounding to the type of `got`."""
    close(got, ref, steps * U * ref.abs())


@pytest.mark.parametrize("types", [(F32, F32), (BF, F32)])
@pytest.mark.parametrize("dim", [4096, 4001])
def test_far_sigmoid_gates(dim, types):
    """One token: h = (1 - a) x, 8 u and the product's; the gradients are their formulas' factors."""
    gate, x = spread(-86.0, 86.0, dim)
    x, gate, h0 = x.to(types[0]), gate.to(types[1]), torch.zeros(1, dim, device="cuda")
    c, a = torch.sigmoid(-gate.double()), torch.sigmoid(gate.double())
    h, final, ck = kda.kda_glr_prefill(x, gate, cu_of([1]), return_checkpoints=True, **SIGMOID)
    near(h, c * x.double(), 9)
    near(final, c * x.double(), 9)
    state = h0.clone()
    near(kda.kda_glr_decode_step(x, gate, state, **SIGMOID), c * x.double(), 9)
    near(state, c * x.double(), 9)
    dh = randn(1, dim, seed=3, dtype=types[0])
    dx, dg, _ = kda.kda_glr_prefill_backward(x, gate, cu_of([1]), dh, checkpoints=ck, **SIGMOID)
    near(dx, c * dh.double(), 9)
    near(dg, -a * c * dh.double() * x.double(), 26)


def test_far_sigmoid_gates_past_fp32():
    """Beyond its range 1 - a is 0, a 1; e^g overflows on the way."""
    inf = float("inf")
    gate = torch.tensor([87.9, 88.0, 88.5, 89.0, 126.0, 1e3, 1e30, inf], device="cuda").repeat(1, 8)
    x = torch.full_like(gate, 3.0)
    h, _, ck = kda.kda_glr_prefill(x, gate, cu_of([1]), return_checkpoints=True, **SIGMOID)
    assert bool((h.abs() <= 2.0 ** -124).all())
    assert bool((kda.kda_glr_decode_step(x, gate, torch.zeros_like(x), **SIGMOID).abs() <= 2.0 ** -124).all())
    grads = kda.kda_glr_prefill_backward(x, gate, cu_of([1]), x, checkpoints=ck, **SIGMOID)
    assert all(bool((g.abs() <= 2.0 ** -122).all()) for g in grads[:2])
    low, _, _ = kda.kda_glr_prefill(x, -gate, cu_of([1]), **SIGMOID)
    assert torch.equal(low, x) and torch.equal(kda.kda_glr_decode_step(x, -gate, torch.ones_like(x), **SIGMOID), x)
