"""Gates of the gated linear recurrence far from 0, element by element relative to their own values, what a single token
keeps of a state, and states that grow.

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


@pytest.mark.parametrize("kind", ["log_decay", "sigmoid"])
@pytest.mark.parametrize("dim", [4096, 4001])
def test_decode_keeps_what_is_left_of_a_state(dim, kind):
    """The state's share of the next one is a h: a to 14 u below 1/2 (sigmoid e c: 5 + 8 + 1; exp 5), the product's rounding; from 1/2 on
    h - c h with c off by 8 u of 1 or less, 16 u of a.  With an input, its own 9 u and the sum's roundings besides."""
    gate, h0 = spread(-80.0, 0.0, dim)
    a = gate.double().exp() if kind == "log_decay" else torch.sigmoid(gate.double())
    for complement in (False, True):
        opts = dict(gate_kind=kind, complement=complement)
        state = h0.clone()
        h = kda.kda_glr_decode_step(torch.zeros_like(h0), gate, state, **opts)
        near(h, a * h0.double(), 18)
        assert torch.equal(h, state)
        x, state = randn(1, dim, seed=5), h0.clone()
        v = x.double() * (1 - a if complement else 1)
        kda.kda_glr_decode_step(x, gate, state, **opts)
        size = (a * h0.double()).abs() + v.abs()
        close(state, a * h0.double() + v, 18 * U * size + (8 * U * x.double().abs() if complement else 0))


def test_decode_of_states_that_are_not_finite():
    """a times an infinite state is infinite, 0 times it NaN, as the formula has it."""
    inf, nan = float("inf"), float("nan")
    state = torch.tensor([inf, -inf, inf, nan, -inf, inf], device="cuda").repeat(1, 6)
    gate = torch.tensor([-0.1, -5.0, -inf, -0.1, -0.01, 0.0], device="cuda").repeat(1, 6)
    want = torch.tensor([inf, -inf, nan, nan, -inf, inf], device="cuda").repeat(1, 6)
    for kind, g in (("log_decay", gate), ("sigmoid", torch.where(gate == -inf, gate, gate + 1))):
        s = state.clone()
        h = kda.kda_glr_decode_step(torch.ones_like(g), g, s, gate_kind=kind)
        for got in (h, s):
            assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(5.0, 1e30, -1e30), want.nan_to_num(5.0, 1e30, -1e30))


@pytest.mark.parametrize("gate", [0.2, 0.3, 0.45, 1.0, 5.0, 40.0, 80.0])
def test_decode_of_states_that_grow(gate):
    """Decays above 1: a to 5 u beyond 1.5; below it h + n h with n off by less than 16 u (5 u of a and the difference's rounding, or less)."""
    h0 = randn(1, 256, seed=1)
    g = torch.full_like(h0, gate)
    h = kda.kda_glr_decode_step(torch.zeros_like(h0), g, h0.clone())
    near(h, g.double().exp() * h0.double(), 18)
    beyond = kda.kda_glr_decode_step(torch.zeros_like(h0), torch.full_like(h0, 100.0), h0.clone())
    assert bool((beyond == h0 * float("inf")).all())


@pytest.mark.parametrize("dim", [64, 33])
def test_growth_while_128_tokens_products_are_finite(dim):
    """Log gates above 0: a token's 1 - a is good to (22 + 1.25 g) u of its value (the difference of e^g, 5 + 1.25 g u, and 1, which
    is less of it below g = 1), its step and joins round by 6 u more.  Sums of one sign, so a token adds 30 u of the state at most.  The
    products over 128 tokens are e^64; a state of zero stays zero."""
    T = 150
    x, gate, h0 = randn(2 * T, dim, seed=1).abs(), torch.full((2 * T, dim), 0.5, device="cuda"), randn(2, dim, seed=3).abs()
    x[:T - 1], h0[0] = 0, 0  # nothing but zeros, and an input at the last token
    dh, cu = randn(2 * T, dim, seed=4).abs(), cu_of([T, T])
    dh[T + 1:] = 0
    h, final, ck = kda.kda_glr_prefill(x, gate, cu, h0, return_checkpoints=True)
    ref, s = torch.empty_like(x, dtype=torch.float64), None
    for t in range(2 * T):
        s = ref[t] = gate[t].double().exp() * (h0[t // T].double() if t % T == 0 else s) + x[t].double()
    assert bool((h[:T - 1] == 0).all())
    near(h, ref, 30 * T)
    near(final, ref[T - 1::T], 30 * T)
    dx, dg, dh0 = kda.kda_glr_prefill_backward(x, gate, cu, dh, h0, checkpoints=ck)
    lam, m = torch.empty_like(ref), None
    for t in reversed(range(2 * T)):
        lam[t] = dh[t].double() + (0 if t % T == T - 1 else m)
        m = gate[t].double().exp() * lam[t]
    assert bool((dx[T + 1:] == 0).all())
    near(dx, lam, 30 * T)
    near(dh0, torch.stack([gate[0].double().exp() * lam[0], gate[T].double().exp() * lam[T]]), 30 * T)
    before = torch.cat([ref[:1] * 0, ref[:-1]])
    before[0], before[T] = h0[0].double(), h0[1].double()
    near(dg, gate.double().exp() * lam * before, 60 * T + 32)


def test_a_gate_of_zero_in_a_captured_decode():
    """A decay of 1 leaves the state, replay after replay."""
    state, gate, x = randn(3, 128, seed=1), torch.zeros(3, 128, device="cuda"), torch.zeros(3, 128, device="cuda")
    keep = state.clone()
    kda.kda_glr_decode_step(x, gate, state)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h = kda.kda_glr_decode_step(x, gate, state)
    for _ in range(3):
        graph.replay()
    assert torch.equal(h, keep) and torch.equal(state, keep)
