"""Synchronous refusals of the gated delta rule's and the RMS norm's entry points (no kernel runs):
fake addresses, which validation rejects before any CUDA call, and the binding's checks on CPU tensors."""
import ctypes

import pytest
import torch

import linear_attention_chunkwise_gb300 as kda
from linear_attention_chunkwise_gb300 import _build

INV, UNS, WS = kda.KDA_ERR_INVALID_ARG, kda.KDA_ERR_UNSUPPORTED, kda.KDA_ERR_WORKSPACE
BASE = 1 << 40
MB = 1 << 20


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return kda.load_library()


def P(x):
    return None if x is None else ctypes.c_void_p(x)


def _prefill(lib, **over):  # T = 128 tokens of 2 q/k and 4 value heads, every buffer a megabyte apart
    a = dict(q=BASE, k=BASE + MB, v=BASE + 2 * MB, dtype=0, ld=BASE + 3 * MB, beta=BASE + 4 * MB, S0=None,
             cu=BASE + 5 * MB, N=1, T=128, Hk=2, Hv=4, dk=128, dv=128, o=BASE + 6 * MB, Sf=BASE + 7 * MB,
             ws=BASE + 8 * MB, wsb=1 << 30, status=None)
    a.update(over)
    return lib.kda_gdn_prefill(P(a["q"]), P(a["k"]), P(a["v"]), a["dtype"], P(a["ld"]), P(a["beta"]), P(a["S0"]),
                               P(a["cu"]), a["N"], a["T"], a["Hk"], a["Hv"], a["dk"], a["dv"], P(a["o"]), P(a["Sf"]),
                               P(a["ws"]), a["wsb"], P(a["status"]), None)


@pytest.mark.parametrize("over,expect", [
    (dict(dk=64), UNS), (dict(dv=256), UNS), (dict(dtype=2), UNS), (dict(Hv=3), INV), (dict(Hk=0), INV),
    (dict(Hv=0), INV), (dict(Hk=8), INV), (dict(N=-1), INV), (dict(T=-1), INV), (dict(T=2 ** 31), INV),
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(ld=None), INV), (dict(beta=None), INV),
    (dict(o=None), INV), (dict(cu=None), INV), (dict(ws=None), INV), (dict(q=BASE + 8), INV), (dict(v=BASE + 2 * MB + 2), INV),
    (dict(ld=BASE + 3 * MB + 2), INV), (dict(cu=BASE + 5 * MB + 1), INV), (dict(S0=BASE + 9 * MB + 8), INV),
    (dict(ws=BASE + 8 * MB + 16), INV), (dict(status=BASE + 2), INV), (dict(wsb=0), WS),
    (dict(o=BASE + MB), INV), (dict(o=BASE + 2 * MB), INV), (dict(Sf=BASE + 6 * MB), INV), (dict(o=BASE + 8 * MB), INV),
    (dict(S0=BASE + 7 * MB + 4096), INV), (dict(Sf=BASE + 5 * MB - 4096), INV), (dict(status=BASE + 6 * MB), INV),
    (dict(N=2 ** 30), INV),
])
def test_prefill_refuses(lib, over, expect):
    assert _prefill(lib, **over) == expect


def test_prefill_takes_the_state_in_place(lib):
    # past validation: no GPU here, so the device check answers
    ok = (kda.KDA_ERR_CUDA, UNS)
    if torch.cuda.is_available():
        pytest.skip("fake addresses")
    assert _prefill(lib, S0=BASE + 7 * MB) in ok
    assert _prefill(lib, T=0, q=None, k=None, v=None, ld=None, beta=None, o=None) in ok


def test_workspace_queries(lib):
    assert kda.kda_gdn_prefill_workspace_bytes(torch.bfloat16, 1, 8192, 16, 32) >= 256
    for bad in ((torch.bfloat16, -1, 10, 2, 2), (torch.bfloat16, 1, 10, 2, 3), (torch.bfloat16, 1, 10, 2, 2, 64, 128),
                (7, 1, 10, 2, 2)):
        assert kda.kda_gdn_prefill_workspace_bytes(*bad) == 0
    assert kda.kda_rms_norm_backward_workspace_bytes(10, 100) >= 10 * 100 * 4
    assert kda.kda_rms_norm_backward_workspace_bytes(-1, 100) == 0
    assert kda.kda_rms_norm_backward_workspace_bytes(1, 0) == 0
    assert kda.kda_rms_norm_backward_workspace_bytes(1, (1 << 20) + 1) == 0


def _decode(lib, **over):
    a = dict(q=BASE, k=BASE + MB, v=BASE + 2 * MB, dtype=0, ld=BASE + 3 * MB, beta=BASE + 4 * MB, S=BASE + 8 * MB,
             slots=8, idx=BASE + 5 * MB, N=4, Hk=2, Hv=4, dk=128, dv=128, o=BASE + 6 * MB, status=None)
    a.update(over)
    return lib.kda_gdn_decode_step(P(a["q"]), P(a["k"]), P(a["v"]), a["dtype"], P(a["ld"]), P(a["beta"]), P(a["S"]),
                                   a["slots"], P(a["idx"]), a["N"], a["Hk"], a["Hv"], a["dk"], a["dv"], P(a["o"]),
                                   P(a["status"]), None)


@pytest.mark.parametrize("over,expect", [
    (dict(dk=1), UNS), (dict(dtype=9), UNS), (dict(Hv=5), INV), (dict(N=-1), INV), (dict(slots=-1), INV),
    (dict(q=None), INV), (dict(S=None), INV), (dict(o=None), INV), (dict(beta=None), INV), (dict(S=BASE + 8 * MB + 4), INV),
    (dict(idx=BASE + 5 * MB + 2), INV), (dict(idx=None, N=9), INV), (dict(o=BASE + 8 * MB), INV), (dict(o=BASE), INV),
    (dict(idx=BASE + 8 * MB), INV), (dict(status=BASE + 8 * MB), INV), (dict(ld=BASE + 8 * MB), INV),
])
def test_decode_refuses(lib, over, expect):
    assert _decode(lib, **over) == expect


def _norm(lib, **over):  # 8 rows of 256
    a = dict(x=BASE, res=BASE + MB, dtype=0, w=BASE + 2 * MB, eps=1e-6, rows=8, dim=256, out=0, group=0, y=BASE + 3 * MB,
             scales=None, h=BASE + 4 * MB)
    a.update(over)
    return lib.kda_rms_norm(P(a["x"]), P(a["res"]), a["dtype"], P(a["w"]), a["eps"], a["rows"], a["dim"], a["out"],
                            a["group"], P(a["y"]), P(a["scales"]), P(a["h"]), None)


S = BASE + 5 * MB


@pytest.mark.parametrize("over,expect", [
    (dict(dtype=3), UNS), (dict(out=3), UNS), (dict(out=-1), UNS), (dict(rows=-1), INV), (dict(rows=2 ** 31), INV),
    (dict(dim=0), INV), (dict(dim=(1 << 20) + 1), INV), (dict(eps=-1.0), INV), (dict(eps=float("nan")), INV),
    (dict(x=None), INV), (dict(y=None), INV), (dict(x=BASE + 8), INV), (dict(h=BASE + 4 * MB + 2), INV),
    (dict(w=BASE + 2 * MB + 2), INV), (dict(group=128), INV), (dict(scales=S), INV), (dict(out=1), INV),
    (dict(out=1, scales=S, group=64), INV), (dict(out=2, scales=S, group=128, dim=200), INV),
    (dict(h=BASE + 16), INV), (dict(h=BASE + MB + 16), INV), (dict(h=BASE + 3 * MB), INV), (dict(h=BASE + 2 * MB), INV),
    (dict(y=BASE + 16), INV), (dict(y=BASE + MB), INV), (dict(y=BASE + 2 * MB), INV), (dict(out=1, scales=S, y=BASE), INV),
    (dict(out=1, scales=BASE), INV), (dict(out=1, scales=BASE + 3 * MB), INV), (dict(out=1, scales=BASE + 4 * MB), INV),
])
def test_norm_refuses(lib, over, expect):
    assert _norm(lib, **over) == expect


def _norm_backward(lib, **over):
    a = dict(dy=BASE, h=BASE + MB, dh=BASE + 2 * MB, dtype=0, w=BASE + 3 * MB, eps=1e-6, rows=8, dim=256, dx=BASE + 4 * MB,
             dw=BASE + 5 * MB, ws=BASE + 6 * MB, wsb=1 << 20)
    a.update(over)
    return lib.kda_rms_norm_backward(P(a["dy"]), P(a["h"]), P(a["dh"]), a["dtype"], P(a["w"]), a["eps"], a["rows"],
                                     a["dim"], P(a["dx"]), P(a["dw"]), P(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("over,expect", [
    (dict(dtype=3), UNS), (dict(rows=-1), INV), (dict(dim=0), INV), (dict(eps=-1e-9), INV), (dict(dy=None), INV),
    (dict(h=None), INV), (dict(dx=None), INV), (dict(ws=None), INV), (dict(wsb=100), WS), (dict(ws=BASE + 6 * MB + 64), INV),
    (dict(dx=BASE + MB), INV), (dict(dx=BASE + 16), INV), (dict(dx=BASE + 3 * MB), INV), (dict(dx=BASE + 5 * MB), INV),
    (dict(dx=BASE + 6 * MB), INV), (dict(dw=BASE + MB), INV), (dict(dw=BASE + 3 * MB), INV), (dict(dw=BASE + 6 * MB), INV),
    (dict(dw=BASE + 5 * MB + 4), INV),
])
def test_norm_backward_refuses(lib, over, expect):
    assert _norm_backward(lib, **over) == expect


def test_binding_refuses_tensors_off_the_gpu():
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    g = torch.zeros(4, 2)
    cu = torch.tensor([0, 4], dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_gdn_prefill(x, x, x, g, g, cu)
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_gdn_decode_step(x, x, x, g, g, torch.zeros(4, 2, 128, 128))
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_rms_norm(x[0])
    with pytest.raises(ValueError, match="CUDA"):
        kda.kda_rms_norm_backward(x[0], x[0])
    with pytest.raises(TypeError):
        kda.kda_rms_norm(None)


def _backward(lib, **over):  # T = 128 tokens of 2 q/k and 4 value heads, every buffer a megabyte apart
    names = ("q", "k", "v", "ld", "beta", "cu", "do", "dq", "dk", "dv", "dld", "db", "ws")
    a = dict({n: BASE + i * MB for i, n in enumerate(names)}, dtype=0, S0=None, N=1, T=128, Hk=2, Hv=4, kd=128, vd=128,
             dS=None, dS0=None, wsb=1 << 30, status=None)
    a.update(over)
    return lib.kda_gdn_prefill_backward(
        P(a["q"]), P(a["k"]), P(a["v"]), a["dtype"], P(a["ld"]), P(a["beta"]), P(a["S0"]), P(a["cu"]), a["N"], a["T"], a["Hk"],
        a["Hv"], a["kd"], a["vd"], P(a["do"]), P(a["dS"]), P(a["dq"]), P(a["dk"]), P(a["dv"]), P(a["dld"]), P(a["db"]),
        P(a["dS0"]), P(a["ws"]), a["wsb"], P(a["status"]), None)


FAR = BASE + 40 * MB


@pytest.mark.parametrize("over,expect", [
    (dict(dtype=1), UNS), (dict(dtype=2), UNS), (dict(kd=64), UNS), (dict(vd=64), UNS), (dict(Hv=3), INV), (dict(Hk=0), INV),
    (dict(Hv=0), INV), (dict(N=-1), INV), (dict(T=-1), INV), (dict(T=2 ** 31), INV), (dict(N=0), INV), (dict(N=2 ** 30), INV),
    *[({n: None}, INV) for n in ("q", "k", "v", "ld", "beta", "cu", "do", "dq", "dk", "dv", "dld", "db", "ws")],
    *[({n: FAR + 8}, INV) for n in ("q", "k", "v", "do", "dq", "dk", "dv", "S0", "dS", "dS0", "ws")],
    *[({n: FAR + 2}, INV) for n in ("ld", "beta", "dld", "db", "cu", "status")],
    (dict(wsb=0), WS), (dict(wsb=2 * 4 * 200000), WS),
    (dict(dq=BASE), INV), (dict(dk=BASE + MB + 16), INV), (dict(dv=BASE + 2 * MB), INV), (dict(dld=BASE + 3 * MB), INV),
    (dict(db=BASE + 10 * MB), INV), (dict(dS=FAR, dS0=FAR), INV), (dict(S0=FAR, dS0=FAR + 4096), INV),
    (dict(dv=BASE + 6 * MB), INV), (dict(ws=BASE + 9 * MB + 256), INV), (dict(status=BASE + 7 * MB), INV),
    (dict(status=BASE + 5 * MB + 4), INV),
])
def test_backward_refuses(lib, over, expect):
    assert _backward(lib, **over) == expect


def test_backward_workspace_queries(lib):
    need = kda.kda_gdn_prefill_backward_workspace_bytes
    assert need(torch.bfloat16, 1, 8192, 16, 32) > need(torch.bfloat16, 1, 4096, 16, 32) > 0
    for bad in ((torch.float32, 1, 64, 2, 2), (torch.bfloat16, -1, 64, 2, 2), (torch.bfloat16, 1, 64, 2, 3),
                (torch.bfloat16, 1, -1, 2, 2), (torch.bfloat16, 1, 64, 2, 2, 64, 128)):
        assert need(*bad) == 0


def _in_chunks(num_seqs, tokens, heads, per_chunk):  # workspace of the chunkwise path, its tables (under 16 KB) apart
    return (-(-tokens // 64) + num_seqs) * heads * per_chunk


@pytest.mark.parametrize("num_seqs,tokens,Hk,Hv", [(65, 129, 2, 4), (1000, 2000, 16, 32), (64, 100, 2, 4), (2000, 2000, 1, 1)])
def test_backward_of_one_long_sequence_among_short_ones_goes_in_chunks(num_seqs, tokens, Hk, Hv):
    need = kda.kda_gdn_prefill_backward_workspace_bytes(torch.bfloat16, num_seqs, tokens, Hk, Hv)
    assert 0 <= need - _in_chunks(num_seqs, tokens, Hv, 27136 + 196608) < 1 << 16


@pytest.mark.parametrize("num_seqs,tokens,Hk,Hv", [(1000, 8000, 16, 32), (256, 1024, 2, 4), (64, 512, 16, 32), (40, 300, 1, 1)])
def test_prefill_of_one_long_sequence_among_short_ones_goes_in_chunks(num_seqs, tokens, Hk, Hv):
    need = kda.kda_gdn_prefill_workspace_bytes(torch.bfloat16, num_seqs, tokens, Hk, Hv)
    assert 0 <= need - _in_chunks(num_seqs, tokens, Hv, 3 * 8192 + 1536) < 1 << 16


@pytest.mark.parametrize("Hk,Hv", [(1, 1), (2, 4), (16, 32), (4, 128)])
@pytest.mark.parametrize("query", ["kda_gdn_prefill_workspace_bytes", "kda_gdn_prefill_backward_workspace_bytes"])
def test_a_workspace_serves_every_smaller_call(query, Hk, Hv):
    need = lambda n, t: getattr(kda, query)(torch.bfloat16, n, t, Hk, Hv)  # noqa: E731
    seqs = [1, 2, 3, 5, 8, 9, 13, 60, 61, 64, 65, 200, 1000]
    tokens = [0, 1, 2, 7, 8, 9, 14, 15, 16, 17, 40, 41, 64, 65, 70, 128, 129, 134, 135, 200, 201, 512, 513, 2000, 2048, 8000, 8001]
    table = [[need(n, t) for t in tokens] for n in seqs]
    for row in table:
        assert row[0] >= 256 and row == sorted(row)
    for column in zip(*table):
        assert list(column) == sorted(column)
    # and a workspace that is smaller than what a call takes is refused
    call = _prefill if query == "kda_gdn_prefill_workspace_bytes" else _backward
    assert call(kda.load_library(), N=1, T=128, Hk=Hk, Hv=Hv, wsb=need(1, 128) - 1) == WS


def test_backward_takes_no_tokens(lib):
    # past validation: no GPU here, so the device check answers
    if torch.cuda.is_available():
        pytest.skip("fake addresses")
    none = {n: None for n in ("q", "k", "v", "ld", "beta", "do", "dq", "dk", "dv", "dld", "db")}
    assert _backward(lib, T=0, **none) in (kda.KDA_ERR_CUDA, UNS)
