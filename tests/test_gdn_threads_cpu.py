"""The entry points of the gated delta rule and of the RMS norm give the interpreter lock up for their C call.

A launch waits while the device's queue is full, possibly behind something that another Python thread has to do
first.  A stand-in for the library, whose entries take a while and return KDA_OK, is called through the binding; a second
thread has to get its turns meanwhile.
"""
import subprocess
import threading
import time
import types

import pytest
import torch

from linear_attention_chunkwise_gb300 import _binding, _gdn

CALL_S = 0.3


@pytest.fixture(scope="module")
def slow_lib(tmp_path_factory):
    d = tmp_path_factory.mktemp("slow")
    body = "".join(f"unsigned long {n}(void) {{ {'' if n.endswith('_workspace_bytes') else f'usleep({int(CALL_S * 1e6)});'} return 0; }}\n"
                   for n in _binding.EXPORTED_SYMBOLS)
    (d / "slow.c").write_text("#include <unistd.h>\n" + body)
    subprocess.run(["gcc", "-shared", "-fPIC", "-o", str(d / "slow.so"), str(d / "slow.c")], check=True)
    return _binding.load_library(str(d / "slow.so"))


def _calls():
    x, g = torch.zeros(4, 2, 128), torch.zeros(4, 2)
    cu, S, rows = torch.tensor([0, 4], dtype=torch.int32), torch.zeros(4, 2, 128, 128), torch.zeros(4, 128)
    return {"kda_gdn_prefill": lambda: _gdn.kda_gdn_prefill(x, x, x, g, g, cu),
            "kda_gdn_prefill_backward": lambda: _gdn.kda_gdn_prefill_backward(x, x, x, g, g, cu, x),
            "kda_gdn_decode_step": lambda: _gdn.kda_gdn_decode_step(x, x, x, g, g, S),
            "kda_rms_norm": lambda: _gdn.kda_rms_norm(rows),
            "kda_rms_norm_backward": lambda: _gdn.kda_rms_norm_backward(rows, rows)}


@pytest.mark.parametrize("name", ["kda_gdn_prefill", "kda_gdn_prefill_backward", "kda_gdn_decode_step", "kda_rms_norm",
                                  "kda_rms_norm_backward"])
def test_other_threads_run_during_a_call(slow_lib, monkeypatch, name):
    # tensors on the CPU in the place of ones on the GPU
    monkeypatch.setattr(_binding, "_lib", slow_lib)
    monkeypatch.setattr(_gdn, "_first", lambda t, n, dims: (types.SimpleNamespace(index=0), _binding.KDA_DTYPE_BF16))
    monkeypatch.setattr(_gdn, "_check", lambda *a: None)
    monkeypatch.setattr(_gdn, "_current_device", lambda: 0)
    monkeypatch.setattr(_gdn, "_current_stream", lambda index: 0)
    monkeypatch.setattr(_gdn, "_allocate", lambda size, stream: 0)
    monkeypatch.setattr(_gdn, "_free", lambda memory: None)
    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: real(*a, **k))
    turns, over = [], threading.Event()

    def other():
        while not over.wait(0.01):
            turns.append(time.monotonic())

    t = threading.Thread(target=other)
    t.start()
    try:
        begin = time.monotonic()
        _calls()[name]()
        end = time.monotonic()
    finally:
        over.set()
        t.join()
    assert end - begin >= CALL_S
    inside = [x for x in turns if begin + 0.1 * CALL_S < x < end - 0.1 * CALL_S]
    assert inside, "no other thread ran while the call was in the library"
