"""The gated delta rule and the RMS norm called from two Python threads, and behind a host callback that needs Python."""
import ctypes
import threading

import pytest
import torch

import linear_attention_chunkwise_gb300 as kda
from tests.conftest import cuda_ok
from tests.test_gpu_gdn import inputs
from tests.test_gpu_gdn_backward import with_grads

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_ok(), reason="needs a CUDA GPU")]


def test_two_threads_on_two_streams():
    def work(x, rows, w):
        g = with_grads(x)
        o, S = kda.kda_gdn_prefill(**x)
        grads = kda.kda_gdn_prefill_backward(**g)
        y, scales, _ = kda.kda_rms_norm(rows, w, quant="e4m3")
        dx, dw = kda.kda_rms_norm_backward(rows, rows, w)
        step = kda.kda_gdn_decode_step(*(x[n][:2].contiguous() for n in ("q", "k", "v", "log_decay", "beta")), S)
        return [o, S, *grads, y.view(torch.uint8), scales, dx, dw, step]

    jobs = []
    for seed, lengths, heads in ((1, [300, 77], (2, 4)), (2, [130, 5], (16, 32))):
        rows = torch.randn(500, 1024 + 8 * seed, device="cuda", generator=torch.Generator("cuda").manual_seed(seed))
        jobs.append((inputs(lengths, *heads, seed=seed), rows.bfloat16(), rows[0].clone()))
    want = [work(*j) for j in jobs]
    torch.cuda.synchronize()
    got, failed = [[], []], []
    start = threading.Barrier(2)

    def run(i):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait(30)
                for _ in range(20):
                    got[i].append(work(*jobs[i]))
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed
    for i in range(2):
        assert len(got[i]) == 20
        for r in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(r, want[i]))


def _cudart():
    with open("/proc/self/maps") as fh:
        paths = {line.split()[-1] for line in fh if "libcudart.so" in line}
    return ctypes.CDLL(sorted(paths)[0])


def test_a_full_queue_behind_a_host_callback():
    """The callback needs the interpreter lock, and ends once another Python thread says so; more launches than the
    device's queue holds stand behind it."""
    rows = torch.randn(4, 256, device="cuda").bfloat16()
    y, want = torch.empty_like(rows), kda.kda_rms_norm(rows)[0]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    gate, queued, seen = threading.Event(), threading.Event(), []
    callback = ctypes.CFUNCTYPE(None, ctypes.c_void_p)(lambda _: seen.append(gate.wait(30)))

    def opener():
        queued.wait(0.5)  # runs out while the launches wait for room in the queue
        gate.set()

    t = threading.Thread(target=opener)
    t.start()
    assert _cudart().cudaLaunchHostFunc(ctypes.c_void_p(stream.cuda_stream), callback, None) == 0
    for _ in range(4000):
        kda.kda_rms_norm(rows, y=y, stream=stream)
    queued.set()
    t.join()
    stream.synchronize()
    assert seen == [True] and torch.equal(y, want)
