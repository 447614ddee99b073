"""Calls of the layer from several host threads, at once with shapes, a workspace and a stream each.

A launch's shared-memory limit is state of the kernel function, not of the launch: calls of other
shapes must not lower it between a thread's setting and its launch."""
import threading

import numpy as np
import pytest

import synth
from conftest import cuda_available
from test_gpu_few import device_call, device_weights, m  # noqa: F401 (m: fixture)

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]


def together(*work):
    """Runs the functions, each on a stream of its own, on threads that start together."""
    import torch
    start, errors = threading.Barrier(len(work)), []

    def body(f):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                f()
                torch.cuda.current_stream().synchronize()
        except Exception as e:  # noqa: BLE001 (reported by the caller)
            errors.append(e)
    threads = [threading.Thread(target=body, args=(f,)) for f in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors


@pytest.mark.parametrize("w", [0, 1, 2, 3])
def test_few_first_call_of_a_thread(m, w):  # noqa: F811
    """A host thread whose first use of the device is this call."""
    import torch
    T, H, I, E = 2, 512, 512, 4
    call = device_call(m, w, T, H, I, E, 2, 1, device_weights(w, 98, E, 1, H, I))
    x = m.to_device(synth.normal_bf16(99, 1, (T, H), 1.0))
    want = call(x).clone()
    call.out.fill_(0)
    stream = torch.cuda.current_stream().cuda_stream
    errors = []

    def body():
        try:
            call(x, stream=stream)
        except m.MoeError as e:
            errors.append(e)
    t = threading.Thread(target=body)
    t.start()
    t.join()
    assert not errors, errors
    assert torch.equal(call.out[:T].view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("w", [0, 1, 2, 3])
def test_few_threads(m, w):  # noqa: F811
    import torch
    calls = []
    for T, H, I, E in ((1, 512, 512, 12), (7, 4096, 1024, 12)):
        call = device_call(m, w, T, H, I, E, 2, 1, device_weights(w, 94, E, 1, H, I))
        x = m.to_device(synth.normal_bf16(95, 1, (T, H), 1.0))
        calls.append((call, x, call(x).clone()))
    torch.cuda.synchronize()

    def many(call, x):
        return lambda: [call(x) for _ in range(6000)]
    together(*(many(call, x) for call, x, _ in calls))
    for call, _, want in calls:
        assert m.moe_read_status(call.ws) == 0
        assert torch.equal(call.out[:call.T].view(torch.int16), want.view(torch.int16))


def test_router_threads(m):  # noqa: F811
    import torch
    T, H, k = 64, 1024, 2
    x = m.to_device(synth.normal_bf16(96, 1, (T, H), 1.0))
    work, checks = [], []
    for E in (16, 352):
        cfg = m.make_config(H, E, k, 0, 512, m.MOE_WDTYPE_BF16)
        rw = m.to_device(synth.normal_bf16(97, E, (E, H), H ** -0.5))
        idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
        gate = torch.empty((T, k), dtype=torch.float32, device="cuda")
        ws = torch.empty(m.moe_workspace_bytes(cfg, T), dtype=torch.uint8, device="cuda")

        def route(cfg=cfg, rw=rw, idx=idx, gate=gate, ws=ws):
            m.moe_route(cfg, T, x, rw, None, idx, gate, None, ws)
        route()
        checks.append((idx, gate, idx.clone(), gate.clone(), ws))
        work.append(lambda route=route: [route() for _ in range(6000)])
    torch.cuda.synchronize()
    together(*work)
    for idx, gate, idx0, gate0, ws in checks:
        assert m.moe_read_status(ws) == 0
        assert torch.equal(idx, idx0) and np.array_equal(gate.cpu().numpy(), gate0.cpu().numpy())
