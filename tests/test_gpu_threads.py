"""Calls of the layer from several host threads."""
import threading

import pytest

import synth
from conftest import cuda_available
from test_gpu_few import device_call, device_weights, m  # noqa: F401 (m: fixture)

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]


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
