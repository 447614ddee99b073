"""How the FP8 layer quantises h, seen in outputs that are single elements of h.

Every expert's W2 is the identity (codes 1.0, scale 1), so that an output is one quantised element
of h, code times block scale, rounded to bf16. The gate sums are 56 (where silu is the identity in
fp32) and the up sums 448 (c_a + c_b) s3 with an up scale s3 of arbitrary mantissa: h holds values
on ties of the E4M3 grid but for the roundings of h, of the scale and of its reciprocal."""
import numpy as np
import pytest

import fp4_ref as ref
import synth
from conftest import cuda_available
from parity import bf16_bits_to_f64
from test_gpu_few import Call, bits, m  # noqa: F401 (m: fixture)

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]

T = E = 8
H = I = 256


def e4m3(v):
    """E4M3 codes of values that have one."""
    t = ref.e4m3_table()[:127]
    c = np.searchsorted(t, np.abs(v))
    assert np.array_equal(t[c], np.abs(v))
    return (c | np.where(np.signbit(v), 128, 0)).astype(np.uint8)


def tie_layer(seed):
    """Token t goes to expert t alone; h of a block is 448 (first feature) and odd values between 16
    and 32 times the block's scale."""
    rng = np.random.default_rng(seed)
    x = np.zeros((T, H), np.float32)
    x[:, :2] = 448.0
    x[np.arange(T), 8 + np.arange(T)] = 448.0
    w1, w3 = np.zeros((E, I, H)), np.zeros((E, I, H))
    w1[:, :, 0] = 1.0
    w3[:, :, 0] = rng.integers(8, 16, (E, I)) * 2
    w3[:, :, 1] = 1.0
    w3[:, ::128, 0], w3[:, ::128, 1] = 448.0, 0.0
    s1 = np.full((E, I // 128, H // 128), 1 / 8, np.float32)
    s3 = (rng.uniform(1, 2, (E, I // 128, H // 128)) * 2.0 ** -8).astype(np.float32)
    rw = np.zeros((E, H), np.float32)
    rw[np.arange(E), 8 + np.arange(E)] = 1.0
    return synth.f32_to_bf16(x), {
        "router_w": synth.f32_to_bf16(rw), "router_bias": None, "w1": e4m3(w1), "w3": e4m3(w3),
        "w2": np.broadcast_to(e4m3(np.eye(H)), (E, H, I)).copy(), "s1": s1, "s3": s3,
        "s2": np.ones((E, H // 128, I // 128), np.float32)}


@pytest.fixture(params=["auto", "single", "pair", "swap"])
def variant(request, m):  # noqa: F811
    m.moe_set_gemm_variant(getattr(m, "MOE_GEMM_" + request.param.upper()))
    yield request.param
    m.moe_set_gemm_variant(m.MOE_GEMM_AUTO)


def forward(m, call, x):  # noqa: F811
    import torch
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    m.moe_forward(call.cfg, T, x, call.w, out, call.ws)
    assert m.moe_read_status(call.ws) == 0
    return out


def test_few_rounds_h_as_the_layer(m, variant):  # noqa: F811
    """moe_forward_few gives the codes and scales of h that moe_forward gives, values on borders included."""
    for seed in range(8):
        xh, wt = tie_layer(seed)
        call = Call(m, 1, T, H, I, E, 1, 0, wt)
        x = m.to_device(xh)
        few = bits(call(x)).copy()
        assert call.idx.cpu().numpy()[:, 0].tolist() == list(range(T))
        assert np.array_equal(few, bits(forward(m, call, x)))
        v = bf16_bits_to_f64(few)
        # codes 448 and 16 to 32 of one scale: 14 at least, less the two bf16 roundings
        assert (v[:, ::128] > 13.8 * v[:, 1::128]).all() and (v > 0).all()
