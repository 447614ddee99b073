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
from parity import bf16_bits_to_f64, rows_rel
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


@pytest.mark.parametrize("size", [1e-19, 3e-21, 3e-23])
def test_tiny_tokens_stay_finite(m, variant, size):  # noqa: F811
    """Tokens whose h blocks have subnormal scales (h goes as x squared), some of h exactly zero: the
    definition's outputs, not the NaN of an infinite reciprocal. At the last size h is a few of the
    smallest fp32 numbers, and the outputs have to be finite."""
    rng = np.random.default_rng(5)
    n, k, S = 4, 2, 1
    wt = {"router_w": synth.f32_to_bf16(np.zeros((n, H), np.float32)),
          "router_bias": np.arange(n, dtype=np.float32)}
    for pre, c in (("", n), ("s", S)):
        for name in "132":
            code = rng.integers(0, 256, (c, H, I)).astype(np.uint8)
            code[(code & 127) > 0x60] &= 0x9F
            if name == "3":
                code[:, ::5] = 0  # no up sum: h is zero
            wt[pre + "w" + name] = code
            wt[pre + "s" + name] = np.full((c, 2, 2), 2.0 ** 40 if name == "2" else 2.0 ** -6, np.float32)
    xh = synth.f32_to_bf16((rng.standard_normal((T, H)) * size).astype(np.float32))
    call = Call(m, 1, T, H, I, n, k, S, wt)
    x = m.to_device(xh)
    outs = [bf16_bits_to_f64(bits(o)) for o in (call(x), forward(m, call, x))]
    assert m.moe_read_status(call.ws) == 0
    e = np.exp([1.0, 0.0])
    idx, gate = np.tile([n - 1, n - 2], (T, 1)), np.tile(e / e.sum(), (T, 1))

    def of(pre):
        return lambda j=0: [ref.e4m3_table()[wt[pre + "w" + i][j]] * np.kron(wt[pre + "s" + i][j], np.ones((128, 128)))
                            for i in "132"]
    for out in outs:
        assert np.isfinite(out).all()
    if size > 1e-21:
        want = ref.layer("fp8", synth.bf16_to_f32(xh).astype(np.float64), idx, gate, of(""), of("s"))
        assert max(rows_rel(out, want).max() for out in outs) < 2e-2


def test_infinite_h_is_not_lost(m, variant):  # noqa: F811
    """Finite tokens whose h overflows to infinity give rows that are not finite; others keep theirs."""
    xh, wt = tie_layer(3)
    call = Call(m, 1, T, H, I, E, 1, 0, wt)
    x = m.to_device(xh)
    few, whole = bits(call(x)).copy(), bits(forward(m, call, x)).copy()
    wt["s1"][[2, 5]], wt["s3"][[2, 5]] = 2.0 ** 70, 2.0 ** 70
    call = Call(m, 1, T, H, I, E, 1, 0, wt)
    for got, want in ((bits(call(x)).copy(), few), (bits(forward(m, call, x)), whole)):
        keep = [t for t in range(T) if t not in (2, 5)]
        assert np.array_equal(got[keep], want[keep])
        assert not np.isfinite(bf16_bits_to_f64(got[[2, 5]])).any()
