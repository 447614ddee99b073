"""Microscaled 4-bit storage on the host: the tests' 64-bit definitions against
closed forms and another package's casts, and the refusals, which need no GPU."""
import ctypes

import numpy as np
import pytest

import fp4_ref as ref
import mixture_experts_histogram_b200 as m
import synth
from mixture_experts_histogram_b200 import build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return m.load()


def test_e2m1_rounding():
    """Midpoints go to the even code, everything else to the nearer value, and 6 is the largest."""
    v = np.array([0, 0.25, 0.26, 0.75, 0.74, 1.25, 1.75, 2.5, 3.5, 5, 5.01, 6, 7, 1e30, -0.0, -0.25, -5])
    want = [0, 0, 0.5, 1, 0.5, 1, 2, 2, 4, 4, 6, 6, 6, 6, 0, 0, -4]
    c = ref.round_codes(v)
    got = np.where(c & 8, -1.0, 1.0) * ref.E2M1[c & 7]
    assert np.array_equal(got, want)
    assert np.array_equal(c >> 3, np.signbit(v).astype(np.uint8))
    assert np.array_equal(ref.E2M1, np.abs(synth.e2m1_value_table()[:8]))


def test_e4m3_table():
    t, s = ref.e4m3_table(), synth.e4m3_value_table()
    fin = np.isfinite(t)
    assert fin.sum() == 254 and np.array_equal(t[fin], s[fin].astype(np.float64))


def test_mx_scales():
    """floor(log2(amax)) - 2 on both sides of powers of two, zero blocks, the ends of the range."""
    for amax, byte in ((1.0, 125), (0.99, 124), (6.0, 127), (7.99, 127), (8.0, 128), (0.0, 127), (2.0 ** -126, 0),
                       (2.0 ** -140, 0), (3.4e38, 252), (np.inf, 255), (np.nan, 255)):
        x = np.zeros(32)
        x[7] = amax
        c, s = ref.mx_quantize(x)
        assert s[0] == byte, amax
    x = np.random.default_rng(0).standard_normal(4096)
    v = ref.mx_values(*ref.mx_quantize(x))
    top = np.repeat(np.abs(x).reshape(-1, 32).max(1), 32)
    # a code is off by half a step, at most 1 of the scale (steps of 2), or by 8 - 6 = 2 where it saturates
    assert np.all(np.abs(v - x) <= 2 * 2.0 ** (np.floor(np.log2(top)) - 2))


def test_nv_quantize_follows_the_generator():
    """The same rule as the synthetic NVFP4 weights, which round fp32 quotients: equal but for ties."""
    codes, scales, g = synth.nvfp4(7, 10, 2, 64, 256, 0.1)
    x = synth.bf16_to_f32(synth.normal_bf16(7, 10, (2, 64, 256), 0.1))
    c, s = ref.nv_quantize(x, g)
    assert np.mean(s != scales) < 1e-3 and np.mean(c != codes) < 1e-3


def test_quantize_refusals(lib):
    MX, NV = m.MOE_WDTYPE_MXFP4, m.MOE_WDTYPE_NVFP4
    q = lib.moe_quantize_fp4  # (format, n_mat, rows, k, x_dtype, x, g, codes, scales, stream)
    assert q(MX, 1, 0, 32, 0, None, None, None, None, None) == m.MOE_OK          # nothing to do
    assert q(MX, 0, 4, 32, 0, None, None, None, None, None) == m.MOE_OK
    assert q(m.MOE_WDTYPE_FP8_E4M3, 1, 4, 32, 0, 1024, None, 2048, 4096, None) == m.MOE_ERR_INVALID_ARG
    assert q(MX, 1, 4, 48, 0, 1024, None, 2048, 4096, None) == m.MOE_ERR_UNSUPPORTED_SHAPE
    assert q(NV, 1, 4, 24, 0, 1024, 512, 2048, 4096, None) == m.MOE_ERR_UNSUPPORTED_SHAPE
    assert q(MX, 1, 4, 32, 2, 1024, None, 2048, 4096, None) == m.MOE_ERR_INVALID_ARG
    assert q(MX, -1, 4, 32, 0, 1024, None, 2048, 4096, None) == m.MOE_ERR_INVALID_ARG
    assert q(MX, 1, -4, 32, 0, 1024, None, 2048, 4096, None) == m.MOE_ERR_INVALID_ARG
    assert q(MX, 1, 4, 0, 0, 1024, None, 2048, 4096, None) == m.MOE_ERR_INVALID_ARG
    assert q(MX, 1 << 20, 1 << 20, 32, 0, 1024, None, 2048, 4096, None) == m.MOE_ERR_UNSUPPORTED_SHAPE
    assert q(MX, 1, 4, 32, 0, None, None, 2048, 4096, None) == m.MOE_ERR_INVALID_ARG
    assert q(MX, 1, 4, 32, 0, 1024, None, None, 4096, None) == m.MOE_ERR_INVALID_ARG
    assert q(MX, 1, 4, 32, 0, 1024, None, 2048, None, None) == m.MOE_ERR_INVALID_ARG
    assert q(NV, 1, 4, 32, 0, 1024, None, 2048, 4096, None) == m.MOE_ERR_INVALID_ARG   # NVFP4 without g
    assert q(MX, 1, 4, 32, 0, 1032, None, 2048, 4096, None) == m.MOE_ERR_MISALIGNED
    assert q(MX, 1, 4, 32, 0, 1024, None, 2056, 4096, None) == m.MOE_ERR_MISALIGNED
    d = lib.moe_dequantize_fp4  # (format, n_mat, rows, k, codes, scales, g, y_dtype, y, stream)
    assert d(MX, 1, 4, 32, None, 1024, None, 0, 2048, None) == m.MOE_ERR_INVALID_ARG
    assert d(NV, 1, 4, 32, 512, 1024, None, 0, 2048, None) == m.MOE_ERR_INVALID_ARG
    assert d(MX, 1, 4, 32, 512, 1024, None, 1, 2052, None) == m.MOE_ERR_MISALIGNED
    assert d(MX, 1, 4, 32, 512, 1024, None, 3, 2048, None) == m.MOE_ERR_INVALID_ARG
    a = lib.moe_fp4_global_scale  # (n_mat, rows, k, x_dtype, x, g, stream)
    assert a(1, 4, 32, 0, 1024, None, None) == m.MOE_ERR_INVALID_ARG
    assert a(1, 4, 40, 0, 1024, 512, None) == m.MOE_ERR_UNSUPPORTED_SHAPE
    assert a(1, 4, 32, 0, 1024, 514, None) == m.MOE_ERR_MISALIGNED
    with pytest.raises(ValueError):
        import torch
        m.moe_quantize_fp4(MX, 1, 1, 32, torch.zeros(32, dtype=torch.float16), None, None, None, 0)


def test_mxfp4_layer_refusals(lib):
    n = ctypes.c_size_t(0)
    for field, value in (("hidden", 256), ("inter", 768)):
        cfg = m.make_config(1024, 16, 2, 1, 512, m.MOE_WDTYPE_MXFP4)
        setattr(cfg, field, value)
        assert lib.moe_workspace_bytes(ctypes.byref(cfg), 4, ctypes.byref(n)) == m.MOE_ERR_UNSUPPORTED_SHAPE
    cfg = m.make_config(1024, 16, 2, 1, 512, m.MOE_WDTYPE_MXFP4)
    fake = {k: 1 << 20 for k in m.WEIGHT_FIELDS}

    def call(**kw):
        w = m.moe_weights(*[{**fake, **kw}[k] for k in m.WEIGHT_FIELDS])
        return lib.moe_forward(ctypes.byref(cfg), 4, 1024, ctypes.byref(w), 2048, None, None, 4096, 16, None)
    assert call() == m.MOE_ERR_WORKSPACE_TOO_SMALL                 # everything else is in order
    assert call(g1=None, g3=None, g2=None, sg1=None, sg3=None, sg2=None) == m.MOE_ERR_WORKSPACE_TOO_SMALL
    assert call(s1=None) == call(ss2=None) == call(sw1=None) == m.MOE_ERR_INVALID_ARG
    assert call(s3=(1 << 20) + 8) == call(ss1=(1 << 20) + 8) == m.MOE_ERR_MISALIGNED
    w = m.moe_weights(*[fake[k] for k in m.WEIGHT_FIELDS])
    g = lib.moe_grouped_gemm
    args = (1024, 2048)  # offsets, a
    for stage, a_scale, out_scale, rc in ((m.MOE_STAGE_DOWN, None, None, m.MOE_ERR_INVALID_ARG),
                                          (m.MOE_STAGE_GATE_UP, 4096, None, m.MOE_ERR_INVALID_ARG),
                                          (m.MOE_STAGE_DOWN, 4096 + 8, None, m.MOE_ERR_MISALIGNED)):
        assert g(ctypes.byref(cfg), stage, 4, *args, a_scale, ctypes.byref(w), None, 8192, out_scale, 16384, 1 << 30,
                 None) == rc


def test_few_refusals(lib):
    cfg = m.make_config(1024, 16, 2, 1, 512, m.MOE_WDTYPE_FP8_E4M3)
    fake = {k: 1 << 20 for k in m.WEIGHT_FIELDS}
    w = m.moe_weights(*[fake[k] for k in m.WEIGHT_FIELDS])

    def call(T=4, x=1024, out=2048, idx=None, gate=None, ws=4096, nb=1 << 30, cfg=cfg, w=w):
        return lib.moe_forward_few(ctypes.byref(cfg), T, x, ctypes.byref(w), out, idx, gate, ws, nb, None)
    assert call(nb=16) == m.MOE_ERR_WORKSPACE_TOO_SMALL            # everything else is in order
    assert call(T=0) == m.MOE_OK                                   # nothing to do
    assert call(T=m.MOE_FEW_MAX_TOKENS + 1) == m.MOE_ERR_UNSUPPORTED_SHAPE
    assert call(T=-1) == call(x=None) == call(out=None) == call(ws=None) == m.MOE_ERR_INVALID_ARG
    assert call(idx=8192) == call(gate=8192) == m.MOE_ERR_INVALID_ARG
    assert call(x=1032) == call(out=2056) == call(ws=4096 + 64) == m.MOE_ERR_MISALIGNED
    assert call(w=m.moe_weights(*[None if k == "s2" else fake[k] for k in m.WEIGHT_FIELDS])) == m.MOE_ERR_INVALID_ARG
    # Activations that leave no room for the weights: T * max(H, I) beyond 65,536 by enough.
    for wdtype in range(4):
        for H, I in ((16384, 512), (512, 16384)):
            big = m.make_config(H, 16, 2, 1, I, wdtype)
            assert call(T=8, cfg=big) == m.MOE_ERR_UNSUPPORTED_SHAPE
            assert call(T=4, cfg=big, nb=16) == m.MOE_ERR_WORKSPACE_TOO_SMALL
    assert call(cfg=m.make_config(1024, 16, 17, 1, 512, 0)) == m.MOE_ERR_UNSUPPORTED_SHAPE


def test_few_workspace(lib):
    """The few-token layer's scratch is part of every workspace that it may be called with."""
    cfg = m.make_config(4096, 352, 8, 1, 1536, m.MOE_WDTYPE_FP8_E4M3)
    sizes = [m.moe_workspace_bytes(cfg, T) for T in range(1, 10)]
    assert all(a < b for a, b in zip(sizes[:8], sizes[1:8]))
    assert sizes[7] > 65 * 8 * 1536 * 4  # h of (8 x 8 + 1) experts in fp32


def test_few_sizes_that_always_fit(lib):
    """What moe.h promises: T * max(H, I) <= 65,536 with H <= 256 x 148 is accepted; a larger H is not."""
    fake = m.moe_weights(*[1 << 20 for _ in m.WEIGHT_FIELDS])

    def call(w, T, H, I):
        cfg = m.make_config(H, 16, 2, 1, I, w)
        return lib.moe_forward_few(ctypes.byref(cfg), T, 1024, ctypes.byref(fake), 2048, None, None, 4096, 16, None)
    for w in range(4):
        unit = (128, 128, 256, 512)[w]
        for T in range(1, m.MOE_FEW_MAX_TOKENS + 1):
            most = 65536 // T // unit * unit
            top = min(most, 37888 // unit * unit)
            for H in {unit, top // 2 // unit * unit, top - unit, top}:
                for I in {unit, most // 2 // unit * unit, most}:
                    assert call(w, T, H, I) == m.MOE_ERR_WORKSPACE_TOO_SMALL, (w, T, H, I)  # all else in order
        for H in (37888 // unit * unit + unit, 40960, 65536):
            assert call(w, 1, H, unit) == m.MOE_ERR_UNSUPPORTED_SHAPE, (w, H)


def test_global_scale_of_empty_matrices_refusals(lib):
    a = lib.moe_fp4_global_scale  # (n_mat, rows, k, x_dtype, x, g, stream)
    assert a(0, 0, 32, 1, None, None, None) == a(0, 4, 32, 1, None, None, None) == m.MOE_OK
    assert a(3, 0, 32, 1, None, None, None) == m.MOE_ERR_INVALID_ARG  # three scales to write
    assert a(3, 0, 32, 1, None, 514, None) == m.MOE_ERR_MISALIGNED
    assert a(1 << 40, 0, 32, 1, None, 512, None) == m.MOE_ERR_UNSUPPORTED_SHAPE
