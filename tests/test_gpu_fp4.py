"""Microscaled 4-bit storage on the GPU: the quantisers, their inverse, and the
MXFP4 expert GEMMs, against the plain 64-bit definitions of fp4_ref.

The quantisers are correctly rounded, so codes and scale bytes must be equal.
The GEMMs get exact cases first: E2M1 codes with power-of-two scales of a small
range make every product and partial sum an exact fp32 number, so the sums (and
the bf16 output) must equal the definition bit for bit; this pins the nibble
order, the scale layout and both K halves of a scale column. The layer is held
to the tolerance of BF16 outputs, 1e-2 (relative Frobenius, pooled and per token).
"""
import numpy as np
import pytest

import fp4_ref as ref
import oracle
import synth
from conftest import cuda_available
from parity import bf16_bits_to_f64, check_routing, frob_rel, rows_rel, unique_tokens

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]


@pytest.fixture(scope="module")
def m():
    import mixture_experts_histogram_b200 as mm
    from mixture_experts_histogram_b200 import build
    build.build()
    mm.load()
    return mm


def _values(seed, n, rows, k, kind):
    """Inputs as fp32 (bf16-representable for kind bf16): normal values, a matrix of ties,
    blocks of zeros, tiny and huge blocks."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((n, rows, k)).astype(np.float32) * 2.0 ** rng.integers(-20, 20, (n, rows, 1)).astype(np.float32)
    x[0] = rng.integers(-28, 29, (rows, k)) * 0.25          # every midpoint of the code grid
    if rows > 1:
        x[-1, 1] = 0.0
        x[-1, 0, :16] = -0.0
    if rows > 2:
        x[0, 2] = x[0, 2] * np.float32(2.0 ** -130)         # below the smallest E8M0 scale
    if rows > 3:
        x[-1, 3] = np.sign(x[-1, 3]) * np.float32(3.0e38)
    if kind == "bf16":
        x = synth.bf16_to_f32(synth.f32_to_bf16(np.clip(x, -3.3e38, 3.3e38)))
    return x


def _tensor(x, kind):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t.to(torch.bfloat16) if kind == "bf16" else t


SIZES = [(1, 1, 32), (1, 3, 64), (3, 5, 96), (2, 7, 4096), (5, 33, 1536), (1, 700, 512)]


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("n,rows,k", SIZES)
def test_mxfp4_quantize_exact(m, n, rows, k, kind):
    import torch
    x = _values(1, n, rows, k, kind)
    codes = torch.full((n * rows * k // 2 + 16,), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full((n * rows * k // 32 + 16,), 0xAA, dtype=torch.uint8, device="cuda")
    m.moe_quantize_fp4(m.MOE_WDTYPE_MXFP4, n, rows, k, _tensor(x, kind), None, codes, scales)
    c, s = ref.mx_quantize(x)
    assert np.array_equal(scales.cpu().numpy()[:-16], s.ravel())
    assert np.array_equal(codes.cpu().numpy()[:-16], c.ravel())
    assert (codes[-16:] == 0xAA).all() and (scales[-16:] == 0xAA).all()  # nothing behind the end
    y = torch.empty((n, rows, k), dtype=torch.float32, device="cuda")
    m.moe_dequantize_fp4(m.MOE_WDTYPE_MXFP4, n, rows, k, codes, scales, None, y)
    assert np.array_equal(y.cpu().numpy().astype(np.float64), ref.mx_values(c, s))


@pytest.mark.parametrize("kind", ["bf16", "f32"])
@pytest.mark.parametrize("n,rows,k", [(1, 1, 16), (3, 5, 48)] + SIZES[2:])
def test_nvfp4_quantize_exact(m, n, rows, k, kind):
    import torch
    x = _values(2, n, rows, k, kind)
    if rows > 3:
        x[-1, 3] = 1.0  # (a matrix with 3e38 would have only zeros beside it)
    xt = _tensor(x, kind)
    g = torch.empty(n, dtype=torch.float32, device="cuda")
    m.moe_fp4_global_scale(n, rows, k, xt, g)
    amax = np.abs(x).max((1, 2))
    want_g = np.where(amax > 0, amax / np.float32(2688), np.float32(1)).astype(np.float32)
    assert np.array_equal(g.cpu().numpy(), want_g)
    codes = torch.empty((n, rows, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((n, rows, k // 16), dtype=torch.uint8, device="cuda")
    y = torch.empty((n, rows, k), dtype=torch.float32, device="cuda")
    # the matrix's own scale, a power of two (ties everywhere) and one that saturates
    for gs in (want_g, np.full(n, 2.0 ** -6, np.float32), want_g / np.float32(40)):
        m.moe_quantize_fp4(m.MOE_WDTYPE_NVFP4, n, rows, k, xt, m.to_device(gs), codes, scales)
        c, s = ref.nv_quantize(x, gs)
        assert np.array_equal(scales.cpu().numpy(), s)
        assert np.array_equal(codes.cpu().numpy(), c)
        m.moe_dequantize_fp4(m.MOE_WDTYPE_NVFP4, n, rows, k, codes, scales, m.to_device(gs), y)
        assert np.array_equal(y.cpu().numpy(), ref.nv_values(c, s, gs).astype(np.float32))  # one rounding


@pytest.mark.parametrize("kind", ["bf16", "f32"])
def test_nvfp4_borders_of_every_amax(m, kind):
    """Every bf16 mantissa as a matrix's largest value and many others below it: quotients on, and a
    rounding of the global scale away from, the borders between codes and between scales; then global
    scales near the ends of the range."""
    import torch
    rng = np.random.default_rng(91)
    n, rows, k = 128, 6, 256
    x = rng.integers(128, 256, (n, rows, k)).astype(np.float32) * np.exp2(rng.integers(-9, 0, (n, rows, 1))).astype(np.float32)
    x *= np.exp2(rng.integers(-4, 1, (n, rows, k))).astype(np.float32) * rng.choice([-1.0, 1.0], (n, rows, k)).astype(np.float32)
    x[:, 0, 0] = np.arange(128, 256)  # the others are below 128
    xt = _tensor(x, kind)
    g = torch.empty(n, dtype=torch.float32, device="cuda")
    m.moe_fp4_global_scale(n, rows, k, xt, g)
    own = (np.abs(x).max((1, 2)) / np.float32(2688)).astype(np.float32)
    assert np.array_equal(g.cpu().numpy(), own)
    codes = torch.empty((n, rows, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((n, rows, k // 16), dtype=torch.uint8, device="cuda")
    for gs, f in ((own, 1.0), (own * np.float32(2.0 ** 105), 2.0 ** 105), (own * np.float32(2.0 ** -115), 2.0 ** -115)):
        xs = x * np.float32(f)
        m.moe_quantize_fp4(m.MOE_WDTYPE_NVFP4, n, rows, k, _tensor(xs, kind), m.to_device(gs), codes, scales)
        c, sc = ref.nv_quantize(xs, gs)
        assert np.array_equal(scales.cpu().numpy(), sc)
        assert np.array_equal(codes.cpu().numpy(), c)


def test_quantize_non_finite_and_bf16_output(m):
    """A block with an infinity or NaN gets the NaN scale and zero codes; its neighbours do not change."""
    import torch
    x = np.random.default_rng(3).standard_normal((1, 2, 128)).astype(np.float32)
    x[0, 0, 5], x[0, 0, 40], x[0, 1, 127] = np.inf, np.nan, -np.inf
    x = synth.bf16_to_f32(synth.f32_to_bf16(np.where(np.isfinite(x), x, 0)) ) + np.where(np.isfinite(x), 0, x)
    xt = torch.from_numpy(x).cuda().to(torch.bfloat16)
    for fmt, blk in ((m.MOE_WDTYPE_MXFP4, 32), (m.MOE_WDTYPE_NVFP4, 16)):
        g = None if fmt == m.MOE_WDTYPE_MXFP4 else torch.full((1,), 0.01, device="cuda")
        codes = torch.empty((1, 2, 64), dtype=torch.uint8, device="cuda")
        scales = torch.empty((1, 2, 128 // blk), dtype=torch.uint8, device="cuda")
        m.moe_quantize_fp4(fmt, 1, 2, 128, xt, g, codes, scales)
        c, s = ref.mx_quantize(x) if g is None else ref.nv_quantize(x, g.cpu().numpy())
        assert np.array_equal(scales.cpu().numpy(), s) and np.array_equal(codes.cpu().numpy(), c)
        y = torch.empty((1, 2, 128), dtype=torch.bfloat16, device="cuda")
        m.moe_dequantize_fp4(fmt, 1, 2, 128, codes, scales, g, y)
        want = ref.mx_values(c, s) if g is None else ref.nv_values(c, s, g.cpu().numpy())
        got = y.float().cpu().numpy()
        nan = np.isnan(want)
        assert nan.sum() == 3 * blk and np.array_equal(np.isnan(got), nan)
        assert np.array_equal(got[~nan], synth.bf16_to_f32(synth.f32_to_bf16(want[~nan].astype(np.float32))))
    bad = torch.tensor([float("nan")], device="cuda")
    m.moe_quantize_fp4(m.MOE_WDTYPE_NVFP4, 1, 2, 128, xt, bad, codes, scales)
    assert (scales == 0x7F).all() and (codes == 0).all()


# ------------------------------------------------------------ grouped GEMMs --

@pytest.fixture(params=["single", "pair"])
def variant(request, m):
    """The MXFP4 GEMMs on single CTAs, or on pairs of them (same results expected)."""
    m.moe_set_gemm_variant(m.MOE_GEMM_SINGLE if request.param == "single" else m.MOE_GEMM_PAIR)
    yield request.param
    m.moe_set_gemm_variant(m.MOE_GEMM_AUTO)


H, I, E = 1024, 512, 5
COUNTS = [0, 1, 129, 300, 64, 200]  # the shared expert last


def _matrices(seed, G, rows, cols, spread=2):
    """Random E2M1 codes with E8M0 scales 2^-spread .. 2^spread, and their values."""
    rng = np.random.default_rng(seed)
    codes = rng.integers(0, 256, (G, rows, cols // 2), dtype=np.uint8)
    scales = (127 + rng.integers(-spread, spread + 1, (G, rows, cols // 32))).astype(np.uint8)
    return codes, scales, ref.mx_values(codes, scales)


def _setup(m):
    import torch
    cfg = m.make_config(H, E, 2, 1, I, m.MOE_WDTYPE_MXFP4)
    mats = {"1": _matrices(1, E + 1, I, H), "3": _matrices(2, E + 1, I, H), "2": _matrices(3, E + 1, H, I)}
    host = {"router_w": synth.normal_bf16(0, 1, (E, H), 0.05)}
    for n, (c, s, _) in mats.items():
        host["w" + n], host["s" + n], host["sw" + n], host["ss" + n] = c[:E], s[:E], c[E:], s[E:]
    dev = m.upload_weights({k: np.ascontiguousarray(v) for k, v in host.items()})
    offsets = np.concatenate([[0], np.cumsum(COUNTS)]).astype(np.int32)
    R = int(offsets[-1])
    ws = torch.empty(m.moe_workspace_bytes(cfg, -(-R // 3)), dtype=torch.uint8, device="cuda")
    return cfg, dev, {n: v for n, (_, _, v) in mats.items()}, offsets, R, np.repeat(np.arange(E + 1), COUNTS), ws


def test_mxfp4_gate_up_exact(m, variant):
    import torch
    cfg, dev, w, offsets, R, group, ws = _setup(m)
    ac, asc, a = _matrices(4, 1, R, H)
    out = torch.full((R + 1, 2, I), float("nan"), dtype=torch.float32, device="cuda")
    m.moe_grouped_gemm(cfg, m.MOE_STAGE_GATE_UP_RAW, R, m.to_device(offsets), m.to_device(ac[0]), m.to_device(asc[0]),
                       m.make_weights(dev), out, ws)
    assert m.moe_read_status(ws) == 0
    want = np.stack([np.einsum("rk,rnk->rn", a[0], w[n][group]) for n in "13"], 1)
    # multiples of 2^-6, magnitude below 2^18: exact in fp32 in any order
    assert np.abs(want).max() < 2.0 ** 18 and np.array_equal(want * 64, np.rint(want * 64))
    bad = np.argwhere(out[:R].cpu().numpy() != want)
    assert bad.size == 0, f"{len(bad)} sums differ, first {bad[:4].tolist()}"
    assert torch.isnan(out[R]).all()  # nothing behind the last row


def test_mxfp4_gate_up_h(m, variant):
    """h leaves as MXFP4 of silu(gate) * up: equal to the quantised definition but where a value
    sits on a border of the code grid, within fp32 noise, and there one code apart."""
    import torch
    cfg, dev, w, offsets, R, group, ws = _setup(m)
    ac, asc, a = _matrices(4, 1, R, H, spread=0)
    a, asc = a * 2.0 ** -8, asc - 8
    out = torch.zeros((R, I // 2), dtype=torch.uint8, device="cuda")
    osc = torch.zeros((R, I // 32), dtype=torch.uint8, device="cuda")
    m.moe_grouped_gemm(cfg, m.MOE_STAGE_GATE_UP, R, m.to_device(offsets), m.to_device(ac[0]), m.to_device(asc[0]),
                       m.make_weights(dev), out, ws, out_scale=osc)
    assert m.moe_read_status(ws) == 0
    g, u = (np.einsum("rk,rnk->rn", a[0], w[n][group]) for n in "13")
    with np.errstate(over="ignore"):
        c, s = ref.mx_quantize(g / (1 + np.exp(-g)) * u)
    got, got_s = ref.unpack(out.cpu().numpy()).astype(int), osc.cpu().numpy().astype(int)
    assert np.mean(got_s != s) < 1e-4 and np.abs(got_s - s).max() <= 1
    same = np.repeat(got_s == s, 32, -1)
    want = ref.unpack(c).astype(int)
    assert np.mean(got[same] != want[same]) < 1e-4
    assert np.abs((got & 7) - (want & 7))[same].max() <= 1


def test_mxfp4_down_exact(m, variant):
    import torch
    cfg, dev, w, offsets, R, group, ws = _setup(m)
    ac, asc, a = _matrices(5, 1, R, I)
    gate = np.random.default_rng(6).choice(np.array([0.5, 1.0, 2.0], np.float32), R)
    y = torch.full((R + 1, H), 7.0, dtype=torch.bfloat16, device="cuda")
    for row_gate in (gate, None):
        m.moe_grouped_gemm(cfg, m.MOE_STAGE_DOWN, R, m.to_device(offsets), m.to_device(ac[0]), m.to_device(asc[0]),
                           m.make_weights(dev), y, ws, row_gate=None if row_gate is None else m.to_device(row_gate))
        assert m.moe_read_status(ws) == 0
        want = np.einsum("rk,rnk->rn", a[0], w["2"][group])
        if row_gate is not None:
            want = want * gate[:, None]
        got = y.view(torch.int16).cpu().numpy().view(np.uint16)
        bad = np.argwhere(got[:R] != synth.f32_to_bf16(want.astype(np.float32)))
        assert bad.size == 0, f"{len(bad)} outputs differ, first {bad[:4].tolist()}"
        assert (y[R] == 7.0).all()


def mx_weights(m, seed, E, S, H, I, bias=False):
    """Quantised normal weights on the device (by the library) and their values by matrix."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    wt = {"router_w": torch.empty((E, H), dtype=torch.bfloat16, device="cuda").normal_(0, H ** -0.5, generator=gen),
          "router_bias": m.to_device(synth.zipf_bias(seed, E)) if bias else None}
    for pre, n in (("", E), ("s", 1))[: 1 + S]:
        for name, rows, cols in (("1", I, H), ("3", I, H), ("2", H, I)):
            x = torch.empty((n, rows, cols), dtype=torch.bfloat16, device="cuda").normal_(0, cols ** -0.5, generator=gen)
            c = torch.empty((n, rows, cols // 2), dtype=torch.uint8, device="cuda")
            s = torch.empty((n, rows, cols // 32), dtype=torch.uint8, device="cuda")
            m.moe_quantize_fp4(m.MOE_WDTYPE_MXFP4, n, rows, cols, x, None, c, s)
            wt[pre + "w" + name], wt[pre + "s" + name] = c, s
    def of(pre):
        return lambda e=0: [ref.mx_values(wt[pre + "w" + n][e].cpu().numpy(), wt[pre + "s" + n][e].cpu().numpy())
                            for n in "132"]
    return wt, of("") , of("s") if S else None


# T, H, I, E, k, S, bias, sampled tokens
LAYERS = [(40, 512, 512, 16, 2, 1, False, None), (300, 1024, 512, 24, 4, 1, True, 40), (77, 512, 1024, 12, 3, 0, False, None),
          (1, 512, 512, 4, 4, 1, False, None), (1000, 512, 512, 3, 1, 0, True, 40), (64, 4096, 1536, 88, 8, 1, False, 10)]


@pytest.mark.parametrize("T,H,I,E,k,S,bias,sample", LAYERS)
def test_mxfp4_layer_parity(m, T, H, I, E, k, S, bias, sample, variant):
    """Quantise the weights, run the whole layer on them, and compare with the definition."""
    import torch
    wt, w, sh = mx_weights(m, 60 + T, E, S, H, I, bias)
    x = synth.normal_bf16(61, 1, (T, H), 1.0)
    rw = wt["router_w"].view(torch.int16).cpu().numpy().view(np.uint16)
    rb = wt["router_bias"].cpu().numpy() if bias else None
    idx_r, gate_r, logits_r = oracle.route(x, rw, rb, k, want_logits=True)
    cfg = m.make_config(H, E, k, S, I, m.MOE_WDTYPE_MXFP4)
    out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
    idx = torch.empty((T, k), dtype=torch.int32, device="cuda")
    gate = torch.empty((T, k), dtype=torch.float32, device="cuda")
    ws = torch.empty(m.moe_workspace_bytes(cfg, T), dtype=torch.uint8, device="cuda")
    m.moe_forward(cfg, T, m.to_device(x), m.make_weights(wt), out, ws, topk_idx=idx, topk_w=gate)
    assert m.moe_read_status(ws) == 0
    check_routing(idx.cpu().numpy(), gate.cpu().numpy(), logits_r, idx_r, gate_r)
    toks = np.flatnonzero(unique_tokens(logits_r, k))
    if sample:
        toks = np.sort(np.random.default_rng(T).choice(toks, sample, False))
    want = ref.layer("mxfp4", synth.bf16_to_f32(x).astype(np.float64), idx_r, gate_r, w, sh, toks)
    got = bf16_bits_to_f64(out.view(torch.int16).cpu().numpy().view(np.uint16)[toks])
    err, per = frob_rel(got, want), rows_rel(got, want)
    print(f"T={T}: rel Frobenius {err:.2e}, per-token max {per.max():.2e}")
    assert err < 1e-2 and per.max() < 1e-2


def test_mxfp4_nan_tokens_stay_alone(m, variant):
    """A token with a NaN or an infinity gives non-finite rows; the others keep their bits."""
    import torch
    T, H, I, E, k = 50, 512, 512, 6, 2
    wt, _, _ = mx_weights(m, 70, E, 1, H, I)
    cfg = m.make_config(H, E, k, 1, I, m.MOE_WDTYPE_MXFP4)
    ws = torch.empty(m.moe_workspace_bytes(cfg, T), dtype=torch.uint8, device="cuda")
    x = m.to_device(synth.normal_bf16(71, 1, (T, H), 1.0))
    idx = torch.stack([torch.randperm(E, generator=torch.Generator().manual_seed(t))[:k] for t in range(T)]).int().cuda()
    gate = torch.full((T, k), 0.5, device="cuda")
    outs = []
    for bad in (False, True):
        xb = x.clone()
        if bad:
            xb[3, 5], xb[20, 511] = float("nan"), float("-inf")
        y = torch.empty((3 * T, H), dtype=torch.bfloat16, device="cuda")
        pos = torch.empty((T, 3), dtype=torch.int32, device="cuda")
        out = torch.empty((T, H), dtype=torch.bfloat16, device="cuda")
        m.moe_experts(cfg, T, xb, idx, gate, m.make_weights(wt), y, pos, ws)
        m.moe_combine(cfg, T, y, pos, out)
        assert m.moe_read_status(ws) == 0
        outs.append(out.float())
    keep = [t for t in range(T) if t not in (3, 20)]
    assert torch.equal(outs[0][keep], outs[1][keep])
    assert not torch.isfinite(outs[1][[3, 20]]).any()


def test_mxfp4_run_together(m):
    """Quantise, route, experts and combine, the whole forward, the expert-parallel shares, and the
    few-token layer: one layer, and what each entry point gives for it."""
    import torch
    T, H, I, E, k = 8, 1024, 512, 16, 4
    wt, _, _ = mx_weights(m, 72, E, 1, H, I)
    cfg = m.make_config(H, E, k, 1, I, m.MOE_WDTYPE_MXFP4)
    ws = torch.empty(m.moe_workspace_bytes(cfg, T), dtype=torch.uint8, device="cuda")
    x = m.to_device(synth.normal_bf16(73, 1, (T, H), 1.0))
    w = m.make_weights(wt)
    new = lambda *s, d=torch.bfloat16: torch.empty(s, dtype=d, device="cuda")
    whole, staged, few, ep = (new(T, H) for _ in range(4))
    m.moe_forward(cfg, T, x, w, whole, ws)
    idx, gate = new(T, k, d=torch.int32), new(T, k, d=torch.float32)
    m.moe_route(cfg, T, x, wt["router_w"], None, idx, gate, None, ws)
    y, pos = new(5 * T, H), new(T, 5, d=torch.int32)
    m.moe_experts(cfg, T, x, idx, gate, w, y, pos, ws)
    m.moe_combine(cfg, T, y, pos, staged)
    assert torch.equal(whole, staged)
    m.moe_forward_few(cfg, T, x, w, few, ws)
    # Both round bf16 outputs (2^-8 at most each); moe_forward rounds each of the five rows before that.
    err = (few.double() - whole.double()).norm() / whole.double().norm()
    assert err < 1e-2, err
    parts = []
    for e0, e1, t0, t1 in ((0, 6, 0, 3), (6, 16, 3, T)):
        mine = {n: (v[e0:e1].contiguous() if n in ("w1", "w3", "w2", "s1", "s3", "s2") else v) for n, v in wt.items()}
        part = new(T, H, d=torch.float32)
        m.moe_forward_ep_partial(cfg, T, x, m.make_weights(mine), e0, e1, t0, t1, part, ws)
        assert m.moe_read_status(ws) == 0
        parts.append((part, mine))
    m.moe_ep_reduce([p for p, _ in parts], T, H, 0, T, ep)
    # The same bf16 rows added in another order in fp32, then one rounding: a bf16 step apart at most.
    assert ((ep.double() - whole.double()).abs() <= 2.0 ** -7 * whole.double().abs() + 1e-6).all()


def test_mxfp4_from_host_and_replayed(m, variant):
    """The host-buffer entry points, and a graph of the forward replayed on other inputs, give the
    device call's bytes."""
    import torch
    T, H, I, E, k = 200, 1024, 512, 3, 2
    wt, _, _ = mx_weights(m, 81, E, 1, H, I)
    cfg = m.make_config(H, E, k, 1, I, m.MOE_WDTYPE_MXFP4)
    w = m.make_weights(wt)
    ws = torch.empty(m.moe_workspace_bytes(cfg, T), dtype=torch.uint8, device="cuda")
    xs = [m.to_device(synth.normal_bf16(82 + i, 1, (T, H), 1.0)) for i in range(2)]
    want = []
    for x in xs:
        want.append(torch.empty(T, H, dtype=torch.bfloat16, device="cuda"))
        m.moe_forward(cfg, T, x, w, want[-1], ws)
    torch.cuda.synchronize()
    back = torch.zeros(T, H, dtype=torch.bfloat16).pin_memory()
    hosts = [x.cpu().pin_memory() for x in xs]
    m.moe_forward_host(cfg, T, hosts[0], w, back, ws)
    assert torch.equal(back.view(torch.int16), want[0].cpu().view(torch.int16))
    m.moe_forward_host_async(cfg, T, hosts[1], w, back, ws)
    torch.cuda.synchronize()
    assert torch.equal(back.view(torch.int16), want[1].cpu().view(torch.int16))
    x, out = xs[0].clone(), torch.zeros(T, H, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            m.moe_forward(cfg, T, x, w, out, ws)
        for i in (1, 0):
            x.copy_(xs[i])
            g.replay()
            side.synchronize()
            assert torch.equal(out.view(torch.int16), want[i].view(torch.int16))


def test_mxfp4_wait_runs_out(m, variant):
    """With no loads issued every wait ends: a timeout is latched and the device stays usable."""
    import torch
    T, H, I, E, k = 16, 512, 512, 4, 2
    wt, _, _ = mx_weights(m, 74, E, 0, H, I)
    cfg = m.make_config(H, E, k, 0, I, m.MOE_WDTYPE_MXFP4)
    ws = torch.empty(m.moe_workspace_bytes(cfg, T), dtype=torch.uint8, device="cuda")
    x = m.to_device(synth.normal_bf16(75, 1, (T, H), 1.0))
    first, again = (torch.empty((T, H), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    m.moe_forward(cfg, T, x, m.make_weights(wt), first, ws)
    m.moe_debug_inject(m.MOE_INJECT_GEMM_NO_LOADS, 50_000_000)
    try:
        m.moe_forward(cfg, T, x, m.make_weights(wt), again, ws)
        assert m.moe_read_status(ws) == m.MOE_ERR_DEVICE_TIMEOUT
    finally:
        m.moe_debug_inject(m.MOE_INJECT_NONE, 0)
    m.moe_forward(cfg, T, x, m.make_weights(wt), again, ws)
    assert m.moe_read_status(ws) == 0 and torch.equal(first, again)


def test_quantize_beyond_32_bits(m):
    """More than 2^32 values: the last blocks are where they belong."""
    import torch
    n, rows, k = 3, 350_000, 4096
    x = torch.zeros((n, rows, k), dtype=torch.bfloat16, device="cuda")
    x[-1, -1] = torch.arange(k, device="cuda") % 7 - 3
    codes = torch.empty((n, rows, k // 2), dtype=torch.uint8, device="cuda")
    for fmt, blk in ((m.MOE_WDTYPE_MXFP4, 32), (m.MOE_WDTYPE_NVFP4, 16)):
        g = None if blk == 32 else torch.ones(n, device="cuda")
        scales = torch.empty((n, rows, k // blk), dtype=torch.uint8, device="cuda")
        m.moe_quantize_fp4(fmt, n, rows, k, x, g, codes, scales)
        last = x[-1:, -1:].float().cpu().numpy()
        c, s = ref.mx_quantize(last) if blk == 32 else ref.nv_quantize(last, [1.0])
        assert np.array_equal(codes[-1, -1].cpu().numpy(), c[0, 0]) and np.array_equal(scales[-1, -1].cpu().numpy(), s[0, 0])
        assert not codes[-1, -2].any() and not codes[0, 0].any()
        y = torch.empty_like(x)
        m.moe_dequantize_fp4(fmt, n, rows, k, codes, scales, g, y)
        assert torch.equal(y, x)


def test_nvfp4_tiniest_matrices(m):
    """Largest values from the smallest fp32 number up, where amax / 2688 rounds to zero or to few bits:
    the matrices read back as the definition says, not as NaN."""
    import torch
    rng = np.random.default_rng(92)
    top = np.array([1, 2, 3, 700, 1343, 1344, 1345, 2688, 4000, 5000, 100000], np.float64)
    n, rows, k = len(top), 3, 64
    x = np.rint(rng.uniform(-1, 1, (n, rows, k)) * top[:, None, None])
    x[:, 0, 0] = top
    x = (x * 2.0 ** -149).astype(np.float32)
    xt = torch.from_numpy(x).cuda()
    g = torch.empty(n, dtype=torch.float32, device="cuda")
    m.moe_fp4_global_scale(n, rows, k, xt, g)
    steps = np.rint(top / 2688)  # in units of 2^-149; halves go to the even one
    assert np.array_equal(g.cpu().numpy().astype(np.float64) * 2.0 ** 149, np.maximum(steps, 1))
    codes = torch.empty((n, rows, k // 2), dtype=torch.uint8, device="cuda")
    scales = torch.empty((n, rows, k // 16), dtype=torch.uint8, device="cuda")
    y = torch.empty((n, rows, k), dtype=torch.float32, device="cuda")
    m.moe_quantize_fp4(m.MOE_WDTYPE_NVFP4, n, rows, k, xt, g, codes, scales)
    c, s = ref.nv_quantize(x, g.cpu().numpy())
    assert np.array_equal(codes.cpu().numpy(), c) and np.array_equal(scales.cpu().numpy(), s)
    m.moe_dequantize_fp4(m.MOE_WDTYPE_NVFP4, n, rows, k, codes, scales, g, y)
    got = y.cpu().numpy()
    assert np.isfinite(got).all()
    assert np.array_equal(got, ref.nv_values(c, s, g.cpu().numpy()).astype(np.float32))


def test_global_scale_of_empty_matrices(m):
    """Matrices without rows have a scale too: that of zeros."""
    import torch
    g = torch.full((301,), float("nan"), device="cuda")
    m.moe_fp4_global_scale(300, 0, 32, torch.empty((300, 0, 32), device="cuda"), g)
    assert (g[:300] == 1).all() and torch.isnan(g[300])


def test_mxfp4_every_scale_byte(m):
    """Every E8M0 byte with every code: exact in fp32, infinite from 2^128 up, NaN for byte 255."""
    import torch
    codes = np.tile(np.arange(0, 256, 1, dtype=np.uint8).reshape(16, 16), (256, 1, 1))
    scales = np.broadcast_to(np.arange(256, dtype=np.uint8)[:, None, None], (256, 16, 1)).copy()
    y = torch.empty((256, 16, 32), dtype=torch.float32, device="cuda")
    m.moe_dequantize_fp4(m.MOE_WDTYPE_MXFP4, 256, 16, 32, m.to_device(codes), m.to_device(scales), None, y)
    with np.errstate(over="ignore", invalid="ignore"):
        want = ref.mx_values(codes, scales).astype(np.float32)
    got = y.cpu().numpy()
    assert np.array_equal(got, want, equal_nan=True) and np.array_equal(np.isnan(got[255]), np.ones((16, 32), bool))
    assert np.isinf(got[253:255]).any() and np.isfinite(got[:253]).all()
