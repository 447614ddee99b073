"""The whole layer for 1 to 8 tokens (moe_forward_few) on the GPU.

Against the plain 64-bit definition of fp4_ref on every expert storage, within
the layer's tolerances (BF16 outputs 1e-2, FP8 2e-2, relative Frobenius per
token), and against what its own contract promises: a token's bits do not depend
on the other tokens of the call, on the call before, or on how it was launched.
"""
import numpy as np
import pytest

import fp4_ref as ref
import oracle
import synth
from conftest import cuda_available
from parity import bf16_bits_to_f64, check_routing, rows_rel, unique_tokens

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not cuda_available(), reason="needs a CUDA device")]

FMT = {0: "bf16", 1: "fp8", 2: "nvfp4", 3: "mxfp4"}


@pytest.fixture(scope="module")
def m():
    import mixture_experts_histogram_b200 as mm
    from mixture_experts_histogram_b200 import build
    build.build()
    mm.load()
    return mm


def host_weights(w, seed, E, S, H, I, bias=False):
    """Weights of one storage on the host; the values of matrix e as a function."""
    wt = {"router_w": synth.normal_bf16(seed, 1, (E, H), H ** -0.5),
          "router_bias": synth.zipf_bias(seed, E) if bias else None}
    tid = 10
    for pre, n in (("", E), ("s", 1))[: 1 + S]:
        for name, rows, cols in (("1", I, H), ("3", I, H), ("2", H, I)):
            tid += 1
            if w == 0:
                wt[pre + "w" + name] = synth.normal_bf16(seed, tid, (n, rows, cols), cols ** -0.5)
            elif w == 1:
                wt[pre + "w" + name], wt[pre + "s" + name] = synth.fp8_blocks(seed, tid, n, rows, cols, cols ** -0.5)
            elif w == 2:
                wt[pre + "w" + name], wt[pre + "s" + name], wt[pre + "g" + name] = synth.nvfp4(seed, tid, n, rows, cols,
                                                                                              cols ** -0.5)
            else:
                # uniform codes (root mean square 2.93) with scales that give variance 1 / cols
                rng = np.random.default_rng(seed * 100 + tid)
                wt[pre + "w" + name] = rng.integers(0, 256, (n, rows, cols // 2), dtype=np.uint8)
                wt[pre + "s" + name] = (127 + round(np.log2(cols ** -0.5 / 2.93))
                                        + rng.integers(-1, 2, (n, rows, cols // 32))).astype(np.uint8)

    def of(pre):
        def values(e=0):
            out = []
            for n in "132":
                c = wt[pre + "w" + n][e]
                s = wt[pre + "s" + n][e] if w else None
                if w == 0:
                    out.append(synth.bf16_to_f32(c).astype(np.float64))
                elif w == 1:
                    out.append(ref.e4m3_table()[c] * np.kron(s.astype(np.float64), np.ones((128, 128))))
                elif w == 2:
                    out.append(ref.nv_values(c, s, wt[pre + "g" + n][e])[0])
                else:
                    out.append(ref.mx_values(c, s))
            return out
        return values
    return wt, of(""), of("s") if S else None


class Call:
    """One layer and its buffers, called as often as a test likes."""

    def __init__(self, m, w, T, H, I, E, k, S, wt, device="cuda"):
        import torch
        self.m, self.T, self.cfg = m, T, m.make_config(H, E, k, S, I, w)
        self.dev = m.upload_weights(wt, device)
        self.w = m.make_weights(self.dev)
        self.out = torch.full((T + 1, H), 7.0, dtype=torch.bfloat16, device=device)
        self.idx = torch.full((T, k), -1, dtype=torch.int32, device=device)
        self.gate = torch.full((T, k), -1.0, dtype=torch.float32, device=device)
        self.ws = torch.full((m.moe_workspace_bytes(self.cfg, T),), 0xFF, dtype=torch.uint8, device=device)

    def __call__(self, x, stream=None, plain=False):
        self.m.moe_forward_few(self.cfg, self.T, x, self.w, self.out, self.ws, topk_idx=None if plain else self.idx,
                               topk_w=None if plain else self.gate, stream=stream)
        return self.out[: self.T]


def bits(t):
    import torch
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


# T, H, I, E, k, S, bias
SHAPES = [(1, 512, 512, 4, 1, 1, False), (2, 1024, 512, 40, 8, 1, False), (8, 512, 1024, 24, 3, 0, True),
          (3, 512, 512, 5, 5, 1, False), (8, 4096, 1536, 16, 8, 1, False), (5, 512, 512, 512, 16, 1, False), (6, 2560, 512, 20, 4, 1, False),
          (7, 512, 512, 1, 1, 0, False), (8, 512, 512, 200, 16, 1, False), (8, 8192, 512, 2, 1, 1, False),
          (8, 512, 8192, 2, 1, 0, False), (1, 16384, 512, 3, 2, 1, False), (1, 1024, 13824, 1, 1, 0, False)]
SMALL = [(1, 128, 128, 4, 2, 1, False), (8, 384, 640, 9, 2, 1, False), (6, 256, 256, 300, 4, 0, True)]


@pytest.mark.parametrize("w", [0, 1, 2, 3], ids=lambda w: FMT[w])
@pytest.mark.parametrize("T,H,I,E,k,S,bias", SHAPES + SMALL)
def test_few_parity(m, w, T, H, I, E, k, S, bias):
    if w >= 2 and (H % (256, 512)[w - 2] or I % (256, 512)[w - 2]):
        pytest.skip("not a shape of this storage")
    wt, values, shared = host_weights(w, 70 + T, E, S, H, I, bias)
    x = synth.normal_bf16(71, 1, (T, H), 1.0)
    idx_r, gate_r, logits_r = oracle.route(x, wt["router_w"], wt["router_bias"], k, want_logits=True)
    call = Call(m, w, T, H, I, E, k, S, wt)
    got = bf16_bits_to_f64(bits(call(m.to_device(x))))
    assert m.moe_read_status(call.ws) == 0
    check_routing(call.idx.cpu().numpy(), call.gate.cpu().numpy(), logits_r, idx_r, gate_r)
    toks = np.flatnonzero(unique_tokens(logits_r, k))
    want = ref.layer(FMT[w], synth.bf16_to_f32(x).astype(np.float64), idx_r, gate_r, values, shared, toks)
    per = rows_rel(got[toks], want)
    print(f"{FMT[w]} T={T}: per-token max {per.max():.2e}")
    assert per.max() < (2e-2 if w == 1 else 1e-2)
    assert (call.out[T] == 7.0).all()  # the row behind the last token


@pytest.mark.parametrize("w", [0, 1, 2, 3], ids=lambda w: FMT[w])
def test_few_is_a_function_of_the_token(m, w):
    """The same bits alone or among others, first or later call, with or without the routing
    outputs, on a side stream, and replayed from a graph whose input changes."""
    import torch
    T, H, I, E, k, S = 6, 1024, 512, 24, 4, 1
    wt, _, _ = host_weights(w, 80, E, S, H, I)
    x = m.to_device(synth.normal_bf16(81, 1, (T, H), 1.0))
    call = Call(m, w, T, H, I, E, k, S, wt)
    first = bits(call(x))
    assert np.array_equal(first, bits(call(x, plain=True)))
    one = Call(m, w, 1, H, I, E, k, S, wt)
    for t in range(T):
        assert np.array_equal(bits(one(x[t:t + 1]))[0], first[t])
    perm = torch.tensor([3, 0, 5, 2, 1, 4], device="cuda")
    assert np.array_equal(bits(call(x[perm].contiguous())), first[perm.cpu().numpy()])
    side = torch.cuda.Stream()
    call.out.fill_(0)
    side.wait_stream(torch.cuda.current_stream())
    call(x, stream=side)
    side.synchronize()
    assert np.array_equal(bits(call.out[:T]), first)
    # a graph: captured once, replayed on other inputs
    buf = x.clone()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call(buf, stream=side)
    buf.copy_(x.flip(0))
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(bits(call.out[:T]), first[::-1])
    g.replay()
    buf.copy_(x)
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(bits(call.out[:T]), first)
    assert m.moe_read_status(call.ws) == 0


def test_few_two_streams_at_once(m):
    """Calls on two streams with a workspace each: cooperative launches, so neither waits on the other forever."""
    import torch
    T, H, I, E, k, S = 4, 1024, 512, 24, 4, 1
    wt, _, _ = host_weights(1, 82, E, S, H, I)
    x = m.to_device(synth.normal_bf16(83, 1, (T, H), 1.0))
    calls = [Call(m, 1, T, H, I, E, k, S, wt) for _ in range(2)]
    first = bits(calls[0](x))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, s in zip(calls, streams):
            c(x, stream=s)
    torch.cuda.synchronize()
    for c in calls:
        assert m.moe_read_status(c.ws) == 0
        assert np.array_equal(bits(c.out[:T]), first)


@pytest.mark.parametrize("w", [0, 1, 2, 3], ids=lambda w: FMT[w])
def test_few_non_finite_tokens_stay_alone(m, w):
    """A token with a NaN or an infinity gives a non-finite row; the others keep their bits."""
    T, H, I, E, k, S = 5, 512, 512, 12, 3, 1
    wt, _, _ = host_weights(w, 84, E, S, H, I)
    xh = synth.normal_bf16(85, 1, (T, H), 1.0)
    call = Call(m, w, T, H, I, E, k, S, wt)
    want = bits(call(m.to_device(xh))).copy()
    bad = xh.copy()
    bad[1, 7], bad[3, 500] = 0x7FC0, 0x7F80
    got = bits(call(m.to_device(bad)))
    keep = [0, 2, 4]
    assert np.array_equal(got[keep], want[keep])
    assert not np.isfinite(bf16_bits_to_f64(got[[1, 3]])).any()
    idx = call.idx.cpu().numpy()
    assert ((idx >= 0) & (idx < E)).all() and all(len(set(r)) == k for r in idx.tolist())
    assert m.moe_read_status(call.ws) == 0


def test_few_ties_and_unrouted_garbage(m):
    """Equal logits go to the lowest experts; an expert full of NaN that nobody chose changes nothing."""
    import torch
    T, H, I, E, k, S = 3, 256, 128, 20, 4, 0
    wt, _, _ = host_weights(0, 86, E, S, H, I)
    wt["router_w"] = np.zeros_like(wt["router_w"])
    wt["router_bias"] = np.zeros(E, np.float32)
    wt["router_bias"][7] = -0.0
    wt["router_bias"][11] = 1.0
    x = m.to_device(synth.normal_bf16(87, 1, (T, H), 1.0))
    call = Call(m, 0, T, H, I, E, k, S, wt)
    first = bits(call(x)).copy()
    assert call.idx.cpu().tolist() == [[11, 0, 1, 2]] * T
    g = call.gate.cpu().numpy()
    e = np.exp([1.0, 0, 0, 0])
    np.testing.assert_allclose(g, np.tile(e / e.sum(), (T, 1)), rtol=1e-6)
    for n in ("w1", "w3", "w2"):
        call.dev[n][5].fill_(float("nan"))
    assert np.array_equal(bits(call(x)), first)
    # an expert that only token 1 chose is NaN: only token 1 is
    wt["router_w"][5, :] = synth.f32_to_bf16(np.full(H, 0.0, np.float32))
    call.dev["router_w"][5] = (x[1].float() * 4 / x[1].float().norm()).to(torch.bfloat16)
    got = bf16_bits_to_f64(bits(call(x)))
    used = (call.idx.cpu().numpy() == 5).any(1)
    assert used[1] and np.isnan(got[used]).all() and np.array_equal(bits(call.out[:T])[~used], first[~used])


def test_few_wait_runs_out(m):
    """With no loads issued every wait ends: the call latches a timeout and the device stays usable."""
    T, H, I, E, k, S = 2, 256, 128, 8, 2, 1
    wt, _, _ = host_weights(0, 88, E, S, H, I)
    x = m.to_device(synth.normal_bf16(89, 1, (T, H), 1.0))
    call = Call(m, 0, T, H, I, E, k, S, wt)
    first = bits(call(x)).copy()
    m.moe_debug_inject(m.MOE_INJECT_GEMM_NO_LOADS, 50_000_000)
    try:
        call(x)
        assert m.moe_read_status(call.ws) == m.MOE_ERR_DEVICE_TIMEOUT
    finally:
        m.moe_debug_inject(m.MOE_INJECT_NONE, 0)
    assert np.array_equal(bits(call(x)), first)
    assert m.moe_read_status(call.ws) == 0


def device_weights(w, seed, E, S, H, I):
    """Random weights of one storage made on the device (variance about 1 / inputs), for tests that
    compare calls with calls."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda").normal_(0, shape[-1] ** -0.5, generator=gen)

    def bytes_of(lo, hi, *shape):
        return torch.randint(lo, hi, shape, dtype=torch.uint8, device="cuda", generator=gen)

    wt = {"router_w": normal(E, H), "router_bias": None}
    for pre, n in (("", E), ("s", 1))[: 1 + S]:
        for name, rows, cols in (("1", I, H), ("3", I, H), ("2", H, I)):
            code, scale, glob = pre + "w" + name, pre + "s" + name, pre + "g" + name
            if w == 0:
                wt[code] = normal(n, rows, cols)
            elif w == 1:
                wt[code] = (normal(n, rows, cols) * 64).to(torch.float8_e4m3fn).view(torch.uint8)
                wt[scale] = torch.full((n, rows // 128, cols // 128), 1 / 64, device="cuda")
            else:  # uniform codes, root mean square 2.93
                wt[code] = bytes_of(0, 256, n, rows, cols // 2)
                if w == 2:
                    wt[scale] = bytes_of(0x30, 0x40, n, rows, cols // 16)  # 0.5 .. 1.9
                    wt[glob] = torch.full((n,), cols ** -0.5 / 3, device="cuda")
                else:
                    mid = 127 + round(np.log2(cols ** -0.5 / 2.93))
                    wt[scale] = bytes_of(mid - 1, mid + 2, n, rows, cols // 32)
    return wt


def device_call(m, w, T, H, I, E, k, S, wt):
    """A Call on weights that are on the device already."""
    call = Call(m, w, T, H, I, E, k, S, {})
    call.dev, call.w = wt, m.make_weights(wt)
    return call


# T, H, I, E, k: the space of x holds 25 to 60 rows of h, and more than 24 experts are chosen
RINGS = [(8, 4096, 512, 200, 8), (5, 4096, 512, 200, 8), (8, 7168, 2048, 48, 8), (8, 4096, 1024, 88, 8)]


@pytest.mark.parametrize("w", [0, 1, 2, 3], ids=lambda w: FMT[w])
@pytest.mark.parametrize("T,H,I,E,k", RINGS)
def test_few_many_rows_of_h(m, w, T, H, I, E, k):
    """Rows of h for more experts than the ring has slots, with room for 25 rows or more (so that the
    slots and not the rows run out): every call gives the bits of one-token calls."""
    import torch
    wt = device_weights(w, 90, E, 1, H, I)
    x = m.to_device(synth.normal_bf16(91, 1, (T, H), 1.0))
    one, call = (device_call(m, w, n, H, I, E, k, 1, wt) for n in (1, T))
    want = torch.cat([one(x[t:t + 1]).clone() for t in range(T)])
    assert torch.isfinite(want.float()).all()
    differ = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(200):
        call.out.fill_(0)
        differ += (call(x).view(torch.int16) != want.view(torch.int16)).sum()
    assert len(set(call.idx.flatten().tolist())) + 1 > 25
    assert differ.item() == 0
    assert m.moe_read_status(call.ws) == 0


@pytest.mark.parametrize("w", [0, 1, 2, 3], ids=lambda w: FMT[w])
def test_few_workspace_of_a_larger_batch(m, w):
    """A 16-token workspace serves the whole layer and the few-token one for 8 tokens; neither
    writes behind the size asked for its own tokens."""
    import torch
    T, H, I, E, k = 8, 1024, 512, 40, 4
    wt = device_weights(w, 92, E, 1, H, I)
    x = m.to_device(synth.normal_bf16(93, 1, (T, H), 1.0))
    call = device_call(m, w, T, H, I, E, k, 1, wt)
    few = call(x).clone()
    whole = torch.empty_like(few)
    m.moe_forward(call.cfg, T, x, call.w, whole, call.ws)
    for nb in (m.moe_workspace_bytes(call.cfg, T), m.moe_workspace_bytes(call.cfg, 16)):
        mem = torch.full((nb + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
        call.ws = mem[:nb]
        assert torch.equal(call(x).view(torch.int16), few.view(torch.int16))
        again = torch.empty_like(whole)
        m.moe_forward(call.cfg, T, x, call.w, again, call.ws)
        assert torch.equal(again.view(torch.int16), whole.view(torch.int16))
        assert (mem[nb:] == 0xA5).all()


@pytest.mark.parametrize("w", [2, 3], ids=lambda w: FMT[w])
def test_few_small_activations_next_to_large_ones(m, w):
    """4-bit storage, where 128 inputs share a power of two: activations at the stated distance below
    the largest of their 128 (NVFP4 2^31, MXFP4 blocks 2^35), whose weights are zero, keep all bits."""
    T, H, I, E, k, S = 3, 1024, 512, 6, 2, 1
    wt, values, shared = host_weights(w, 95, E, S, H, I)
    rng = np.random.default_rng(96)
    big = np.zeros(H, bool)
    if w == 2:
        big[::128] = True
        x = rng.integers(128, 256, (T, H)) * 2.0 ** -7 * rng.choice([-1.0, 1.0], (T, H))  # magnitudes in [1, 2)
        x[:, big] = 1.5 * 2.0 ** 31
    else:
        big.reshape(-1, 32)[::4] = True
        x = rng.choice([1.0, 1.5, 2.0, 3.0, 4.0, 6.0], (T, H)) * rng.choice([-1.0, 1.0], (T, H))
        x[:, 33::32] = 6.0  # every block's largest: scale 1
        x[:, big] = 6.0 * 2.0 ** 35
    for pre in ("", "s"):
        for name in "13":
            c = wt[pre + "w" + name]
            codes = np.stack((c & 15, c >> 4), -1).reshape(*c.shape[:-1], H)
            codes[..., big] = 0
            wt[pre + "w" + name] = (codes[..., 0::2] | (codes[..., 1::2] << 4)).astype(np.uint8)
    wt["router_w"] = np.zeros_like(wt["router_w"])
    wt["router_bias"] = np.arange(E, dtype=np.float32)
    xh = synth.f32_to_bf16(x.astype(np.float32))
    assert np.array_equal(synth.bf16_to_f32(xh), x.astype(np.float32))
    e = np.exp([1.0, 0.0])
    idx, gate = np.tile([E - 1, E - 2], (T, 1)), np.tile(e / e.sum(), (T, 1))
    call = Call(m, w, T, H, I, E, k, S, wt)
    got = bf16_bits_to_f64(bits(call(m.to_device(xh))))
    want = ref.layer(FMT[w], x, idx, gate, values, shared)
    assert m.moe_read_status(call.ws) == 0
    assert rows_rel(got, want).max() < 1e-2


@pytest.mark.parametrize("w", [0, 1, 2, 3], ids=lambda w: FMT[w])
@pytest.mark.parametrize("T,H,I,E,k,S", [(1, 37888, 512, 2, 1, 1), (1, 512, 65536, 2, 2, 0), (2, 32768, 512, 3, 2, 0),
                                         (4, 512, 16384, 3, 2, 0)])
def test_few_largest_layers(m, w, T, H, I, E, k, S):
    """The ends of the sizes that always fit: 256 output rows a CTA, one row of h at a time."""
    import torch
    wt, values, shared = host_weights(w, 97, E, S, H, I)
    xh = synth.normal_bf16(98, 1, (T, H), 1.0)
    idx_r, gate_r, logits_r = oracle.route(xh, wt["router_w"], None, k, want_logits=True)
    call = Call(m, w, T, H, I, E, k, S, wt)
    x = m.to_device(xh)
    got = bits(call(x)).copy()
    assert m.moe_read_status(call.ws) == 0
    check_routing(call.idx.cpu().numpy(), call.gate.cpu().numpy(), logits_r, idx_r, gate_r)
    toks = np.flatnonzero(unique_tokens(logits_r, k))
    want = ref.layer(FMT[w], synth.bf16_to_f32(xh).astype(np.float64), idx_r, gate_r, values, shared, toks)
    assert rows_rel(bf16_bits_to_f64(got)[toks], want).max() < (2e-2 if w == 1 else 1e-2)
    for _ in range(50):
        assert torch.equal(call(x).view(torch.int16).cpu(), torch.from_numpy(got.view(np.int16)))
