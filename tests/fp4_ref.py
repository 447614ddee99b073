"""Plain 64-bit definitions of the microscaled 4-bit formats and of the layer on
them (numpy, on the CPU), for the tests; they share no code with the library."""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)


def e4m3_table():
    """Value of every E4M3 byte (0x7f and 0xff are NaN)."""
    b = np.arange(256)
    e, m = (b >> 3) & 15, b & 7
    v = np.where(e == 0, m / 8 * 2.0 ** -6, (1 + m / 8) * 2.0 ** (e - 7.0))
    v[(b & 127) == 127] = np.nan
    return np.where(b & 128, -v, v)


def round_codes(v):
    """Nearest E2M1 code of each value: ties to the even code, saturating, sign kept."""
    a = np.abs(v)[..., None]
    d = np.abs(np.minimum(a, 6.0) - E2M1)
    best = d == d.min(-1, keepdims=True)
    even = best & (np.arange(8) % 2 == 0)
    mag = np.where(best.sum(-1) > 1, even.argmax(-1), best.argmax(-1))
    return (mag | np.where(np.signbit(v), 8, 0)).astype(np.uint8)


def pack(c):
    return (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)


def unpack(p):
    return np.stack((p & 15, p >> 4), -1).reshape(*p.shape[:-1], -1)


def code_values(p):
    c = unpack(p)
    return np.where(c & 8, -1.0, 1.0) * E2M1[c & 7]


def mx_quantize(x):
    """(packed codes, E8M0 bytes) of the last axis of x."""
    x = np.asarray(x, np.float64)
    b = x.reshape(*x.shape[:-1], -1, 32)
    top = np.abs(b).max(-1)
    bad = ~np.isfinite(top)
    e = np.clip(np.frexp(np.where((top > 0) & ~bad, top, 4.0))[1] - 3, -127, 127)
    byte = np.where(bad, 255, np.where(top > 0, e + 127, 127)).astype(np.uint8)
    v = np.where(bad[..., None], 0.0, b) * 2.0 ** -np.where(bad, 0, byte.astype(int) - 127)[..., None].astype(np.float64)
    c = np.where(bad[..., None], 0, round_codes(v)).astype(np.uint8)
    return pack(c.reshape(x.shape)), byte


def mx_values(codes, scales):
    s = np.where(scales == 255, np.nan, 2.0 ** (scales.astype(np.float64) - 127))
    return code_values(codes) * np.repeat(s, 32, -1)


def nv_quantize(x, g):
    """(packed codes, E4M3 bytes) of x [n, rows, k] with global scales g [n]."""
    x = np.asarray(x, np.float64)
    b = x.reshape(*x.shape[:-1], -1, 16)
    gg = np.asarray(g, np.float64).reshape(-1, 1, 1)
    top = np.abs(b).max(-1)
    with np.errstate(divide="ignore", invalid="ignore"):
        q = np.minimum(top / (6 * gg), 448.0)
    bad = ~np.isfinite(top) | ~(np.isfinite(gg) & (gg > 0))
    pos = e4m3_table()[:127]  # ascending
    q = np.where(bad, 0.0, q)
    hi = np.clip(np.searchsorted(pos, q), 1, 126)
    lo = hi - 1
    mid = (pos[lo] + pos[hi]) / 2
    byte = np.where(q > mid, hi, np.where(q < mid, lo, np.where(lo % 2 == 0, lo, hi)))
    s = pos[byte]
    ok = ~bad & (s > 0)
    v = np.where(ok[..., None], b, 0.0) / np.where(ok, s * np.broadcast_to(gg, s.shape), 1.0)[..., None]
    c = np.where(ok[..., None], round_codes(v), 0).astype(np.uint8)
    return pack(c.reshape(x.shape)), np.where(bad, 127, byte).astype(np.uint8)


def nv_values(codes, scales, g):
    return code_values(codes) * np.repeat(e4m3_table()[scales], 16, -1) * np.asarray(g, np.float64).reshape(-1, 1, 1)


def fp8_values(x):
    """x as E4M3 codes times one fp32 scale per 128 inputs (blockmax / 448, quotients in fp32)."""
    b = np.asarray(x, np.float32).reshape(*x.shape[:-1], -1, 128)
    top = np.abs(b).max(-1, keepdims=True)
    s = np.where(top > 0, top / np.float32(448), np.float32(1)).astype(np.float32)
    q = np.abs(b / s).astype(np.float64)
    ulp = 2.0 ** (np.maximum(np.frexp(q)[1] - 1, -6) - 3.0)
    v = np.copysign(np.minimum(np.rint(q / ulp) * ulp, 448.0), b)
    return (v * s.astype(np.float64)).reshape(x.shape)


def activations(fmt, x):
    if fmt == "mxfp4":
        return mx_values(*mx_quantize(x))
    return fp8_values(x) if fmt == "fp8" else np.asarray(x, np.float64)


def expert(fmt, a, w1, w3, w2):
    """SwiGLU MLP of rows a (already the storage's activations) on value matrices."""
    g, u = a @ w1.T, a @ w3.T
    return activations(fmt, g / (1 + np.exp(-g)) * u) @ w2.T


def layer(fmt, x, idx, gate, w, shared=None, tokens=None):
    """out [tokens, H] for a routing idx, gate [T, k]; w(e) and shared() give (w1, w3, w2) in 64 bits."""
    tokens = np.arange(x.shape[0]) if tokens is None else tokens
    a = activations(fmt, x[tokens])
    out = np.zeros(a.shape)
    for e in np.unique(idx[tokens]):
        t, j = np.nonzero(idx[tokens] == e)
        out[t] += gate[tokens][t, j][:, None] * expert(fmt, a[t], *w(e))
    if shared is not None:
        out += expert(fmt, a, *shared())
    return out
