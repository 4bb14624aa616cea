"""Plain 64-bit implementations of the norm, E4M3 and expert product operators, for their tests."""

import numpy as np


def blocks(n):
    return (n + 127) // 128


# ---------------------------------------------------------------------------------- E4M3

def _e4m3_table():
    v = np.zeros(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = (m / 8) * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
        if c & 127 == 127:
            x = np.nan
        v[c] = -x if c & 128 else x
    return v


E4M3 = _e4m3_table()


def decode(codes):
    return E4M3[np.asarray(codes, np.uint8)]


def encode(q):
    """E4M3FN codes of values within +-448, to nearest, ties to even."""
    q = np.asarray(q, np.float64)
    a = np.abs(q)
    e = np.maximum(np.floor(np.log2(np.maximum(a, 2.0 ** -6))), -6)
    k = np.rint(a / 2.0 ** (e - 3))  # in eighths of 2^e (np.rint: ties to even)
    code = np.where(k < 8, k, k + 8 * (e + 6)).astype(np.int64)  # the carry runs into the exponent
    return np.where(np.signbit(q), code | 128, code).astype(np.uint8)


def quantize_fp8(x):
    """(codes, scales float32 [N, blocks]) of rows whose values are fp32 or 16-bit ones."""
    x = np.asarray(x, np.float32)
    N, H = x.shape
    codes = np.zeros((N, H), np.uint8)
    scales = np.zeros((N, blocks(H)), np.float32)
    for b in range(blocks(H)):
        v = x[:, b * 128:(b + 1) * 128]
        nan = np.isnan(v).any(1)
        inf = np.isinf(v).any(1) & ~nan
        with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
            s = (np.abs(v).max(1) / np.float32(448)).astype(np.float32)
            q = (v / s[:, None]).astype(np.float32)
        s[nan] = np.nan
        q = np.where(s[:, None] == 0, np.copysign(0, v), q)
        q = np.where(np.isfinite(q), q, 0)
        c = encode(np.clip(q, -448, 448))
        c = np.where(inf[:, None], np.where(np.isinf(v), 0x7F, np.where(np.signbit(v), 0x80, 0)), c)
        codes[:, b * 128:(b + 1) * 128] = np.where(nan[:, None], 0x7F, c)
        scales[:, b] = s
    return codes, scales


# ---------------------------------------------------------------------------------- norm

def norm(x, w, eps, residual=None):
    """(y, h) in float64; eps is the fp32 value that the call takes."""
    eps = np.float64(np.float32(eps))
    h = np.asarray(x, np.float64)
    if residual is not None:
        h = h + np.asarray(residual, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        return h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * np.asarray(w, np.float64), h


def norm_backward(x, w, g, eps, through=None):
    """(grad_x, grad_w, bound of grad_x's terms, bound of grad_w's terms)."""
    eps = np.float64(np.float32(eps))
    x, w, g = (np.asarray(v, np.float64) for v in (x, w, g))
    r = 1 / np.sqrt((x * x).mean(1, keepdims=True) + eps)
    n = x * r
    gw = g * w
    d = r * (gw - n * (gw * n).mean(1, keepdims=True))
    size = r * (np.abs(gw) + np.abs(n) * np.abs(gw * n).mean(1, keepdims=True))
    if through is not None:
        d = d + np.asarray(through, np.float64)
    return d, (g * n).sum(0), size, np.abs(g * n).sum(0)


# ------------------------------------------------------------------------------- products

def silu(x):
    with np.errstate(over="ignore"):
        return x / (1 + np.exp(-x))


def silu_grad(x):
    with np.errstate(over="ignore"):
        p = 1 / (1 + np.exp(-x))
    return p * (1 + x * (1 - p))


def spread(scales, inner):
    """Scales of blocks of 128 on the last axis, one for each channel."""
    return np.repeat(np.asarray(scales, np.float64), 128, -1)[..., :inner]


def weight_scales(ws, outer, inner, gated):
    """[blocks, blocks] -> [outer, inner]; gated: each half of the channels has blocks of its own."""
    halves = np.split(np.asarray(ws, np.float64), 2) if gated else [np.asarray(ws, np.float64)]
    n = outer // len(halves)
    return spread(np.concatenate([np.repeat(h, 128, 0)[:n] for h in halves]), inner)


def gate(y):
    half = y.shape[1] // 2
    return silu(y[:, :half]) * y[:, half:]


def gate_backward(pre, d):
    half = pre.shape[1] // 2
    g, u = pre[:, :half], pre[:, half:]
    return np.concatenate([d * u * silu_grad(g), d * silu(g)], 1)
