"""fp64 CPU oracle of the 8-bit activation operators (plain numpy; shares no
code with the CUDA path).

Storage: per group of columns of a row, a = max |x|, scale = fp32(a / 127)
capped so that 127 * scale stays finite, code = the integer nearest to the
exact quotient 127 x / a, ties to even.  The code is decided in exact integer
arithmetic, not by a division."""
from __future__ import annotations

import numpy as np

SCALE_MAX = np.float32(8454659.0 * 2.0 ** 98)


def _spans(cols, group):
    width = group if group else max(cols, 1)
    return [(c, min(c + width, cols)) for c in range(0, cols, width)]


def nearest_code(x, a):
    """rint(127 x / a) for finite fp32 x, a > 0 by comparing 254 |x| with
    (2 k + 1) a in exact integers."""
    x = np.asarray(x, np.float32)
    q = np.rint(127.0 * np.abs(x).astype(np.float64) / np.float64(a))      # a first guess, within one
    out = np.empty(x.shape, np.int64)
    ma, ea = np.frexp(np.float64(a))
    A = int(ma * 2 ** 53)
    flat, guess, res = np.abs(x).ravel(), q.ravel(), out.ravel()
    # only elements near a border need the exact comparison
    frac = 127.0 * flat.astype(np.float64) / np.float64(a)
    near = np.abs(np.abs(frac - np.floor(frac)) - 0.5) < 1e-9
    res[:] = guess
    for i in np.nonzero(near)[0]:
        mx, ex = np.frexp(np.float64(flat[i]))
        X = int(mx * 2 ** 53)
        k = int(np.floor(frac[i]))
        left, right = 254 * X, (2 * k + 1) * A
        if ex >= ea:
            left <<= int(ex - ea)
        else:
            right <<= int(ea - ex)
        res[i] = k + 1 if left > right else (k if left < right else k + (k & 1))
    return (np.sign(x) * out).astype(np.int8)


def pack(x, group=0):
    """(codes int8, scales fp32) of a 2-D fp32 array (16-bit inputs widened)."""
    x = np.asarray(x, np.float32)
    rows, cols = x.shape
    spans = _spans(cols, group)
    codes = np.zeros((rows, cols), np.int8)
    scales = np.zeros((rows, len(spans)), np.float32)
    for r in range(rows):
        for k, (c0, c1) in enumerate(spans):
            v = x[r, c0:c1]
            if np.isnan(v).any():
                scales[r, k] = np.nan
            elif np.isinf(v).any():
                scales[r, k] = np.inf
            else:
                a = np.abs(v).max()
                scales[r, k] = min(np.float32(a) / np.float32(127.0), SCALE_MAX)
                if a > 0:
                    codes[r, c0:c1] = nearest_code(v, a)
    return codes, scales


def unpack32(codes, scales, group=0):
    """The values as the codec defines them: one fp32 multiply."""
    rows, cols = codes.shape
    out = np.zeros((rows, cols), np.float32)
    with np.errstate(invalid="ignore"):
        for k, (c0, c1) in enumerate(_spans(cols, group)):
            out[:, c0:c1] = codes[:, c0:c1].astype(np.float32) * scales[:, k:k + 1]
    return out


def values64(codes, scales, group=0):
    """The stored values without rounding."""
    rows, cols = codes.shape
    out = np.zeros((rows, cols))
    for k, (c0, c1) in enumerate(_spans(cols, group)):
        out[:, c0:c1] = codes[:, c0:c1].astype(np.float64) * scales[:, k:k + 1].astype(np.float64)
    return out


def matmul(xc, xs, wc, ws, bias=None):
    """(product, product + bias) of the scaled integer product."""
    acc = xc.astype(np.int64) @ wc.astype(np.int64).T
    p = acc * xs.astype(np.float64).reshape(-1, 1) * ws.astype(np.float64).reshape(1, -1)
    return p, p if bias is None else p + np.asarray(bias, np.float64)


def sigmoid(x):
    return np.where(x >= 0, 1.0 / (1.0 + np.exp(-np.abs(x))), np.exp(-np.abs(x)) / (1.0 + np.exp(-np.abs(x))))


def swiglu(gate, up):
    gate, up = np.asarray(gate, np.float64), np.asarray(up, np.float64)
    return gate * sigmoid(gate) * up


def swiglu_grad(dh, gate, up):
    dh, gate, up = (np.asarray(t, np.float64) for t in (dh, gate, up))
    s = sigmoid(gate)
    return dh * up * s * (1.0 + gate * (1.0 - s)), dh * gate * s
