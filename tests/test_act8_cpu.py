"""The 8-bit activation operators without a GPU: the oracle's pins, the code
rule of the kernels restated, and the refusals of the C entry points (all
returned before a device is touched)."""
import ctypes as C

import numpy as np
import pytest

from bit_quantized_shampoo_b200 import _lib as L
from oracle import act8_oracle as A

INVALID, WORKSPACE = 1, 5


# ---- the codec's definition

def test_every_code_is_nearest_and_round_trips():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((5, 300)) * np.exp(rng.standard_normal((5, 1)))).astype(np.float32)
    for group in (0, 32, 128):
        codes, scales = A.pack(x, group)
        v = A.values64(codes, scales, group)
        step = np.repeat(scales, group or 300, axis=1)[:, :300].astype(np.float64)
        # half a step, plus the rounding of the scale itself (2^-24 of at most 127 steps)
        assert np.all(np.abs(v - x) <= step * (0.5 + 127 * 2.0 ** -24))
        again, s2 = A.pack(A.unpack32(codes, scales, group), group)
        assert np.array_equal(again, codes)


def test_ties_go_to_even():
    a = np.float32(254.0)                          # 127 x / a = x / 2
    x = np.arange(-254, 255, dtype=np.float32)
    want = np.rint(x.astype(np.float64) / 2)
    assert np.array_equal(A.nearest_code(x, a), want.astype(np.int8))


def test_special_groups():
    x = np.zeros((5, 64), np.float32)
    x[1, 3] = np.nan
    x[2, 4] = -np.inf
    x[3, 5] = np.float32(3.4028235e38)
    x[4, 6] = np.float32(1e-45)
    codes, scales = A.pack(x, 32)
    assert scales[0].tolist() == [0, 0] and not codes[:3].any()
    assert np.isnan(scales[1, 0]) and scales[1, 1] == 0 and np.isposinf(scales[2, 0])
    assert np.isfinite(np.float32(127) * scales[3, 0]) and codes[3, 5] == 127
    assert codes[4, 6] == 127
    assert np.isnan(A.unpack32(codes, scales, 32)[1:3, :32]).all()


def test_scale_cap_is_the_largest_with_a_finite_top_code():
    assert np.isfinite(np.float32(127) * A.SCALE_MAX)
    with np.errstate(over="ignore"):
        assert np.isinf(np.float32(127) * np.nextafter(A.SCALE_MAX, np.float32(np.inf), dtype=np.float32))


def _kernel_code(x, a, ulps, bits):
    """The kernels' rule: factors 4 ulps below and above 127 * rcp(a), rcp
    being off by up to an ulp; products rounded to integers in one step (fp64
    holds the product of two fp32 numbers exactly).  16-bit types take the
    upper one, unless 127 divides a's mantissa; else, where the two disagree,
    the sign of 254 |x| - (2 k + 1) a decides."""
    rcp = np.float32(1.0) / np.float32(a)
    rcp = (rcp.view(np.int32) + np.int32(ulps)).view(np.float32)
    r = (np.float32(127.0) * rcp).view(np.int32)
    lo, hi = ((r + np.int32(d)).view(np.float32) for d in (-4, 4))
    p, q = (np.rint(x.astype(np.float64) * np.float64(f)) for f in (lo, hi))
    if bits < 24 and ((int(np.float32(a).view(np.uint32)) & 0x7FFFFF) | 0x800000) % 127:
        return q.astype(np.int8)
    k = np.minimum(np.abs(p), np.abs(q))
    y = np.abs(x).astype(np.float64)                          # fp64 holds both products exactly
    d = 254.0 * y - (2 * k + 1) * np.float64(a)
    up = (d > 0) | ((d == 0) & (k % 2 == 1))
    return np.where(p == q, p, np.copysign(k + up, x)).astype(np.int8)


@pytest.mark.parametrize("bits", [8, 11, 24])
def test_the_fast_rule_gives_the_exact_code(bits):
    """bits: significand bits of the inputs (bfloat16, half, fp32)."""
    rng = np.random.default_rng(bits)
    for n in range(300):
        m = rng.integers(2 ** (bits - 1), 2 ** bits)
        if n % 10 == 0:                            # mantissas with the factor 127, where every code has ties
            m = m // 127 * 127 or 127
        a = np.float32(np.ldexp(float(m), int(rng.integers(-60, 60))))
        e = np.frexp(np.float64(a))[1] - bits
        x = np.ldexp(rng.integers(-m, m + 1, 400).astype(np.float64), int(e))
        x[::2] = np.ldexp(rng.integers(-2 ** bits, 2 ** bits, 200), int(e) - rng.integers(1, 12, 200))
        x = np.concatenate([x, [float(a) / 2, -float(a) / 2, float(a), 0.0]]).astype(np.float32)
        x = x[np.abs(x) <= a]
        want = A.nearest_code(x, a)
        for ulps in (-1, 0, 1):
            assert np.array_equal(_kernel_code(x, a, ulps, bits), want)


# ---- refusals

def P(v):
    return C.c_void_p(v)


OK16 = 1 << 20            # a well-aligned fake device address: every call below is refused or empty


def _call(fn, *args):
    return getattr(L.lib(), fn)(*args)


def _pack(x=OK16, dt=0, rows=4, cols=64, ldx=64, group=0, codes=OK16, ldc=64, scales=OK16):
    return _call("act8_pack", P(x), dt, rows, cols, ldx, group, P(codes), ldc, P(scales), P(0))


@pytest.mark.parametrize("kw", [
    dict(x=0), dict(codes=0), dict(scales=0), dict(dt=3), dict(dt=-1), dict(rows=-1), dict(cols=-1), dict(ldx=63),
    dict(group=48), dict(group=-1), dict(group=512), dict(codes=OK16 + 8), dict(ldc=72), dict(ldc=48),
    dict(scales=OK16 + 2), dict(x=OK16 + 2), dict(dt=1, x=OK16 + 1), dict(rows=(1 << 30) + 1), dict(cols=(1 << 26) + 1, ldx=1 << 27, ldc=1 << 27)])
def test_pack_refuses(kw):
    assert _pack(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(rows=0), dict(cols=0), dict(rows=0, x=0, codes=0, scales=0)])
def test_empty_pack_does_nothing(kw):
    assert _pack(**kw) == 0


def _unpack(codes=OK16, ldc=64, scales=OK16, rows=4, cols=64, group=0, x=OK16, dt=0, ldx=64):
    return _call("act8_unpack", P(codes), ldc, P(scales), rows, cols, group, P(x), dt, ldx, P(0))


@pytest.mark.parametrize("kw", [dict(x=0), dict(codes=0), dict(scales=0), dict(dt=3), dict(rows=-1), dict(ldx=63),
                                dict(group=7), dict(codes=OK16 + 4), dict(ldc=68)])
def test_unpack_refuses(kw):
    assert _unpack(**kw) == INVALID


def _matmul(xc=OK16, ldxc=64, xs=OK16, wc=OK16, ldwc=64, ws=OK16, bias=0, tokens=4, out=8, inner=64, y=OK16, dt=0,
            ldy=8, flags=0):
    return _call("act8_matmul", P(xc), ldxc, P(xs), P(wc), ldwc, P(ws), P(bias), tokens, out, inner, P(y), dt, ldy,
                 P(flags), P(0))


@pytest.mark.parametrize("kw", [
    dict(xc=0), dict(xs=0), dict(wc=0), dict(ws=0), dict(y=0), dict(tokens=-1), dict(out=-1), dict(inner=-1),
    dict(inner=(1 << 17) + 1, ldxc=1 << 18, ldwc=1 << 18), dict(dt=9), dict(ldy=7), dict(ldxc=60), dict(ldwc=32),
    dict(xc=OK16 + 1), dict(bias=OK16 + 1), dict(flags=OK16 + 2)])
def test_matmul_refuses(kw):
    assert _matmul(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(tokens=0), dict(out=0)])
def test_empty_matmul_does_nothing(kw):
    assert _matmul(**kw) == 0


def _linear(x=OK16, xdt=1, ldx=64, wc=OK16, ldwc=64, ws=OK16, bias=0, tokens=4, out=8, inner=64, xc=OK16, ldxc=64,
            xs=OK16, y=OK16, ydt=1, ldy=8, flags=0):
    return _call("act8_linear", P(x), xdt, ldx, P(wc), ldwc, P(ws), P(bias), tokens, out, inner, P(xc), ldxc, P(xs),
                 P(y), ydt, ldy, P(flags), P(0))


@pytest.mark.parametrize("kw", [
    dict(x=0), dict(xc=0), dict(xs=0), dict(wc=0), dict(ws=0), dict(y=0), dict(xdt=4), dict(ydt=4), dict(ldx=3),
    dict(ldy=3), dict(ldxc=65), dict(tokens=-1), dict(inner=1 << 18, ldx=1 << 18, ldxc=1 << 18, ldwc=1 << 18)])
def test_linear_refuses(kw):
    assert _linear(**kw) == INVALID


def _wgrad(dy=OK16, dt=1, lddy=8, xc=OK16, ldxc=64, xs=OK16, group=0, tokens=4, out=8, inner=64, dw=OK16, res=0,
           lddw=64, acc=0, ws=OK16, n=1 << 30, flags=0):
    return _call("act8_weight_grad", P(dy), dt, lddy, P(xc), ldxc, P(xs), group, tokens, out, inner, P(dw), res, lddw,
                 acc, P(ws), n, P(flags), P(0))


def _igrad(dy=OK16, dt=1, lddy=8, wc=OK16, ldwc=64, w=OK16, tokens=4, out=8, inner=64, dx=OK16, res=0, lddx=64, acc=0,
           ws=OK16, n=1 << 30, flags=0):
    return _call("act8_input_grad", P(dy), dt, lddy, P(wc), ldwc, P(w), tokens, out, inner, P(dx), res, lddx, acc,
                 P(ws), n, P(flags), P(0))


@pytest.mark.parametrize("kw,want", [
    (dict(dy=0), INVALID), (dict(xc=0), INVALID), (dict(xs=0), INVALID), (dict(dw=0), INVALID), (dict(dt=5), INVALID),
    (dict(res=5), INVALID), (dict(group=100), INVALID), (dict(lddy=7), INVALID), (dict(lddw=63), INVALID),
    (dict(ldxc=72), INVALID), (dict(tokens=-4), INVALID), (dict(ws=0), INVALID), (dict(ws=OK16 + 16), INVALID),
    (dict(n=16), WORKSPACE), (dict(flags=OK16 + 1), INVALID)])
def test_weight_grad_refuses(kw, want):
    assert _wgrad(**kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(dy=0), INVALID), (dict(wc=0), INVALID), (dict(w=0), INVALID), (dict(dx=0), INVALID), (dict(dt=5), INVALID),
    (dict(lddy=7), INVALID), (dict(lddx=63), INVALID), (dict(ldwc=72), INVALID), (dict(ws=0), INVALID),
    (dict(n=16), WORKSPACE)])
def test_input_grad_refuses(kw, want):
    assert _igrad(**kw) == want


@pytest.mark.parametrize("kw", [dict(out=0), dict(inner=0), dict(tokens=0, acc=1)])
def test_empty_weight_grad_does_nothing(kw):
    assert _wgrad(**kw) == 0


def test_grad_workspace_sizes():
    n = C.c_size_t()

    def size(weight, dt, res, t, o, i):
        L.call("act8_grad_workspace", weight, dt, res, t, o, i, 128 if weight else 0, C.byref(n))
        return n.value
    assert size(1, L.ACT8_BF16, L.ACT8_BF16, 64, 64, 64) < size(1, L.ACT8_BF16, L.ACT8_FP32, 64, 64, 64) \
        < size(1, L.ACT8_FP32, L.ACT8_FP32, 64, 64, 64)
    assert size(1, 0, 0, 0, 64, 64) == 0
    assert _call("act8_grad_workspace", 1, 7, 0, 1, 1, 1, 0, C.byref(n)) == INVALID
    assert _call("act8_grad_workspace", 1, 0, 0, 1, 1, 1, 5, C.byref(n)) == INVALID
    assert _call("act8_grad_workspace", 1, 0, 0, -1, 1, 1, 0, C.byref(n)) == INVALID
    assert _call("act8_grad_workspace", 1, 0, 0, 1, 1, 1, 0, None) == INVALID


def _swiglu(g=OK16, ldg=64, u=OK16, ldu=64, dt=1, rows=4, cols=64, group=32, h=OK16, ldh=64, gc=OK16, ldgc=64,
            gs=OK16, uc=OK16, lduc=64, us=OK16):
    return _call("act8_swiglu", P(g), ldg, P(u), ldu, dt, rows, cols, group, P(h), ldh, P(gc), ldgc, P(gs), P(uc),
                 lduc, P(us), P(0))


def _swiglu_bwd(dh=OK16, lddh=64, dt=1, gc=OK16, ldgc=64, gs=OK16, uc=OK16, lduc=64, us=OK16, rows=4, cols=64,
                group=32, dg=OK16, lddg=64, du=OK16, lddu=64):
    return _call("act8_swiglu_backward", P(dh), lddh, dt, P(gc), ldgc, P(gs), P(uc), lduc, P(us), rows, cols, group,
                 P(dg), lddg, P(du), lddu, P(0))


@pytest.mark.parametrize("kw", [dict(g=0), dict(u=0), dict(h=0), dict(gc=0), dict(us=0), dict(dt=3), dict(group=31),
                                dict(ldg=63), dict(ldu=63), dict(ldh=63), dict(ldgc=63), dict(uc=OK16 + 8),
                                dict(rows=-1)])
def test_swiglu_refuses(kw):
    assert _swiglu(**kw) == INVALID


@pytest.mark.parametrize("kw", [dict(dh=0), dict(dg=0), dict(du=0), dict(gc=0), dict(us=0), dict(dt=3),
                                dict(group=31), dict(lddh=63), dict(lddg=63), dict(lddu=63), dict(lduc=63)])
def test_swiglu_backward_refuses(kw):
    assert _swiglu_bwd(**kw) == INVALID


def test_empty_swiglu_does_nothing():
    assert _swiglu(rows=0) == 0 and _swiglu_bwd(cols=0) == 0


def test_python_calls_refuse_host_tensors():
    import torch
    from bit_quantized_shampoo_b200 import api
    x = torch.zeros(4, 64)
    c = torch.zeros(4, 64, dtype=torch.int8)
    s = torch.zeros(4, 1)
    for f in (lambda: api.act8_pack(x), lambda: api.act8_unpack(c, s), lambda: api.act8_linear(x, c, s),
              lambda: api.act8_matmul(c, s, c, s), lambda: api.act8_weight_grad(x, c, s),
              lambda: api.act8_input_grad(x.new_zeros(4, 4), c, s), lambda: api.act8_swiglu(x, x),
              lambda: api.act8_swiglu_backward(x, (c, s, c, s))):
        with pytest.raises((TypeError, ValueError)):
            f()
