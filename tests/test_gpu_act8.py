"""The 8-bit activation operators on the GPU against the fp64 oracle.

Tolerances, from the arithmetic (a rounding is off by at most half a step,
eps / 2 relative to the value: fp32 2^-24, fp16 2^-11, bf16 2^-8):
 - codec: codes, scales and unpacked values equal bit for bit;
 - integer product p: the sum is exact; conversion, two scalings and the bias
   addition round in fp32, the result once;
 - gradients, with S = sum |dy| |x| the sum of the products' magnitudes:
   bfloat16 dy and result: each value rounds to one bfloat16 (2^-8), and the
   tensor core adds 16 products at a time to an fp32 accumulator with
   truncation, at most 2^-22 of S per addition;
   one scale per row: F = dy * scale rounds to fp32 (2^-24) and to fixed
   point, off by half of max|F| / 8355704 (and by a rounding 2^-24 max|F| of
   the factor and of the product) per code; the integer sums are exact, and
   joining and scaling them takes 6 fp32 roundings (2^-24 each);
   groups: value and dy as two halves are off by 2^-22 each and by 2^-39 of
   the tensor's largest, the omitted product of the lower halves is at most
   2^-22; of K / 16 additions per product kind at most 16 are in one
   accumulator; its sum is then added in fp32, once per 256 k.
"""
import numpy as np
import pytest
import torch

from bit_quantized_shampoo_b200 import _lib as L
from oracle import act8_oracle as A

pytestmark = pytest.mark.gpu

DT = {"fp32": torch.float32, "bf16": torch.bfloat16, "fp16": torch.float16}
TINY = {"fp32": 2.0 ** -149, "bf16": 2.0 ** -133, "fp16": 2.0 ** -24}


def _api():
    from bit_quantized_shampoo_b200 import api
    return api


def half_step(dtype):
    return torch.finfo(DT[dtype]).eps / 2


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def data(rows, cols, dtype, seed, pad=0, offset=0, scale=1.0):
    """A rows x cols CUDA matrix inside a larger buffer: pad columns behind
    each row, offset elements before the first; token rows of different
    magnitude, loud channels, a zero row."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((rows, cols)) * np.exp(0.5 * rng.standard_normal((rows, 1))) * scale
    x[:, rng.random(cols) < 0.02] *= 16
    if rows > 4:
        x[rows // 2] = 0
    buf = torch.full((rows * (cols + pad) + offset,), 7.0, dtype=DT[dtype], device="cuda")
    view = buf[offset:].view(rows, cols + pad)[:, :cols]
    view.copy_(torch.from_numpy(x).to(DT[dtype]))
    return view


def stored(rows, cols, seed, group=0, scale=1.0):
    """Codes and scales on the GPU, and as numpy."""
    rng = np.random.default_rng(seed)
    x = (rng.standard_normal((rows, cols)) * np.exp(0.5 * rng.standard_normal((rows, 1))) * scale).astype(np.float32)
    if rows > 4:
        x[rows // 3] = 0
    codes, scales = A.pack(x, group)
    return to_gpu(codes, scales), codes, scales


def to_gpu(codes, scales):
    rows, cols = codes.shape
    room = torch.full((rows, (cols + 15) // 16 * 16), 99, dtype=torch.int8, device="cuda")
    room[:, :cols] = torch.from_numpy(codes)
    return room[:, :cols], torch.from_numpy(scales).cuda()


def same(a, b):
    """Bit for bit, NaN of any kind equal to NaN."""
    a, b = np.asarray(a, np.float32), np.asarray(b, np.float32)
    nan = np.isnan(a) & np.isnan(b)
    return bool(np.all(nan | (a.view(np.uint32) == b.view(np.uint32))))


def within(got, want, tol):
    err = np.abs(got - want)
    bad = ~(err <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4].tolist(), got[bad][:4], want[bad][:4], (err / np.maximum(tol, 1e-300)).max())


# ------------------------------------------------------------------- codec

def check_codec(x, group, dtype):
    api = _api()
    want_c, want_s = A.pack(x.float().cpu().numpy(), group)
    codes, scales = api.act8_pack(x, group=group)
    assert np.array_equal(codes.cpu().numpy(), want_c)
    assert same(scales.cpu().numpy(), want_s)
    for out in ("fp32", dtype):
        back = api.act8_unpack(codes, scales, group=group, dtype=DT[out])
        want = torch.from_numpy(A.unpack32(want_c, want_s, group)).to(DT[out])
        assert same(back.float().cpu().numpy(), want.float().numpy())


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("group", [0, 32, 64, 128, 256])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (3, 31), (2, 33), (5, 256), (9, 257), (17, 2048), (3, 2049),
                                       (4, 4104), (2, 8200), (2, 16385)])
def test_codec(rows, cols, group, dtype):
    check_codec(data(rows, cols, dtype, rows * 1000 + cols), group, dtype)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("group", [0, 64])
@pytest.mark.parametrize("pad,offset", [(3, 0), (8, 0), (0, 1), (5, 3)])
def test_codec_strides_and_alignment(pad, offset, group, dtype):
    check_codec(data(6, 523, dtype, 5, pad, offset), group, dtype)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("group", [0, 32])
def test_codec_special_groups(group, dtype):
    rows = [np.zeros(96), np.full(96, 254.0), np.arange(96) - 48.0]
    for v in (np.nan, np.inf, -np.inf):
        r = np.ones(96)
        r[37] = v
        rows.append(r)
    r = np.ones(96)
    r[3], r[5] = np.nan, np.inf
    rows.append(r)
    top = float(torch.finfo(DT[dtype]).max)
    low = {"fp32": 2.0 ** -149, "bf16": 2.0 ** -133, "fp16": 2.0 ** -24}[dtype]
    rows += [np.linspace(-top, top, 96), np.linspace(-1, 1, 96) * low * 7, np.full(96, -low)]
    rows.append(np.where(np.arange(96) % 2 == 0, 127.0, 0.5))          # ties at 0.5
    rows.append((np.arange(96) - 48.0) * 2.0)                           # largest 96: exact multiples
    r = np.arange(-48, 48) + 0.0
    r[0] = 254.0                                                         # x / 2: every odd value a tie
    rows.append(r)
    check_codec(torch.from_numpy(np.stack(rows)).to(DT[dtype]).cuda(), group, dtype)


def test_codec_near_every_border():
    """fp32 values one and two steps around each border between two codes."""
    rows = []
    for a in (1.0, 1.7, 254.0, 3.0e-20, 1.1e-38, 3.0e38):
        a = np.float32(a)
        mid = ((np.arange(127) + 0.5) * np.float64(a) / 127.0).astype(np.float32)
        near = [mid]
        for _ in range(2):
            near.append(np.nextafter(near[-1], np.float32(np.inf)))
        lower = mid
        for _ in range(2):
            lower = np.nextafter(lower, np.float32(0))
            near.append(lower)
        r = np.concatenate(near + [-near[1], [a]]).astype(np.float32)
        rows.append(r)
    x = torch.from_numpy(np.stack(rows)).cuda()
    check_codec(x, 0, "fp32")


def test_pack_leaves_what_is_outside():
    api = _api()
    x = data(5, 100, "bf16", 3)
    room = torch.full((8, 128), 55, dtype=torch.int8, device="cuda")
    scales = torch.full((5, 1), -1.0, device="cuda")
    api.act8_pack(x, codes=room[1:6, :100], scales=scales)
    assert torch.all(room[0] == 55) and torch.all(room[6:] == 55) and torch.all(room[:, 100:] == 55)
    out = torch.full((7, 110), 9.0, device="cuda")
    api.act8_unpack(room[1:6, :100], scales, out=out[1:6, 3:103])
    assert torch.all(out[0] == 9) and torch.all(out[6] == 9) and torch.all(out[:, :3] == 9) and torch.all(out[:, 103:] == 9)


# --------------------------------------------------------- integer product

def check_product(y, xc, xs, wc, ws, bias, dtype):
    p, want = A.matmul(xc, xs, wc, ws, bias)
    tol = 1.01 * (3 * 2.0 ** -24 * np.abs(p) + 2.0 ** -24 * np.abs(want) + half_step(dtype) * np.abs(want)) + TINY[dtype]
    within(f64(y), want, tol)


@pytest.mark.parametrize("tokens,out,inner", [
    (1, 1, 1), (1, 64, 64), (2, 7, 15), (3, 257, 127), (16, 300, 128), (17, 128, 129), (31, 255, 640), (33, 1000, 96),
    (64, 512, 1000), (65, 130, 4096), (48, 4100, 2050), (1, 4096, 4096), (13, 11008, 512), (127, 256, 256), (128, 256, 385), (129, 257, 768), (300, 513, 1111), (700, 40, 2304)])
@pytest.mark.parametrize("dtype", list(DT))
def test_matmul(tokens, out, inner, dtype):
    api = _api()
    x, xc, xs = stored(tokens, inner, tokens)
    w, wc, ws = stored(out, inner, out + 1, scale=0.05)
    bias = np.random.default_rng(2).standard_normal(out).astype(np.float32) if inner % 2 else None
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = api.act8_matmul(*x, *w, bias=None if bias is None else torch.from_numpy(bias).cuda(), dtype=DT[dtype],
                        flags=flags)
    check_product(y, xc, xs, wc, ws, bias, dtype)
    assert int(flags.item()) == 0


@pytest.mark.parametrize("tokens", [1, 5, 40])
def test_matmul_longest_inner_sum_is_exact(tokens):
    """All codes 127 over 2^17 columns: the integer sum 127^2 2^17 is just
    below 2^31."""
    api = _api()
    inner, out = 1 << 17, 3
    xc = np.full((tokens, inner), 127, np.int8)
    wc = np.full((out, inner), 127, np.int8)
    wc[1] = -127
    one = lambda n: np.ones((n, 1), np.float32)      # noqa: E731
    y = api.act8_matmul(*to_gpu(xc, one(tokens)), *to_gpu(wc, one(out)), dtype=torch.float32)
    want = np.tile(np.float32(127 * 127 * inner) * np.array([1, -1, 1], np.float32), (tokens, 1))
    assert np.array_equal(y.cpu().numpy(), want)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("tokens", [1, 9, 130])
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (3, 1)])
def test_linear(tokens, pad, offset, dtype):
    api = _api()
    x = data(tokens, 523, dtype, 40 + tokens, pad, offset)
    w, wc, ws = stored(261, 523, 41, scale=0.05)
    bias = torch.randn(261, device="cuda")
    xc, xs = A.pack(x.float().cpu().numpy())
    room = torch.full((tokens, 270), 3.0, dtype=DT[dtype], device="cuda")
    y, codes, scales = api.act8_linear(x, *w, bias=bias, out=room[:, 5:266], checkpoint=True)
    assert np.array_equal(codes.cpu().numpy(), xc) and same(scales.cpu().numpy(), xs)
    check_product(y, xc, xs, wc, ws, bias.cpu().numpy(), dtype)
    assert torch.all(room[:, :5] == 3) and torch.all(room[:, 266:] == 3)
    assert torch.equal(api.act8_linear(x, *w, bias=bias), y)


@pytest.mark.parametrize("tokens", [2, 20])
def test_linear_non_finite_and_zero_rows(tokens):
    api = _api()
    x = data(tokens, 300, "fp32", 8)
    x[0, 17] = float("nan")
    x[1, 5] = float("inf")
    w, wc, ws = stored(70, 300, 9)
    y = api.act8_linear(x, *w)
    assert torch.isnan(y[:2]).all() and torch.isfinite(y[2:]).all()
    z = api.act8_linear(torch.zeros(tokens, 300, device="cuda"), *w)
    assert torch.all(z == 0)


@pytest.mark.parametrize("tokens,out,inner", [(0, 8, 16), (4, 0, 16), (4, 8, 0)])
def test_linear_empty(tokens, out, inner):
    api = _api()
    x = torch.zeros(tokens, inner, device="cuda")
    wc = torch.zeros(out, (inner + 15) // 16 * 16, dtype=torch.int8, device="cuda")[:, :inner]
    ws = torch.zeros(out, 1 if inner else 0, device="cuda")
    bias = torch.arange(out, dtype=torch.float32, device="cuda")
    y = api.act8_linear(x, wc, ws, bias=bias)
    assert tuple(y.shape) == (tokens, out) and torch.equal(y, bias.expand(tokens, out))


# --------------------------------------------------------------- gradients

def grad_tolerance(dy, codes, scales, group, dtype, result, weight):
    a, b = np.abs(dy), np.abs(A.values64(codes, scales, group))
    K = codes.shape[0]
    S = (a.T if weight else a) @ b
    # bfloat16 with one scale per row and few result tiles goes through fixed point
    tiles = -(-S.shape[0] // 256) * -(-S.shape[1] // 256)
    if dtype == "bf16" and result == "bf16" and (group or (S.shape[0] > 640 and tiles >= 48)):
        return S * (1.01 * 2.0 ** -8 + (-(-K // 16) + 1) * 2.0 ** -22)
    if group == 0:
        s = scales.astype(np.float64)
        F = a * (s if weight else s.T)
        top = F.max(axis=0 if weight else 1, initial=0.0).reshape(-1, 1) if F.size else np.zeros((S.shape[0], 1))
        count = np.abs(codes.astype(np.float64)).sum(axis=0, keepdims=True)
        return top * count * (0.5 / 8355704 + 2 * 2.0 ** -24) + S * 7 * 2.0 ** -24
    kinds = 3 if dtype == "fp32" else 2
    floor = 2.0 ** -39 * (a.max(initial=0.0) * (b.sum(axis=0, keepdims=True) if weight else b.max(initial=0.0) * K)
                          + b.max(initial=0.0) * a.sum(axis=0).reshape(-1, 1))
    return S * (4 * 2.0 ** -22 + kinds * 17 * 2.0 ** -22 + (K // 256 + 1) * 2.0 ** -24) + floor


SHAPES = [(1, 1, 1), (1, 64, 300), (2, 7, 17), (63, 130, 65), (64, 128, 256), (65, 256, 257), (200, 129, 520),
          (513, 300, 96), (1100, 64, 128), (30, 1500, 700), (3000, 140, 260), (16, 500, 2900), (17, 2500, 130), (70, 1800, 1700),
          (1800, 90, 1700), (4100, 70, 33), (2000, 300, 90)]
TYPES = [("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"), ("fp32", "fp32"), ("bf16", "fp16"), ("fp32", "bf16")]


@pytest.mark.parametrize("dtype,result", TYPES)
@pytest.mark.parametrize("tokens,out,inner", SHAPES)
def test_weight_grad(tokens, out, inner, dtype, result):
    api = _api()
    group = [0, 32, 128][(tokens + out) % 3]
    dy = data(tokens, out, dtype, 50 + tokens, scale=0.01)
    x, xc, xs = stored(tokens, inner, 51, group)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    dw = api.act8_weight_grad(dy, *x, group=group, dtype=DT[result], flags=flags)
    xv, d = A.values64(xc, xs, group), f64(dy)
    want = d.T @ xv
    within(f64(dw), want, grad_tolerance(d, xc, xs, group, dtype, result, True) + half_step(result) * np.abs(want)
           + TINY[result])
    assert int(flags.item()) == 0


@pytest.mark.parametrize("dtype,result", TYPES)
@pytest.mark.parametrize("tokens,out,inner", SHAPES)
def test_input_grad(tokens, out, inner, dtype, result):
    api = _api()
    dy = data(tokens, out, dtype, 60 + tokens, scale=0.01)
    w, wc, ws = stored(out, inner, 61, scale=0.05)
    dx = api.act8_input_grad(dy, *w, dtype=DT[result])
    wv, d = A.values64(wc, ws), f64(dy)
    want = d @ wv
    within(f64(dx), want, grad_tolerance(d, wc, ws, 0, dtype, result, False) + half_step(result) * np.abs(want)
           + TINY[result])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("pad,offset", [(8, 0), (3, 0), (0, 1)])
def test_grads_strides_and_accumulation(pad, offset, dtype):
    api = _api()
    dy = data(90, 200, dtype, 70, pad, offset, scale=0.01)
    x, xc, xs = stored(90, 133, 71, 64)
    w, wc, ws = stored(200, 133, 72)
    d = f64(dy)
    for weight, codes, scales, group in ((True, xc, xs, 64), (False, wc, ws, 0)):
        vals = A.values64(codes, scales, group)
        rows = 200 if weight else 90
        room = torch.full((rows, 150), 2.0, dtype=DT[dtype], device="cuda")
        out = room[:, 4:137]
        start = torch.randn(rows, 133, device="cuda").to(DT[dtype])
        out.copy_(start)
        if weight:
            api.act8_weight_grad(dy, *x, group=64, out=out, accumulate=True)
        else:
            api.act8_input_grad(dy, *w, out=out, accumulate=True)
        want = f64(start) + (d.T if weight else d) @ vals
        tol = grad_tolerance(d, codes, scales, group, dtype, dtype, weight)
        within(f64(out), want, tol + (2.0 ** -23 + half_step(dtype)) * np.abs(want) + 2.0 ** -23 * np.abs(f64(start))
               + TINY[dtype])
        assert torch.all(room[:, :4] == 2) and torch.all(room[:, 137:] == 2)


@pytest.mark.parametrize("group", [0, 64])
def test_weight_grad_over_a_long_contraction(group):
    """More tokens than an integer sum can take at once: equal signs, the
    largest codes and digits, two and a half sums of 2^17."""
    api = _api()
    tokens = 5 << 16
    dy = torch.full((tokens, 3), 0.5, device="cuda")
    dy[:, 1] = -0.25
    dy[1::2, 2] = -0.5
    codes = torch.full((tokens, 16), 127, dtype=torch.int8, device="cuda")
    scales = torch.full((tokens, 1), 1.0 / 64, device="cuda")
    dw = f64(api.act8_weight_grad(dy, codes, scales, group=group))
    per = 127 / 64 * tokens
    # digits: q = 8355704 for every element but for a few roundings; groups: at most 17 * 3 * 2^-22 of the sum and
    # one rounding per 256 tokens (1280 of them)
    bound = per * (8 * 2.0 ** -24 if group == 0 else 51 * 2.0 ** -22 + 1280 * 2.0 ** -24)
    within(dw, np.tile(np.array([[0.5 * per], [-0.25 * per], [0.0]]), (1, 16)), bound)


def test_offsets_past_32_bits():
    """Matrices of more than 2^32 elements: the last rows against the same
    rows alone."""
    api = _api()
    rows, cols, tail = 66000, 65552, 5
    x = torch.randn(rows, cols, dtype=torch.bfloat16, device="cuda")
    for group in (0, 128):
        codes, scales = api.act8_pack(x, group=group)
        c, s = api.act8_pack(x[-tail:], group=group)
        assert torch.equal(codes[-tail:], c) and torch.equal(scales[-tail:], s)
        back = api.act8_unpack(codes, scales, group=group, dtype=torch.bfloat16)
        assert torch.equal(back[-tail:], api.act8_unpack(c, s, group=group, dtype=torch.bfloat16))
        h, kept = api.act8_swiglu(x, back, group=group)
        h2, kept2 = api.act8_swiglu(x[-tail:], back[-tail:], group=group)
        assert torch.equal(h[-tail:], h2) and all(torch.equal(a[-tail:], b) for a, b in zip(kept, kept2))
        dg, du = api.act8_swiglu_backward(x, kept, group=group)
        dg2, du2 = api.act8_swiglu_backward(x[-tail:], kept2, group=group)
        assert torch.equal(dg[-tail:], dg2) and torch.equal(du[-tail:], du2)
        del back, h, kept, dg, du
    # the result of a product, and each operand of a gradient
    a, b = api.act8_pack(x[:, :128]), api.act8_pack(x[:cols, 128:256])
    y = api.act8_matmul(*a, *b)
    assert torch.equal(y[-tail:], api.act8_matmul(a[0][-tail:], a[1][-tail:], *b))
    del y
    w = api.act8_pack(x[:128])
    dx = api.act8_input_grad(x[:, :128], *w, dtype=torch.float32)
    assert torch.equal(dx[-tail:], api.act8_input_grad(x[-tail:, :128], *w, dtype=torch.float32))
    del dx
    dw = api.act8_weight_grad(x[:128, -300:], *w)
    dw2 = api.act8_weight_grad(x, *api.act8_pack(x[:, :16]), dtype=torch.float32)
    part = api.act8_weight_grad(x[:, -7:], *api.act8_pack(x[:, :16]), dtype=torch.float32)
    assert torch.equal(dw2[-7:], part)
    assert torch.isfinite(dw).all()


def test_grads_empty():
    api = _api()
    x, _, _ = stored(3, 20, 1)
    none = (x[0][:0], x[1][:0])
    dw = api.act8_weight_grad(torch.zeros(0, 6, device="cuda"), *none)
    assert tuple(dw.shape) == (6, 20) and torch.all(dw == 0)
    kept = torch.full((6, 20), 4.0, device="cuda")
    api.act8_weight_grad(torch.zeros(0, 6, device="cuda"), *none, out=kept, accumulate=True)
    assert torch.all(kept == 4)
    dx = api.act8_input_grad(torch.zeros(5, 0, device="cuda"), *none)
    assert tuple(dx.shape) == (5, 20) and torch.all(dx == 0)
    assert api.act8_input_grad(torch.zeros(0, 3, device="cuda"), *x).shape == (0, 20)


@pytest.mark.parametrize("dtype", list(DT))
def test_grads_show_non_finite_inputs(dtype):
    api = _api()
    dy = data(40, 50, dtype, 80, scale=0.01)
    dy[3, 7] = float("inf")
    dy[5, 9] = float("nan")
    x, _, _ = stored(40, 60, 81)
    dw = api.act8_weight_grad(dy, *x, dtype=DT[dtype])
    assert not torch.isfinite(dw[7]).any() and not torch.isfinite(dw[9]).any()
    rest = [i for i in range(50) if i not in (7, 9)]
    assert torch.isfinite(dw[rest]).all()


def test_fp32_gradient_of_huge_values_stays_finite():
    """Values next to fp32's largest: their bfloat16 part must not overflow."""
    api = _api()
    dy = torch.zeros(2, 4, device="cuda")
    dy[0] = 3.4e38
    codes = np.zeros((2, 8), np.int8)
    codes[0] = 127
    scales = np.full((2, 1), 1 / 127, np.float32)
    dw = api.act8_weight_grad(dy, *to_gpu(codes, scales))
    within(f64(dw), np.full((4, 8), float(np.float32(3.4e38)) * 127 * float(scales[0, 0])), 3.4e38 * 2.0 ** -13)


@pytest.mark.parametrize("tokens,out,inner", [(1, 40, 33), (3, 5000, 40), (9, 70, 500), (700, 130, 300), (2000, 7, 64),
                                              (5, 70000, 33), (2, 9, 70000), (300, 2100, 40)])
def test_grouped_gradient_scales_by_the_largest_wherever_it_is(tokens, out, inner):
    """One loud element in dy or in x, in a corner of it: a search that missed
    it would scale it past a half's range."""
    api = _api()
    for t, o, i in ((0, 0, 0), (tokens - 1, out - 1, inner - 1), (tokens // 2, out // 3, inner // 2)):
        dy = data(tokens, out, "fp32", 72)
        dy[t, o] = 1e6
        rng = np.random.default_rng(73)
        x = rng.standard_normal((tokens, inner)).astype(np.float32)
        x[t, i] = -1e6
        codes, scales = A.pack(x, 32)
        dw = api.act8_weight_grad(dy, *to_gpu(codes, scales), group=32)
        want = f64(dy).T @ A.values64(codes, scales, 32)
        within(f64(dw), want, grad_tolerance(f64(dy), codes, scales, 32, "fp32", "fp32", True)
               + half_step("fp32") * np.abs(want) + TINY["fp32"])


@pytest.mark.parametrize("tokens", [60, 1000])                # the contraction whole, and split
def test_grouped_gradient_of_tiny_and_huge_values(tokens):
    """The powers that scale the two operands multiply to more than fp32
    holds, where the result does not."""
    api = _api()
    x, codes, scales = stored(tokens, 96, 70, 32, 1e-20)
    dy = data(tokens, 40, "fp32", 71, scale=1e-18).abs()
    dw = api.act8_weight_grad(dy, *x, group=32)
    want = f64(dy).T @ A.values64(codes, scales, 32)
    within(f64(dw), want, grad_tolerance(f64(dy), codes, scales, 32, "fp32", "fp32", True)
           + half_step("fp32") * np.abs(want))
    assert dw.abs().max() > 1e-37
    x, codes, scales = stored(tokens, 96, 70, 32, 1e30)
    dy = data(tokens, 40, "fp32", 71, scale=1e30)
    dy[:, 3] = 0
    dw = api.act8_weight_grad(dy, *x, group=32)
    # the products overflow (1e60): infinite, or NaN where a split contraction's sums are infinite with both signs
    assert torch.all(dw[3] == 0) and not torch.isfinite(dw[:3]).any() and not torch.isfinite(dw[4:]).any()


# --------------------------------------------------------- gated activation

def swiglu_tol(dtype, want, extra=0.0):
    return (2.0 ** -21 + half_step(dtype)) * np.abs(want) + extra + 2 * TINY[dtype] + 1e-36


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("group", [0, 32, 128])
@pytest.mark.parametrize("rows,cols,pad,offset", [(1, 1, 0, 0), (3, 33, 0, 0), (7, 256, 0, 0), (5, 1023, 0, 0),
                                                  (2, 5000, 0, 0), (4, 300, 8, 0), (4, 300, 5, 3)])
def test_swiglu(rows, cols, pad, offset, group, dtype):
    api = _api()
    gate, up = data(rows, cols, dtype, 90, pad, offset, 2.0), data(rows, cols, dtype, 91, pad, offset)
    room = torch.full((rows, cols + 9), 5.0, dtype=DT[dtype], device="cuda")
    h, kept = api.act8_swiglu(gate, up, group=group, out=room[:, 4:4 + cols])
    g, u = f64(gate), f64(up)
    want = A.swiglu(g, u)
    within(f64(h), want, swiglu_tol(dtype, want))
    assert torch.all(room[:, :4] == 5) and torch.all(room[:, 4 + cols:] == 5)
    vals = []
    for x, c, s in ((gate, kept[0], kept[1]), (up, kept[2], kept[3])):
        want_c, want_s = A.pack(x.float().cpu().numpy(), group)
        assert np.array_equal(c.cpu().numpy(), want_c) and same(s.cpu().numpy(), want_s)
        vals.append(A.values64(want_c, want_s, group))
    dh = data(rows, cols, dtype, 92, pad, offset, 0.01)
    both = torch.full((rows, 2 * cols + 3), 5.0, dtype=DT[dtype], device="cuda")
    dg, du = api.act8_swiglu_backward(dh, kept, group=group, dgate=both[:, :cols], dup=both[:, cols:2 * cols])
    d, (g, u) = f64(dh), vals
    want_g, want_u = A.swiglu_grad(d, g, u)
    s = A.sigmoid(g)
    # code * scale rounds once (2^-24): the gradients move by their derivative in g, at most 1.1 |d u| per unit,
    # and 1 + g (1 - s) cancels near -1.28
    extra = np.abs(d * u) * (s * (np.abs(g) * 2.0 ** -21 + 2.0 ** -23) + np.abs(g) * 2.0 ** -23)
    within(f64(dg), want_g, swiglu_tol(dtype, want_g, extra))
    within(f64(du), want_u, swiglu_tol(dtype, want_u, np.abs(d * g) * 2.0 ** -22 * (s + np.abs(g) * s)))
    assert torch.all(both[:, 2 * cols:] == 5)


def test_swiglu_gradient_against_differences():
    """Inputs that the codec stores exactly: the gradients are those of h."""
    api = _api()
    rng = np.random.default_rng(4)
    gate = np.rint(rng.uniform(-127, 127, (3, 64))) / 32
    up = np.rint(rng.uniform(-127, 127, (3, 64))) / 64
    gate[:, ::32], up[:, ::32] = 127 / 32, 127 / 64               # each group's largest: scale a power of two
    dh = rng.standard_normal((3, 64)).astype(np.float32)
    t = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()   # noqa: E731
    _, kept = api.act8_swiglu(t(gate), t(up), group=32)
    dg, du = api.act8_swiglu_backward(t(dh), kept, group=32)
    e = 1e-5
    num_g = dh * (A.swiglu(gate + e, up) - A.swiglu(gate - e, up)) / (2 * e)
    num_u = dh * (A.swiglu(gate, up + e) - A.swiglu(gate, up - e)) / (2 * e)
    # central differences: e^2 times the third derivative (below 10 here) plus fp64 rounding over e
    within(f64(dg), num_g, 1e-8 + 4e-6 * np.abs(dh) * (1 + np.abs(up)))
    within(f64(du), num_u, 1e-8 + 4e-6 * np.abs(dh) * (1 + np.abs(gate)))


def test_swiglu_saturates():
    api = _api()
    gate = torch.tensor([[-1e4, -200.0, -90.0, 90.0, 1e4, 0.0]], device="cuda")
    up = torch.full_like(gate, 2.0)
    h, kept = api.act8_swiglu(gate, up)
    within(f64(h), A.swiglu(f64(gate), f64(up)), np.abs(A.swiglu(f64(gate), f64(up))) * 2.0 ** -21 + 1e-36)
    dg, du = api.act8_swiglu_backward(torch.ones_like(gate), kept)
    assert torch.isfinite(dg).all() and torch.isfinite(du).all()


def test_swiglu_gradient_where_dh_up_passes_the_range():
    """dh up overflows fp32, dgate does not (gate -60).  The exponential moves
    by 60 times its argument's 2^-24; 16 more roundings of 2^-24 follow."""
    api = _api()
    gate = torch.full((4, 40), -60.0, device="cuda")
    up, dh = torch.full_like(gate, 1e25), torch.full_like(gate, 1e25)
    _, kept = api.act8_swiglu(gate, up, group=32)
    g, u = (A.values64(c.cpu().numpy(), s.cpu().numpy(), 32) for c, s in (kept[:2], kept[2:]))
    dg, du = api.act8_swiglu_backward(dh, kept, group=32)
    want_g, want_u = A.swiglu_grad(f64(dh), g, u)
    within(f64(dg), want_g, np.abs(want_g) * 76 * 2.0 ** -24)
    within(f64(du), want_u, np.abs(want_u) * 76 * 2.0 ** -24)


# ------------------------------------------------------------- used together

def layer(api, x, wg, wu, wd, dy):
    """One gated feed-forward layer, forward and backward, on 8-bit codes."""
    xc, xs = api.act8_pack(x)
    gate = api.act8_matmul(xc, xs, *wg, dtype=x.dtype)
    up = api.act8_matmul(xc, xs, *wu, dtype=x.dtype)
    h, kept = api.act8_swiglu(gate, up)
    y, hc, hs = api.act8_linear(h, *wd, checkpoint=True)
    dh = api.act8_input_grad(dy, *wd)
    dwd = api.act8_weight_grad(dy, hc, hs)
    dgate, dup = api.act8_swiglu_backward(dh, kept)
    dwg = api.act8_weight_grad(dgate, xc, xs)
    dwu = api.act8_weight_grad(dup, xc, xs)
    dx = api.act8_input_grad(dgate, *wg)
    api.act8_input_grad(dup, *wu, out=dx, accumulate=True)
    return y, dx, dwg, dwu, dwd


def _layer_inputs(tokens=70, width=96, hidden=200, dtype="fp32"):
    x = data(tokens, width, dtype, 100)
    ws = [stored(*s, 101 + i, scale=0.1) for i, s in enumerate([(hidden, width), (hidden, width), (width, hidden)])]
    return x, ws, data(tokens, width, dtype, 105, scale=0.01)


def test_layer_matches_the_oracle():
    api = _api()
    x, ws, dy = _layer_inputs()
    got = layer(api, x, *(w[0] for w in ws), dy)
    (wg, wu, wd) = (A.values64(w[1], w[2]) for w in ws)
    xv = A.values64(*A.pack(x.cpu().numpy()))
    # intermediate results in fp32 as the calls return them: their codes are the stages' inputs
    xc = api.act8_pack(x)
    gate, up = (api.act8_matmul(*xc, *w[0], dtype=torch.float32) for w in ws[:2])
    h = api.act8_swiglu(gate, up)[0]
    hv = A.values64(*A.pack(h.cpu().numpy()))
    kept = [A.values64(*A.pack(t.cpu().numpy(), 128), 128) for t in (gate, up)]
    d = f64(dy)
    dg, du = A.swiglu_grad(d @ wd, *kept)
    wants = [hv @ wd.T, dg @ wg + du @ wu, dg.T @ xv, du.T @ xv, d.T @ hv]
    for g, want in zip(got, wants):
        # a stage's bound: with random signs and these lengths (at most 200) the sums of magnitudes, and the rows'
        # largest elements times the codes' counts, are below 16 and 256 times the result; twice over
        assert np.linalg.norm(f64(g) - want) <= 2 * (16 * 7 * 2.0 ** -24 + 256 * 3 * 2.0 ** -24) * np.linalg.norm(want)


def test_layer_gradients_feed_the_optimizer_step():
    api = _api()
    x, ws, dy = _layer_inputs()
    grads = list(layer(api, x, *(w[0] for w in ws), dy)[2:])
    sh = api.Shampoo4([tuple(g.shape) for g in grads])
    sh.update_stats(grads)
    sh.refresh_roots()
    out = sh.precondition(grads)
    # 70 tokens leave statistics of a dimension of 96 or 200 rank-deficient: the informational QR fallback may be up
    assert sh.status_flags() & ~L.FLAG_QR_FALLBACK == 0 and all(torch.isfinite(o).all() for o in out)


def test_weight_grads_of_a_handle():
    """The handle's gradients: those of the calls one by one, micro-batches
    added up, and refusals."""
    api = _api()
    shapes = [(130, 70), (64, 200)]
    sh = api.Shampoo4(shapes)
    dys = [data(50, r, "bf16", 200 + r, scale=0.01) for r, _ in shapes]
    xs = [stored(50, c, 201 + c)[0] for _, c in shapes]
    grads = sh.weight_grads(dys, xs)
    for g, d, k in zip(grads, dys, xs):
        assert torch.equal(g, api.act8_weight_grad(d, *k))
    twice = sh.weight_grads(dys, xs, grads=[g.clone() for g in grads], accumulate=True)
    for a, b in zip(twice, grads):
        assert torch.equal(a, 2 * b)               # g + g rounds to nothing
    sh.update_stats(grads)
    assert sh.status_flags() == 0
    for f in (lambda: sh.weight_grads(dys[:1], xs), lambda: sh.weight_grads(dys, xs[::-1]),
              lambda: sh.weight_grads(dys, xs, accumulate=True), lambda: sh.weight_grads(dys[::-1], xs),
              lambda: sh.weight_grads(dys, xs, grads=[g.t() for g in grads]), lambda: sh.weight_grads(dys, xs, group=32)):
        with pytest.raises((TypeError, ValueError)):
            f()


def test_other_stream_and_graph_replay_match():
    api = _api()
    x, ws, dy = _layer_inputs(dtype="bf16")
    w = [v[0] for v in ws]
    want = [t.clone() for t in layer(api, x, *w, dy)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layer(api, x, *w, dy)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    xin, din = torch.zeros_like(x), torch.zeros_like(dy)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer(api, xin, *w, din)
    for _ in range(2):
        xin.copy_(x)
        din.copy_(dy)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        xin.zero_()
        graph.replay()
    del graph


@pytest.mark.parametrize("tokens,out,inner,dtype,result", [(4, 125, 129, "fp32", "fp32"), (31, 239, 422, "bf16", "bf16"),
                                                           (900, 400, 512, "bf16", "fp32")])
def test_grouped_gradients_back_to_back_and_replayed(tokens, out, inner, dtype, result):
    """Calls that follow each other at once, each with its own inputs (their
    passes overlap), and the same captured and replayed."""
    api = _api()
    ins = [(data(tokens, out, dtype, 80 + k, scale=10.0 ** (k - 1)), *stored(tokens, inner, 90 + k, 64, 10.0 ** (1 - k))[0])
           for k in range(3)]

    def run():
        return [api.act8_weight_grad(dy, c, s, group=64, dtype=DT[result]) for dy, c, s in ins]

    want = []
    for dy, c, s in ins:
        want.append(api.act8_weight_grad(dy, c, s, group=64, dtype=DT[result]))
        torch.cuda.synchronize()
    for _ in range(5):
        got = run()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    del graph


def test_explicit_stream_argument():
    api = _api()
    side = torch.cuda.Stream()
    x, ws, dy = _layer_inputs(dtype="bf16")
    torch.cuda.synchronize()
    y = api.act8_linear(x, *ws[0][0], stream=side)
    c, s = api.act8_pack(x, stream=side)
    dw = api.act8_weight_grad(dy, c, s, stream=side)
    side.synchronize()
    assert torch.equal(y, api.act8_linear(x, *ws[0][0]))
    assert torch.equal(dw, api.act8_weight_grad(dy, c, s))


def test_results_dropped_early_stay_with_the_given_stream():
    """Results made for another stream and dropped at once: what is allocated
    next must not share their memory while that stream still writes."""
    api = _api()
    side = torch.cuda.Stream()
    x = data(4096, 4096, "fp32", 95)
    codes, scales = api.act8_pack(x)
    torch.cuda.synchronize()
    bad = 0
    for _ in range(5):
        for _ in range(4):
            api.act8_unpack(codes, scales, stream=side)
        mark = torch.full((4096, 4096), 3.0, device="cuda")
        side.synchronize()
        bad += int((mark != 3.0).any())
        del mark
    assert bad == 0


def test_two_streams_at_once_do_not_mix():
    api = _api()
    x, ws, dy = _layer_inputs(tokens=300, dtype="bf16")
    w = [v[0] for v in ws]
    x2 = (x.float() * 1.5 + 0.1).to(x.dtype)
    want = [[t.clone() for t in layer(api, v, *w, dy)] for v in (x, x2)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(3):
        for k, v in enumerate((x, x2)):
            with torch.cuda.stream(streams[k]):
                got[k] = layer(api, v, *w, dy)
    torch.cuda.synchronize()
    for g, v in zip(got, want):
        for a, b in zip(g, v):
            assert torch.equal(a, b)


def test_refusals_on_the_device():
    api = _api()
    x = torch.zeros(4, 64, device="cuda")
    c, s = api.act8_pack(x)
    odd = torch.zeros(4, 60, dtype=torch.int8, device="cuda")
    cases = [
        lambda: api.act8_pack(x.t()), lambda: api.act8_pack(x[0]), lambda: api.act8_pack(x.double()),
        lambda: api.act8_pack(x, group=48), lambda: api.act8_pack(x, codes=c),
        lambda: api.act8_pack(x, codes=odd, scales=s), lambda: api.act8_unpack(c, s, group=32),
        lambda: api.act8_unpack(c, s, dtype=torch.float64), lambda: api.act8_unpack(odd, s),
        lambda: api.act8_matmul(c, s, c[:, :32], s), lambda: api.act8_matmul(c, s, c, s, bias=torch.zeros(3).cuda()),
        lambda: api.act8_matmul(c, s, c, s, out=torch.zeros(4, 5, device="cuda")),
        lambda: api.act8_linear(x[:, :32], c, s), lambda: api.act8_weight_grad(x[:3], c, s),
        lambda: api.act8_weight_grad(x, c, s, accumulate=True), lambda: api.act8_input_grad(x, c, s),
        lambda: api.act8_swiglu(x, x.half()), lambda: api.act8_swiglu(x, x[:, :32]),
        lambda: api.act8_swiglu_backward(x.half()[:, :32], (c, s, c, s)),
        lambda: api.act8_matmul(c, s, c, s, flags=torch.zeros(1, device="cuda"))]
    for k, f in enumerate(cases):
        with pytest.raises((TypeError, ValueError)):
            f()
            raise AssertionError(f"case {k} was not refused")
    with pytest.raises(RuntimeError):
        api.act8_pack(x[:1].expand(4, 64))             # overlapping rows
