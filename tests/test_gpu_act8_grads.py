"""The gradients of the 8-bit product where their arithmetic could lose
something: results in bfloat16, long contractions, magnitudes far apart.

Tolerances, from the arithmetic (a rounding is off by at most half a step,
eps / 2 relative to the value: fp32 2^-24, fp16 2^-11, bf16 2^-8) are derived
at each test; S is the sum of the products' magnitudes.
"""
import numpy as np
import pytest
import torch

from oracle import act8_oracle as A
from test_gpu_act8 import DT, TINY, data, f64, half_step, stored, to_gpu, within

pytestmark = pytest.mark.gpu


def _api():
    from bit_quantized_shampoo_b200 import api
    return api


def values64(k, group=0):
    """Stored codes and scales as fp64 values on the GPU."""
    codes, scales = k
    cols = codes.shape[1]
    index = torch.arange(cols, device="cuda") // group if group else torch.zeros(cols, dtype=torch.long, device="cuda")
    return codes.double() * scales.double()[:, index]


# ---------------------------------------------------- results in bfloat16

@pytest.mark.parametrize("weight,tokens,out,inner,group", [
    (False, 1100, 1900, 3100, 0), (True, 1900, 1100, 3100, 0), (False, 2100, 1300, 6300, 0), (True, 1300, 2100, 6300, 0),
    (True, 700, 200, 320, 64), (True, 1300, 900, 3200, 128),
    (False, 300, 500, 400, 0)])
def test_bfloat16_gradients_are_the_rounded_result(weight, tokens, out, inner, group):
    """The error is that of rounding the exact result to bfloat16, whatever
    the form that the sizes choose.  Values rounded to a half on the way would
    add 2^-11 / sqrt(3) = 2.8e-4 of a product's magnitude at most (root mean
    square, signs at random), in quadrature to about 2^-8 / sqrt(3) * 0.72 =
    1.6e-3: 1.5%; bounded at 3%."""
    api = _api()
    dy = data(tokens, out, "bf16", 1, scale=0.01)
    k = stored(tokens if weight else out, inner, 2, group)[0]
    v = values64(k, group)
    if weight:
        got, want = api.act8_weight_grad(dy, *k, group=group, dtype=torch.bfloat16), dy.double().t() @ v
    else:
        got, want = api.act8_input_grad(dy, *k), dy.double() @ v
    assert got.dtype == torch.bfloat16
    best = (want.bfloat16().double() - want).norm()
    assert (got.double() - want).norm() <= 1.03 * best


@pytest.mark.parametrize("group", [0, 32])
def test_bfloat16_gradient_of_values_above_its_range(group):
    """Stored values beyond bfloat16's largest number, finite in fp32: their
    products with small gradients are finite, with zeros zero."""
    api = _api()
    codes = np.full((40, 64), 127, np.int8)
    codes[:, 1::2] = -100
    scales = np.full((40, 1 if group == 0 else 2), np.float32(3.4e38) / np.float32(127), np.float32)
    dy = torch.full((40, 24), 2.0 ** -60, dtype=torch.bfloat16, device="cuda")
    dy[:, 5] = 0
    dw = api.act8_weight_grad(dy, *to_gpu(codes, scales), group=group, dtype=torch.bfloat16)
    want = f64(dy).T @ A.values64(codes, scales, group)
    # values as one half at least (2^-11), the digits' step and fp32 sums far below that, and the result's rounding
    within(f64(dw), want, np.abs(want) * (2.0 ** -11 + 2.0 ** -16 + half_step("bf16")))


@pytest.mark.parametrize("group", [0, 64])
def test_bfloat16_gradient_over_millions_of_tokens(group):
    """Terms of one sign: sums that are cut off at each step drift by its
    count.  Beside the result's rounding (2^-8): values as halves (2^-11),
    and fp32 sums joined once per 1024 tokens, rounded to nearest (at random,
    so by the root of their count: 8 standard deviations of sqrt(2^13) 2^-24
    / sqrt(3)), with at most 64 truncated additions of 2^-22 within each."""
    api = _api()
    tokens = 1 << 23
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    codes = torch.randint(90, 128, (tokens, 16), generator=g, dtype=torch.int8, device="cuda")
    scales = torch.full((tokens, 1), 1.0037 / 64, device="cuda")
    dy = torch.rand(tokens, 2, generator=g, device="cuda").add_(0.5).bfloat16()
    got = api.act8_weight_grad(dy, codes, scales, group=group, dtype=torch.bfloat16).double()
    want = dy.double().t() @ (codes.double() * scales.double())
    tol = 2.0 ** -11 + 64 * 2.0 ** -22 + 8 * 2.0 ** 6.5 * 2.0 ** -24 / 3 ** 0.5 + half_step("bf16")
    assert ((got - want).abs() <= tol * want).all()


# ------------------------------------------ magnitudes far apart, in groups

def group_tops(values, cols, group):
    """Per column the largest magnitude that its group of columns reaches
    over all rows, at least (a code may be 126.5 / 127 of its scale's top)."""
    top = np.abs(values).max(axis=0)
    out = np.zeros(cols)
    for c in range(0, cols, group):
        out[c:c + group] = top[c:c + group].max(initial=0.0)
    return out * 1.01


def grouped_tolerance(dy, codes, scales, group, dtype, result):
    """dy and value as two halves (a 16-bit dy as one, exact) are off by 2^-22
    of themselves and by 2^-39 of the largest that dy's column and the value's
    group of columns have over the tokens; the omitted product of the lower
    halves is at most 2^-22; at most 17 truncated additions of 2^-22 for each
    of three kinds of products, a rounding per 256 tokens, and four of the
    factors and of joining up to 32 shares; a bfloat16 result: the value as
    one half (2^-11), 65 additions."""
    v = A.values64(codes, scales, group)
    a, b, tokens = np.abs(dy), np.abs(v), dy.shape[0]
    S = a.T @ b
    floor = 2.0 ** -39 * (a.max(axis=0).reshape(-1, 1) * b.sum(axis=0) + a.sum(axis=0).reshape(-1, 1)
                          * group_tops(v, v.shape[1], group))
    one = dtype == result == "bf16"
    rel = 2.0 ** -11 + 65 * 2.0 ** -22 if one else (4 + 3 * 17) * 2.0 ** -22
    return S * (rel + (tokens // 256 + 36) * 2.0 ** -24) + floor


@pytest.mark.parametrize("dtype,result", [("fp32", "fp32"), ("bf16", "fp32"), ("bf16", "bf16"), ("fp32", "bf16")])
@pytest.mark.parametrize("tokens,out,inner,group", [(70, 24, 96, 32), (1500, 130, 200, 64), (3000, 9, 520, 256)])
def test_grouped_gradient_beside_a_loud_channel(tokens, out, inner, group, dtype, result):
    """One output channel 10^14 times the others, and one group of input
    columns 10^10 times the others: the quiet results are as precise as alone."""
    api = _api()
    rng = np.random.default_rng(tokens)
    dy = rng.standard_normal((tokens, out)) * 1e-8
    dy[:, 2] *= 1e14
    dy[:, 5] = 0
    x = rng.standard_normal((tokens, inner)).astype(np.float32)
    x[:, :group] *= 1e10
    d = torch.from_numpy(dy).to(DT[dtype]).cuda()
    codes, scales = A.pack(x, group)
    got = f64(api.act8_weight_grad(d, *to_gpu(codes, scales), group=group, dtype=DT[result]))
    want = f64(d).T @ A.values64(codes, scales, group)
    within(got, want, grouped_tolerance(f64(d), codes, scales, group, dtype, result)
           + half_step(result) * np.abs(want) + TINY[result])
    assert np.all(got[5] == 0)


@pytest.mark.parametrize("up,down", [(1e36, 1e-30), (1e-30, 1e36), (1e-37, 1e-2), (3e-39, 1.0), (1e-20, 1e-20)])
def test_grouped_gradient_over_the_whole_range(up, down):
    """The factors that undo the two scalings multiply to more than fp32
    holds, or to less, where the result does not; and dy next to fp32's
    smallest numbers keeps its bits (2^126 dy as two halves: a half's smallest
    step is 2^-24, so dy is off by 2^-151, less than its own step)."""
    api = _api()
    rng = np.random.default_rng(7)
    dy = torch.from_numpy((rng.standard_normal((90, 40)) * up)).float().cuda()
    x = (rng.standard_normal((90, 96)) * down).astype(np.float32)
    codes, scales = A.pack(x, 32)
    got = f64(api.act8_weight_grad(dy, *to_gpu(codes, scales), group=32))
    want = f64(dy).T @ A.values64(codes, scales, 32)
    # two factors one after the other may round a subnormal result twice
    within(got, want, grouped_tolerance(f64(dy), codes, scales, 32, "fp32", "fp32")
           + half_step("fp32") * np.abs(want) + 2 * TINY["fp32"])
    assert np.abs(got).max() > 0


@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 0), (3, 1)])
@pytest.mark.parametrize("weight", [False, True])
def test_large_bfloat16_gradients_at_any_magnitude(weight, pad, offset):
    """Tokens (output channels) from 10^-18 to 10^18 side by side, one of them
    zero, weights (inputs) of 10^-12 and 10^12, unaligned rows, into a part of
    a larger result that is added to: each result's row is as precise as
    alone.  One operand as one half (2^-11) and 65 truncated additions of
    2^-22 (K below 2048: twice, and one rounding); an element is never coarser
    than 2^-39 of its row's largest over the contraction."""
    api = _api()
    tokens, out, inner = (1300, 2100, 6300) if weight else (2100, 1300, 6300)
    rng = np.random.default_rng(11)
    size = 10.0 ** rng.integers(-18, 19, out if weight else tokens)
    size[7] = 0
    dy = rng.standard_normal((tokens, out)) * (size if weight else size.reshape(-1, 1))
    room = torch.zeros(tokens * (out + pad) + offset, dtype=torch.bfloat16, device="cuda")
    d = room[offset:].view(tokens, out + pad)[:, :out]
    d.copy_(torch.from_numpy(dy))
    for scale in (1e-12, 1e12):
        k = stored(tokens if weight else out, inner, 12, 0, scale)[0]
        v = values64(k)
        F = d.double() if weight else d.double() * k[1].double().t()      # what is scaled per row of the result
        cols = v if weight else k[0].double()
        want = F.t() @ cols if weight else F @ cols
        S = F.abs().t() @ cols.abs() if weight else F.abs() @ cols.abs()
        K = cols.shape[0]
        top = F.abs().amax(dim=0 if weight else 1).reshape(-1, 1)
        floor = 2.0 ** -39 * top * cols.abs().sum(dim=0)
        if weight:                                 # the values share one power of two
            floor += 2.0 ** -39 * F.abs().sum(dim=0).reshape(-1, 1) * cols.abs().max() * 1.01
        both = torch.full((want.shape[0], inner + 6), 5.0, dtype=torch.bfloat16, device="cuda")
        part = both[:, 2:-4]
        f = api.act8_weight_grad if weight else api.act8_input_grad
        kw = dict(dtype=torch.bfloat16) if weight else {}
        got = f(d, *k, **kw).double()
        tol = S * (2.0 ** -11 + 2 * 65 * 2.0 ** -22 + 4 * 2.0 ** -24) + floor
        half = half_step("bf16")
        assert ((got - want).abs() <= tol + half * want.abs() + TINY["bf16"]).all()
        assert (got[7] == 0).all()
        part.fill_(2.0)
        f(d, *k, out=part, accumulate=True)
        assert ((part.double() - (want + 2)).abs()
                <= tol + (half + 2.0 ** -23) * (want + 2).abs() + 2.0 ** -23 * 2 + TINY["bf16"]).all()
        assert (both[:, :2] == 5).all() and (both[:, -4:] == 5).all()


# --------------------------------------------- non-finite and huge elements

# weight, tokens, out, inner, group, dtype, result: digits in one-CTA tiles and in pairs, two halves, one half,
# one half per row
WAYS = [(True, 70, 40, 96, 0, "fp32", "fp32"), (True, 1501, 1003, 2601, 0, "bf16", "fp32"),
        (True, 300, 130, 200, 32, "fp32", "fp32"), (True, 300, 130, 200, 64, "fp16", "bf16"),
        (True, 300, 130, 200, 64, "bf16", "bf16"), (True, 600, 2100, 6300, 0, "bf16", "bf16"),
        (False, 40, 70, 96, 0, "fp16", "fp16"), (False, 1003, 1501, 2601, 0, "fp32", "fp32"),
        (False, 2100, 600, 6300, 0, "bf16", "bf16")]


@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("weight,tokens,out,inner,group,dtype,result", WAYS)
def test_non_finite_elements_show_where_they_enter(weight, tokens, out, inner, group, dtype, result, value):
    """An element of dy reaches its output channel's (token's) results, a
    scale those of its group of columns (all, with one scale per row), both
    all of them, zeros in the other factor or not; the others stay finite."""
    api = _api()
    f = api.act8_weight_grad if weight else api.act8_input_grad
    kw = dict(group=group) if weight else {}
    dy = data(tokens, out, dtype, 21, scale=0.01)
    codes, scales = stored(tokens if weight else out, inner, 22, group)[0]
    bad = dy.clone()
    bad[tokens // 2, out // 2] = value                     # a row of zeros otherwise
    got = torch.isfinite(f(bad, codes, scales, dtype=DT[result], **kw))
    row = out // 2 if weight else tokens // 2
    assert not got[row].any() and got[:row].all() and got[row + 1:].all()
    worse = scales.clone()
    g = scales.shape[1] // 2
    worse[scales.shape[0] // 3, g] = value                 # a row of zero codes
    got = torch.isfinite(f(dy, codes, worse, dtype=DT[result], **kw))
    c0, c1 = (g * group, min((g + 1) * group, inner)) if group else (0, inner)
    assert not got[:, c0:c1].any() and got[:, :c0].all() and got[:, c1:].all()


@pytest.mark.parametrize("group", [0, 32])
@pytest.mark.parametrize("dtype,result", [("fp32", "fp32"), ("bf16", "bf16")])
def test_gradient_next_to_the_largest_number(group, dtype, result):
    """One term of 3.38e38.  Digits: a step of 1 / 8355704 and 7 roundings of
    2^-24; halves: 2^-22 of each factor and of the lower parts; one half
    2^-11; then the result's rounding."""
    api = _api()
    dy = torch.zeros(40, 6, dtype=DT[dtype], device="cuda")
    dy[0] = 3.38e38
    codes = np.zeros((40, 96), np.int8)
    codes[0] = 127
    scales = np.full((40, 3 if group else 1), 1 / 127, np.float32)
    got = f64(api.act8_weight_grad(dy, *to_gpu(codes, scales), group=group, dtype=DT[result]))
    want = f64(dy).T @ A.values64(codes, scales, group)
    rel = 2.0 ** -11 if group and result == "bf16" else 3 * 2.0 ** -22 + 8 * 2.0 ** -24
    within(got, want, want * (rel + half_step(result)))
