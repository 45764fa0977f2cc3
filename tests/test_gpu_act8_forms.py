"""The products' forms, each against the definition in 64 bits, and calls that
follow each other at once."""
import pytest
import torch

from act8_shapes import INPUT, MATMUL, WEIGHT
from bit_quantized_shampoo_b200 import _lib as L
from test_gpu_act8 import DT, TINY, data, half_step, stored

pytestmark = pytest.mark.gpu


def _api():
    from bit_quantized_shampoo_b200 import api
    return api


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def some_codes(rows, cols, group, seed, scale=1.0):
    """Codes and scales of rows of different magnitude, a row of zeros."""
    g = _generator(seed)
    codes = torch.randint(-127, 128, (rows, (cols + 15) // 16 * 16), generator=g, device="cuda", dtype=torch.int8)
    groups = -(-cols // group) if group else 1
    scales = torch.exp(0.5 * torch.randn(rows, groups, generator=g, device="cuda")) * (scale / 127)
    if rows > 4:
        codes[rows // 3] = 0
        scales[rows // 3] = 0
    return codes[:, :cols], scales


def some_gradients(rows, cols, dtype, seed):
    g = _generator(seed)
    x = torch.randn(rows, cols, generator=g, device="cuda") * torch.exp(0.5 * torch.randn(rows, 1, generator=g, device="cuda"))
    if rows > 4:
        x[rows // 2] = 0
    return (x * 0.01).to(DT[dtype])


def values64(codes, scales, group):
    cols = codes.shape[1]
    index = torch.arange(cols, device="cuda") // group if group else torch.zeros(cols, dtype=torch.long, device="cuda")
    return codes.double() * scales.double()[:, index]


def within(got, want, tol):
    bad = ~((got.double() - want).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist(), got[bad][:4], want[bad][:4])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("tokens,out,inner,rows,split", MATMUL)
def test_product(tokens, out, inner, rows, split, dtype):
    """The sum is exact; conversion, two scalings and the bias round in fp32
    (2^-24 each), the result once."""
    api = _api()
    x, w = some_codes(tokens, inner, 0, 1), some_codes(out, inner, 0, 2, 0.05)
    bias = torch.randn(out, generator=_generator(3), device="cuda") if out % 2 else None
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    y = api.act8_matmul(*x, *w, bias=bias, dtype=DT[dtype], flags=flags)
    p = (x[0].double() @ w[0].double().t()) * x[1].double() * w[1].double().t()
    want = p if bias is None else p + bias.double()
    within(y, want, 1.01 * (3 * 2.0 ** -24 * p.abs() + (2.0 ** -24 + half_step(dtype)) * want.abs()) + TINY[dtype])
    assert int(flags.item()) == 0


def gradient_tolerance(way, parts, dy, k, group, dtype, weight, K):
    """Beside the result's rounding; S the sum of the products' magnitudes.
    Digits: F = dy scale rounds to fp32, and to a step of its row's largest /
    8355704 (with a rounding of the factor and of the product); sums exact, 6
    roundings to join and scale them.  Halves: dy and value off by 2^-22 each
    (one half: 2^-11), their lower parts' product at most 2^-22, at most 17
    additions of 2^-22 for each of up to three kinds of products (one product:
    65), a rounding per 256 k (1024) and up to 36 to join shares; an element
    is no coarser than 2^-39 of the largest over the contraction."""
    codes, scales = k
    a, b = dy.double().abs(), values64(codes, scales, group).abs()
    S = (a.t() if weight else a) @ b
    if way == L.ACT8_WAY_DIGITS:
        F = a * (scales.double() if weight else scales.double().t())
        top = F.amax(dim=0 if weight else 1).reshape(-1, 1)
        count = codes.double().abs().sum(dim=0, keepdim=True)
        return top * count * (0.5 / 8355704 + 2 * 2.0 ** -24) + S * 7 * 2.0 ** -24
    if way == L.ACT8_WAY_ROW_HALVES:
        F = a * scales.double().t()
        floor = 2.0 ** -39 * F.amax(dim=1, keepdim=True) * codes.double().abs().sum(dim=0, keepdim=True)
    else:
        floor = 2.0 ** -39 * (a.amax(dim=0).reshape(-1, 1) * b.sum(dim=0) + a.sum(dim=0).reshape(-1, 1) * b.max() * 1.01)
    rel = 2.0 ** -11 + 65 * 2.0 ** -22 if parts == 1 else (4 + 17 * (3 if dtype == "fp32" else 2)) * 2.0 ** -22
    return S * (rel + (K // 256 + 36) * 2.0 ** -24) + floor


def check_gradient(weight, case):
    api = _api()
    tokens, out, inner, dtype, result, group, way, rows, split, parts = case
    dy = some_gradients(tokens, out, dtype, 4)
    k = some_codes(tokens if weight else out, inner, group, 5, 1.0 if weight else 0.05)
    v = values64(*k, group)
    want = (dy.double().t() if weight else dy.double()) @ v
    tol = gradient_tolerance(way, parts, dy, k, group, dtype, weight, v.shape[0])
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    f = api.act8_weight_grad if weight else api.act8_input_grad
    kw = dict(group=group, flags=flags) if weight else dict(flags=flags)
    got = f(dy, *k, dtype=DT[result], **kw)
    half = half_step(result)
    within(got, want, tol + half * want.abs() + TINY[result])
    start = torch.randn(want.shape, generator=_generator(6), device="cuda").to(DT[result])
    room = torch.full((want.shape[0], inner + 5), 3.0, dtype=DT[result], device="cuda")
    part = room[:, 2:-3]
    part.copy_(start)
    f(dy, *k, out=part, accumulate=True, **kw)
    total = want + start.double()
    within(part, total, tol + (half + 2.0 ** -23) * total.abs() + 2.0 ** -23 * start.double().abs() + TINY[result])
    assert (room[:, :2] == 3).all() and (room[:, -3:] == 3).all() and int(flags.item()) == 0


@pytest.mark.parametrize("case", WEIGHT)
def test_weight_gradient(case):
    check_gradient(True, case)


@pytest.mark.parametrize("case", INPUT)
def test_input_gradient(case):
    check_gradient(False, case)


@pytest.mark.parametrize("tokens,out,inner", [(1, 700, 900), (40, 500, 300), (2100, 2600, 400)])
def test_layers_back_to_back_take_their_own_scales(tokens, out, inner):
    """Calls whose scratch and scales lie where the call before them had its
    own, at other magnitudes; each product starts under the pass that writes
    them."""
    api = _api()
    w = stored(out, inner, 1)[0]
    xs = [data(tokens, inner, "bf16", 2 + k, scale=10.0 ** (3 * k - 6)) for k in range(5)]
    dys = [data(tokens, out, "bf16", 9 + k, scale=10.0 ** (6 - 3 * k)) for k in range(5)]
    ys, dxs = [], []
    for x, dy in zip(xs, dys):
        ys.append(api.act8_linear(x, *w))
        dxs.append(api.act8_input_grad(dy, *w))
        torch.cuda.synchronize()
    for _ in range(4):
        for k in (3, 0, 4, 1, 2):
            y, dx = api.act8_linear(xs[k], *w), api.act8_input_grad(dys[k], *w)
            assert torch.equal(y, ys[k]) and torch.equal(dx, dxs[k])
            y, dx = None, None


def test_gradients_on_two_streams_and_replayed():
    """Every way of the gradients, on two streams at once (each call has its
    own scratch) and captured with three passes in a row: the results are those
    of the calls one by one, bit for bit."""
    api = _api()
    calls = []
    for weight, cases in ((True, WEIGHT), (False, INPUT)):
        for n, (tokens, out, inner, dtype, result, group, *_) in enumerate(cases):
            dy = some_gradients(tokens, out, dtype, 10 + n)
            k = some_codes(tokens if weight else out, inner, group, 30 + n)
            f = api.act8_weight_grad if weight else api.act8_input_grad
            kw = dict(group=group, dtype=DT[result]) if weight else dict(dtype=DT[result])
            calls.append(lambda f=f, dy=dy, k=k, kw=kw: f(dy, *k, **kw))
    want = []
    for c in calls:
        want.append(c())
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(2):
        got = [[], []]
        for c in calls:
            for s, g in zip(streams, got):
                with torch.cuda.stream(s):
                    g.append(c())
        torch.cuda.synchronize()
        for g in got:
            assert all(torch.equal(a, b) for a, b in zip(g, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = [c() for c in calls]
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    del graph
