"""Shampoo4.weight_grads: a handle's gradients from 8-bit checkpoints.  What
cannot be done is refused before anything is written, results on a given
stream stay allocated, and an expired wait shows in the handle's flags."""
import pytest
import torch

from bit_quantized_shampoo_b200 import _lib as L
from test_gpu_act8 import data, stored

pytestmark = pytest.mark.gpu


def _api():
    from bit_quantized_shampoo_b200 import api
    return api


SHAPES = [(130, 70), (64, 200), (33, 48)]


def _layers(group=0, tokens=50):
    dys = [data(tokens, r, "bf16", 200 + r, scale=0.01) for r, _ in SHAPES]
    xs = [stored(tokens, c, 201 + c, group)[0] for _, c in SHAPES]
    return dys, xs


BAD = {
    "tokens": lambda dys, xs, gs: dys.__setitem__(2, dys[2][:-1]),
    "type of dy": lambda dys, xs, gs: dys.__setitem__(2, dys[2].double()),
    "columns of dy": lambda dys, xs, gs: dys.__setitem__(2, dys[2][:, :-1]),
    "dy on the host": lambda dys, xs, gs: dys.__setitem__(2, dys[2].cpu()),
    "rows of dy that overlap": lambda dys, xs, gs: dys.__setitem__(2, dys[2][:1].expand(50, 33)),
    "alignment of codes": lambda dys, xs, gs: xs.__setitem__(
        2, (torch.zeros(50, 56, dtype=torch.int8, device="cuda")[:, 8:], xs[2][1])),
    "scales": lambda dys, xs, gs: xs.__setitem__(2, (xs[2][0], xs[2][1][:-1])),
    "type of codes": lambda dys, xs, gs: xs.__setitem__(2, (xs[2][0].float(), xs[2][1])),
    "a single tensor": lambda dys, xs, gs: xs.__setitem__(2, xs[2][0]),
    "shape of grads": lambda dys, xs, gs: gs.__setitem__(2, gs[2].t()),
    "type of grads": lambda dys, xs, gs: gs.__setitem__(2, gs[2].half()),
    "rows of grads that overlap": lambda dys, xs, gs: gs.__setitem__(2, gs[2][:1].expand(33, 48)),
    "one gradient inside another": lambda dys, xs, gs: gs.__setitem__(2, gs[1].view(-1)[:33 * 48].view(33, 48)),
    "a gradient over its input": lambda dys, xs, gs: gs.__setitem__(2, xs[0][1].expand(-1, 48)[:33]),
}


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("what", list(BAD))
def test_a_bad_last_layer_leaves_the_others_as_they_were(what, accumulate):
    api = _api()
    sh = api.Shampoo4(SHAPES)
    dys, xs = _layers()
    grads = [torch.full(s, 3.0, device="cuda") for s in SHAPES]
    keep = list(grads)
    BAD[what](dys, xs, grads)
    with pytest.raises((TypeError, ValueError, RuntimeError)):
        sh.weight_grads(dys, xs, grads=grads, accumulate=accumulate)
    torch.cuda.synchronize()
    assert all(torch.all(g == 3) for g in keep)


@pytest.mark.parametrize("group", [0, 32])
@pytest.mark.parametrize("tokens", [0, 1, 50, 700])
def test_gradients_are_those_of_the_calls(tokens, group):
    api = _api()
    sh = api.Shampoo4(SHAPES)
    dys, xs = _layers(group, tokens)
    grads = sh.weight_grads(dys, xs, group=group)
    want = [api.act8_weight_grad(d, *x, group=group) for d, x in zip(dys, xs)]
    assert all(torch.equal(g, w) for g, w in zip(grads, want))
    room = [torch.full((r, c + 5), 2.0, device="cuda") for r, c in SHAPES]
    given = [g[:, 3:-2] for g in room]
    assert sh.weight_grads(dys, xs, group=group, grads=given) is given
    assert all(torch.equal(g, w) for g, w in zip(given, want))
    assert all(torch.all(g[:, :3] == 2) and torch.all(g[:, -2:] == 2) for g in room)
    sh.weight_grads(dys, xs, group=group, grads=given, accumulate=True)
    assert all(torch.equal(g, 2 * w) for g, w in zip(given, want))
    assert sh.status_flags() == 0


def test_gradients_dropped_early_stay_with_the_given_stream():
    """Gradients made for another stream and dropped at once: what is
    allocated next must not share their memory while that stream still writes."""
    api = _api()
    shapes = [(1024, 4096), (1024, 4096)]
    sh = api.Shampoo4(shapes)
    side = torch.cuda.Stream()
    dys = [data(4096, 1024, "bf16", 5, scale=0.01) for _ in shapes]
    xs = [stored(4096, 4096, 6)[0]] * 2
    sh.weight_grads(dys, xs, stream=side)
    torch.cuda.synchronize()
    bad = 0
    for _ in range(5):
        for _ in range(4):
            sh.weight_grads(dys, xs, stream=side)
        mark = [torch.full(s, 3.0, device="cuda") for s in shapes]
        side.synchronize()
        bad += sum(int((m != 3.0).any()) for m in mark)
        del mark
    assert bad == 0


def test_gradients_captured_and_replayed():
    api = _api()
    sh = api.Shampoo4(SHAPES)
    dys, xs = _layers()
    want = [g.clone() for g in sh.weight_grads(dys, xs)]
    ins = [torch.zeros_like(d) for d in dys]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        grads = sh.weight_grads(ins, xs)
    for a, b in zip(ins, dys):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(grads, want))
    del graph


def test_an_expired_wait_is_in_the_handles_flags():
    """With a limit of 1 ns the epilogue gives up on a sum over 20000 tokens
    (some 40 us; a wait below a few us ends inside the first try and cannot
    run out), the products on their accumulators; the loads are waited for with
    the ordinary limit, and the call returns.  With the default limit the next
    call is right."""
    api = _api()
    shape, tokens = (1024, 2048), 20000
    sh = api.Shampoo4([shape])
    dys = [data(tokens, shape[0], "bf16", 7, scale=0.01)]
    xs = [stored(tokens, shape[1], 8)[0]]
    want = [g.clone() for g in sh.weight_grads(dys, xs)]
    assert sh.status_flags() == 0
    L.call("shampoo4_debug_wait_limit", sh._h, 1)
    sh.weight_grads(dys, xs)
    assert sh.status_flags() & L.FLAG_TIMEOUT
    L.call("shampoo4_debug_wait_limit", sh._h, 0)
    got = sh.weight_grads(dys, xs)
    assert sh.status_flags() == 0 and torch.equal(got[0], want[0])


def test_time_spent_by_the_operand_pass_does_not_count():
    """The product starts under the pass that writes its operand and waits for
    it.  The pass over 2^23 tokens of 64 columns has 8 CTAs and takes about 14
    ms; the longest wait of the product itself, for 1024 k-blocks, is below
    half a millisecond and must not run out at 4 ms."""
    api = _api()
    sh = api.Shampoo4([(64, 64)])
    tokens = 1 << 23
    dys = [torch.ones(tokens, 64, dtype=torch.bfloat16, device="cuda")]
    xs = [(torch.ones(tokens, 64, dtype=torch.int8, device="cuda"), torch.ones(tokens, 1, device="cuda"))]
    L.call("shampoo4_debug_wait_limit", sh._h, 4000000)
    g, = sh.weight_grads(dys, xs)
    assert sh.status_flags() == 0
    # exact sums of 2^17 tokens, 64 of them added in fp32, six roundings of digits and scales
    assert ((g.double() - tokens).abs() <= tokens * 70 * 2.0 ** -24).all()
