"""shampoo4_weight_grads without a GPU: its workspace and what it refuses
(everything is checked before a device is touched, readiness last)."""
import ctypes as C

import pytest

from bit_quantized_shampoo_b200 import _lib as L

INVALID, NOT_READY, WORKSPACE = 1, 3, 5
SHAPES = [(64, 96), (32, 48)]
MB = 1 << 20


@pytest.fixture(scope="module")
def handle():
    cfg = L.Config(0.95, 1e-6, 1024, 64, 5, L.PREC_TF32, 0, 0, 1, 0, 0, 0, 0)
    params = (L.Param * 2)(*[L.Param(r, c) for r, c in SHAPES])
    h = C.c_void_p()
    L.call("shampoo4_init", C.byref(cfg), params, 2, C.byref(h))
    yield h
    L.lib().shampoo4_destroy(h)


def layers(**last):
    """Fake, well-aligned device addresses a MiB apart; ``last`` changes the
    second layer."""
    out = []
    for i, (r, c) in enumerate(SHAPES):
        kw = dict(dy=(1 + 4 * i) * MB, dtype=L.ACT8_BF16, lddy=r, codes=(2 + 4 * i) * MB, ldc=c, scales=(3 + 4 * i) * MB,
                  tokens=10)
        kw.update(last if i else {})
        out.append(L.Layer(*[kw[n] for n, _ in L.Layer._fields_]))
    return (L.Layer * 2)(*out)


def call(h, ls=None, group=0, grads=(16 * MB, 17 * MB), ld=(96, 48), acc=0, ws=32 * MB, n=1 << 30):
    return L.lib().shampoo4_weight_grads(h, layers() if ls is None else ls, group, L.ptr_array(list(grads)),
                                         L.i64_array(list(ld)), acc, C.c_void_p(ws), n, C.c_void_p(0))


def test_good_arguments_get_as_far_as_the_missing_buffers(handle):
    assert call(handle) == NOT_READY and call(handle, group=32, acc=1) == NOT_READY


@pytest.mark.parametrize("bad", [dict(dy=0), dict(dtype=3), dict(lddy=31), dict(codes=0), dict(codes=6 * MB + 8),
                                 dict(ldc=40), dict(ldc=56), dict(scales=0), dict(scales=7 * MB + 2), dict(tokens=-1),
                                 dict(dy=5 * MB + 1), dict(tokens=(1 << 30) + 1)])
def test_a_bad_layer_is_refused(handle, bad):
    assert call(handle, layers(**bad)) == INVALID


@pytest.mark.parametrize("kw", [
    dict(group=48), dict(grads=(16 * MB, 0)), dict(grads=(16 * MB, 17 * MB + 2)), dict(ld=(96, 47)), dict(ws=0),
    dict(ws=32 * MB + 128), dict(grads=(16 * MB, 16 * MB)), dict(grads=(16 * MB, 16 * MB + 4 * 95)),
    dict(grads=(16 * MB, 1 * MB)), dict(grads=(16 * MB, 2 * MB)), dict(grads=(16 * MB, 3 * MB)),
    dict(grads=(5 * MB, 17 * MB))])
def test_bad_gradients_and_workspaces_are_refused(handle, kw):
    assert call(handle, **kw) == INVALID


def test_workspace(handle):
    n, one = C.c_size_t(), C.c_size_t()
    sizes = []
    for group in (0, 32):
        L.call("shampoo4_weight_grads_workspace", handle, layers(), group, C.byref(n))
        for r, c in SHAPES:
            L.call("act8_grad_workspace", 1, L.ACT8_BF16, L.ACT8_FP32, 10, r, c, group, C.byref(one))
            sizes.append(one.value)
        assert n.value == max(sizes[-2:])
        assert call(handle, group=group, n=n.value) == NOT_READY
        assert call(handle, group=group, n=n.value - 1) == WORKSPACE
    L.call("shampoo4_weight_grads_workspace", handle, layers(tokens=0), 0, C.byref(n))
    assert n.value == sizes[0]
    f = L.lib().shampoo4_weight_grads_workspace
    assert f(handle, None, 0, C.byref(n)) == INVALID and f(handle, layers(), 0, None) == INVALID
    assert f(handle, layers(dtype=9), 0, C.byref(n)) == INVALID and f(handle, layers(), 5, C.byref(n)) == INVALID


def test_no_layers(handle):
    assert L.lib().shampoo4_weight_grads(None, layers(), 0, None, None, 0, None, 0, None) == INVALID
    assert L.lib().shampoo4_weight_grads(handle, layers(), 0, None, None, 0, None, 0, None) == INVALID
    assert L.lib().shampoo4_weight_grads(handle, None, 0, L.ptr_array([16 * MB, 17 * MB]), L.i64_array([96, 48]), 0,
                                         C.c_void_p(32 * MB), 1 << 30, None) == INVALID
