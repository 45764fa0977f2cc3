"""Which form each size takes: the sizes that the GPU tests compare with the
definition reach every form, and a rule that moved a border would show here."""
import ctypes as C

import pytest

from act8_shapes import DTYPE, INPUT, MATMUL, WEIGHT
from bit_quantized_shampoo_b200 import _lib as L

INVALID = 1


def form(call, tokens, out, inner, dtype="bf16", result="bf16", group=0):
    f = L.Form()
    L.call("act8_product_form", call, DTYPE[dtype], DTYPE[result], tokens, out, inner, group, C.byref(f))
    return f


@pytest.mark.parametrize("tokens,out,inner,rows,split", MATMUL)
def test_products(tokens, out, inner, rows, split):
    f = form(0, tokens, out, inner)
    assert (f.way, f.tile_rows, f.shares > 1) == (L.ACT8_WAY_CODES, rows, split)


@pytest.mark.parametrize("call,case", [(1, c) for c in WEIGHT] + [(2, c) for c in INPUT])
def test_gradients(call, case):
    tokens, out, inner, dtype, result, group, way, rows, split, parts = case
    f = form(call, tokens, out, inner, dtype, result, group)
    assert (f.way, f.tile_rows, f.shares > 1, f.code_parts) == (way, rows, split, parts)


@pytest.mark.parametrize("call", [0, 1, 2])
@pytest.mark.parametrize("sizes", [(0, 0, 0), (0, 8, 8), (8, 0, 8), (8, 8, 0), (8, 0, 0), (0, 0, 8)])
def test_empty(call, sizes):
    for group in ([0, 32] if call == 1 else [0]):
        assert form(call, *sizes, group=group).shares == 0


def test_every_form_is_among_them():
    assert {(r, s) for *_, r, s in MATMUL} == {(16, False), (16, True), (64, False), (64, True), (128, False),
                                               (128, True), (0, False)}
    digits = {(r, s) for c in (WEIGHT, INPUT) for *_, way, r, s, _ in c if way == L.ACT8_WAY_DIGITS}
    assert digits == {(16, False), (16, True), (32, False), (32, True), (0, False)}
    assert {(d, s, p) for _, _, _, d, _, _, way, _, s, p in WEIGHT if way == L.ACT8_WAY_HALVES} \
        >= {("bf16", False, 1), ("fp32", False, 2), ("bf16", False, 2), ("fp16", True, 2)}


@pytest.mark.parametrize("args", [(3, 0, 0, 1, 1, 1, 0), (-1, 0, 0, 1, 1, 1, 0), (1, 3, 0, 1, 1, 1, 0),
                                  (1, 0, 3, 1, 1, 1, 0), (1, 0, 0, -1, 1, 1, 0), (1, 0, 0, 1, 1, -1, 0),
                                  (1, 0, 0, 1, 1, 1, 5), (2, 0, 0, 1, 1, 1, 32)])
def test_refusals(args):
    assert L.lib().act8_product_form(*args, C.byref(L.Form())) == INVALID
    assert L.lib().act8_product_form(1, 0, 0, 1, 1, 1, 0, None) == INVALID
