"""Sizes that reach every form of the 8-bit products: (tokens, out, inner), and
the form that they have to take.  Rows 0 are tiles of a pair of CTAs; those
sizes have more tiles than a B200 has pairs (74), or more k-blocks than the
longest ring of stages (8), odd sizes and partial tiles."""
from bit_quantized_shampoo_b200 import _lib as L

DTYPE = {"fp32": L.ACT8_FP32, "bf16": L.ACT8_BF16, "fp16": L.ACT8_FP16}

# tokens, out, inner, rows of a tile, contraction split
MATMUL = [
    (1, 700, 64, 16, False), (36, 3533, 787, 16, False), (58, 105, 16426, 16, True),
    (105, 10829, 88, 64, False), (301, 2304, 3999, 64, True),
    (777, 2304, 767, 128, False), (250, 9001, 500, 128, False), (4172, 9, 3247, 128, True),
    (2101, 2603, 1499, 0, False), (4126, 2445, 10, 0, False), (600, 9001, 4098, 0, False),
]
# tokens, out, inner, dtype, result, group, way, rows of a tile, contraction split, halves of a value
WEIGHT = [
    (639, 9, 17416, "fp32", "fp32", 0, L.ACT8_WAY_DIGITS, 16, False, 0),
    (5757, 9, 1931, "bf16", "fp32", 0, L.ACT8_WAY_DIGITS, 16, True, 0),
    (90, 105, 16426, "fp16", "fp16", 0, L.ACT8_WAY_DIGITS, 32, False, 0),
    (3173, 986, 33, "fp32", "bf16", 0, L.ACT8_WAY_DIGITS, 32, True, 0),
    (1501, 1003, 2601, "fp32", "fp32", 0, L.ACT8_WAY_DIGITS, 0, False, 0),
    (1003, 4101, 2999, "bf16", "fp32", 0, L.ACT8_WAY_DIGITS, 0, False, 0),
    (1301, 2101, 6299, "bf16", "bf16", 0, L.ACT8_WAY_HALVES, 0, False, 1),
    (2303, 2309, 2601, "bf16", "bf16", 64, L.ACT8_WAY_HALVES, 0, False, 1),
    (1501, 2101, 2601, "fp32", "fp32", 128, L.ACT8_WAY_HALVES, 0, False, 2),
    (1501, 2101, 2601, "bf16", "fp32", 32, L.ACT8_WAY_HALVES, 0, False, 2),
    (9001, 130, 513, "fp16", "fp32", 256, L.ACT8_WAY_HALVES, 0, True, 2),
]
INPUT = [
    (9, 639, 17416, "fp32", "fp32", 0, L.ACT8_WAY_DIGITS, 16, False, 0),
    (9, 5757, 1931, "bf16", "bf16", 0, L.ACT8_WAY_DIGITS, 16, True, 0),
    (105, 90, 16426, "fp16", "fp16", 0, L.ACT8_WAY_DIGITS, 32, False, 0),
    (986, 3173, 33, "fp32", "bf16", 0, L.ACT8_WAY_DIGITS, 32, True, 0),
    (1003, 1501, 2601, "fp32", "fp32", 0, L.ACT8_WAY_DIGITS, 0, False, 0),
    (4101, 1003, 2999, "fp16", "fp16", 0, L.ACT8_WAY_DIGITS, 0, False, 0),
    (2101, 1301, 6299, "bf16", "bf16", 0, L.ACT8_WAY_ROW_HALVES, 0, False, 1),
]
