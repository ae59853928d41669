"""Sizes that reach every kernel form of the products: tile, stages and splits
as dc_linear_form and dc_orthogonalize_form give them."""
import numpy as np

from gradient_reduction_amd import dc

BF16, F32 = dc.DC_BF16, dc.DC_F32

# {dtype: {(tile, stages, cut into several sums): (rows, columns, sum) of the
# product}}: multiples of 8 that end inside a tile and a stage
LINEAR = {
    BF16: {(64, 3, False): (72, 136, 72), (64, 3, True): (72, 136, 1032), (128, 2, False): (776, 5000, 72),
           (128, 4, False): (776, 2504, 72), (128, 4, True): (72, 1504, 4104), (256, 2, False): (2000, 4104, 72),
           (256, 2, True): (776, 5000, 4104)},
    F32: {(64, 3, False): (72, 136, 72), (64, 3, True): (72, 136, 520), (128, 2, False): (1504, 5000, 72),
          (128, 2, True): (200, 4104, 4104), (128, 4, False): (1504, 2056, 72), (128, 4, True): (200, 4104, 1032),
          (256, 2, False): (4072, 4008, 72), (256, 2, True): (1504, 4104, 4104)},
}
KINDS = {"forward": dc.DC_PRODUCT_FORWARD, "dx": dc.DC_PRODUCT_DX, "dw": dc.DC_PRODUCT_DW}


def layer_sizes(kind, rows, cols, depth):
    """(T, N, K) of the layer whose product of that kind is rows x cols over
    depth."""
    return {"forward": (rows, cols, depth), "dx": (rows, depth, cols), "dw": (depth, rows, cols)}[kind]


def linear_form(dtype, kind, rows, cols, depth):
    tile, stages, splits = dc.dc_linear_form(dtype, KINDS[kind], *layer_sizes(kind, rows, cols, depth))
    return tile, stages, splits > 1


def odd(sizes):
    """One less of each: an odd number, and no whole 16 bytes a row."""
    return tuple(v - 1 for v in sizes)


def orthogonal_forms(dtype, out_dtype, hold, shapes, update):
    """(tile, stages) of A, B, a step and the last step for the list's first
    matrix."""
    m = np.zeros(len(shapes), dc.MATRIX_DTYPE)
    m["rows"], m["cols"] = [s[0] for s in shapes], [s[1] for s in shapes]
    return [f[:2] for f in dc.dc_orthogonalize_form(dtype, out_dtype, hold, m, len(m), 1 if update else 0, 0)]


# lists whose products take, between them, every form (tests/test_product_forms.py)
ORTHOGONAL = [
    [(63, 65)],                 # 64
    [(777, 130)] * 16,          # X: 128, four stages
    [(520, 1000)] * 16,         # A, B: 128, four stages; X: 128, two
    [(1025, 700)] * 16,         # A, B: 128, two stages; transposed
    [(600, 5000)] * 4,          # X: 256
    [(5000, 603)] * 4,          # X: 256, transposed
    [(2050, 2050)] * 16,        # A, B, X: 256
]
