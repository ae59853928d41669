"""The sizes that the GPU tests take reach every kernel form of the products
(host only: the library's own choice), and the form queries' refusals."""
import numpy as np
import pytest

from gradient_reduction_amd import dc
from tests import product_forms as pf
from tests.test_abi import expect
from tests.test_products_abi import mats

TILES = {(64, 3), (128, 2), (128, 4), (256, 2)}


@pytest.mark.parametrize("dtype", [pf.BF16, pf.F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("kind", list(pf.KINDS))
def test_layer_sizes_reach_every_form(kind, dtype):
    assert {f[:2] for f in pf.LINEAR[dtype]} == TILES
    assert {f[0] for f in pf.LINEAR[dtype] if f[2]} == {64, 128, 256}
    for form, sizes in pf.LINEAR[dtype].items():
        assert pf.linear_form(dtype, kind, *sizes) == form
        assert pf.linear_form(dtype, kind, *pf.odd(sizes)) == form


@pytest.mark.parametrize("hold", [dc.DC_HOLD_ONE, dc.DC_HOLD_PAIR])
@pytest.mark.parametrize("update", [False, True])
def test_lists_reach_every_form(update, hold):
    seen = [set(), set(), set(), set()]
    for shapes in pf.ORTHOGONAL:
        for s, f in zip(seen, pf.orthogonal_forms(pf.BF16, pf.F32, hold, shapes, update)):
            s.add(f)
    assert seen[:3] == [TILES] * 3
    # the last step of an update takes 128 tiles in the place of 256
    assert seen[3] == (TILES - {(256, 2)} if update else TILES)


def test_few_rows_have_a_kernel_of_their_own():
    for T in (0, 1, 64):
        assert dc.dc_linear_form(0, dc.DC_PRODUCT_FORWARD, T, 4096, 4096) == (0, 0, 0)
        assert dc.dc_linear_form(0, dc.DC_PRODUCT_DX, T, 4096, 4096)[0] in (64, 128, 256)


def test_refusals():
    out = np.zeros(3, np.int32)
    call = dc.lib().dc_linear_form
    for code, args in [(dc.DC_ERR_DTYPE, (2, 0, 4, 4, 4)), (dc.DC_ERR_ARG, (0, -1, 4, 4, 4)),
                       (dc.DC_ERR_ARG, (0, 3, 4, 4, 4)), (dc.DC_ERR_ARG, (0, 0, -1, 4, 4)),
                       (dc.DC_ERR_ARG, (0, 0, 4, 0, 4)), (dc.DC_ERR_SHAPE, (0, 0, 4, 4, 1 << 29))]:
        expect(code, dc.dc_linear_form, *args)
    assert call(0, 0, 4, 4, 4, None) == dc.DC_ERR_NULL and not out.any()
    m = mats((30, 40), (50, 60))
    for code, args in [(dc.DC_ERR_DTYPE, (2, 0, 0, m, 2, 0, 0)), (dc.DC_ERR_DTYPE, (0, 2, 0, m, 2, 0, 0)),
                       (dc.DC_ERR_ARG, (0, 0, 3, m, 2, 0, 0)), (dc.DC_ERR_ARG, (0, 0, 0, m, 2, 2, 0)),
                       (dc.DC_ERR_ARG, (0, 0, 0, m, 2, 0, 2)), (dc.DC_ERR_ARG, (0, 0, 0, m, 2, 0, -1)),
                       (dc.DC_ERR_ARG, (0, 0, 0, m, 0, 0, 0)), (dc.DC_ERR_NULL, (0, 0, 0, None, 2, 0, 0)),
                       (dc.DC_ERR_ARG, (0, 0, 0, mats((0, 3)), 1, 0, 0))]:
        expect(code, dc.dc_orthogonalize_form, *args)
    assert dc.lib().dc_orthogonalize_form(0, 0, 0, m.ctypes.data, 2, 0, 0, None) == dc.DC_ERR_NULL
    # every matrix of a list of several chunks has its form
    many = mats(*[(300, 20 + k) for k in range(300)])
    for k in (0, 127, 128, 299):
        assert {f[0] for f in dc.dc_orthogonalize_form(0, 1, 0, many, 300, 1, k)} <= {64, 128}
