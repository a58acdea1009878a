"""Sizes that the experts' entry points refuse because their kernels count columns
in 32 bits, without a GPU (addresses here are never dereferenced)."""
import pytest

from test_mx_refusals import B, GOOD, rc  # noqa: F401  (B: the fixture)

MOST = (1 << 31) - 1024


@pytest.mark.parametrize("cols", [MOST + 1, (1 << 31) - 8, (1 << 31) - 1, 1 << 31])
def test_columns_that_no_int_counts_are_refused(B, cols):  # noqa: F811
    x, y = GOOD, 1 << 50
    for w, rf, cf in ((None, 1, 0), (None, 2, 3), (GOOD, 3, 0), (GOOD, 0, 2)):
        for k, E in ((2, 8), (1, 1)):
            assert rc(B, B.ez_moe_dispatch, x, cols, 1, cols, GOOD, GOOD, GOOD, k, E, w, rf, GOOD, GOOD, cf, GOOD, GOOD, 0) == B.EZ_ERR_UNSUPPORTED
    for rows in (0, 1, 128):
        assert rc(B, B.ez_moe_combine, x, cols, rows, cols, GOOD, None, 1, 1, y, cols, 0) == B.EZ_ERR_UNSUPPORTED
        assert rc(B, B.ez_moe_weight_gradient, x, cols, y, cols, rows, cols, GOOD, 1, 1, GOOD, 0) == B.EZ_ERR_UNSUPPORTED
    # where there is nothing to be done it does not matter
    assert rc(B, B.ez_moe_dispatch, None, cols, 0, cols, GOOD, GOOD, GOOD, 1, 1, None, 1, GOOD, GOOD, 0, None, None, 0) == B.EZ_OK
    assert rc(B, B.ez_moe_combine, None, cols, 0, cols, GOOD, None, 0, 1, None, cols, 0) == B.EZ_OK
    assert rc(B, B.ez_moe_weight_gradient, None, cols, None, cols, 1, cols, GOOD, 1, 0, None, 0) == B.EZ_OK
