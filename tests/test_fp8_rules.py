"""The host-side rules of the block-scaled fp8 products, without a GPU."""
import pytest

from tests import fp8_rules

LIMIT = 1 << 32


@pytest.mark.parametrize("rows", [128, 256])
def test_rows_whose_offsets_fit_32_bits(rows):
    """The kernels count bytes inside a tile of `rows` rows in 32 bits: rows * ld + K < 2^32, for any ld."""
    fit = fp8_rules.lib().rows_fit_32
    edge = LIMIT // rows
    for K in (0, 1, 16, 128, 4096):
        lds = [0, 16, 4096, edge - 32, edge - 16, edge, edge + 16, 2 * edge, 2 ** 40, 2 ** 55, 2 ** 56, 2 ** 57,
               2 ** 62, 2 ** 63 - 16]
        for ld in lds:
            assert bool(fit(rows, ld, K)) == (rows * ld + K < LIMIT), (rows, ld, K)
