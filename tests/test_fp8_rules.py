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


def test_kernel_of_each_size():
    r = fp8_rules.lib()
    dense, rows, wgrad = r.choose_dense, r.choose_rows, r.choose_wgrad
    S, T64, T128, T256 = fp8_rules.STREAM16, fp8_rules.TILE64, fp8_rules.TILE128, fp8_rules.TILE256
    for exact in (0, 1):
        assert [dense(M, 4096, 4096, exact) for M in (1, 16, 17, 512, 1024)] == [S, S, T64, T64, T128]
        assert dense(4096, 4096, 4096, exact) == (T128 if exact else T256)
        assert [rows(n, 8, 4096, exact) for n in (33, 512, 8192)] == [T64, T64, T128]
        assert [wgrad(256, 256, n, exact) for n in (8, 64)] == [T64, T128]
        assert wgrad(256, 256, 256, exact) == (T128 if exact else T256)
    assert [rows(n, 8, 4096, 1) for n in (1, 32)] == [S, S] and rows(32, 8, 4096, 0) == T64
