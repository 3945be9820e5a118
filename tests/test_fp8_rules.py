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
    dense, rows, wgrad = fp8_rules.dense, fp8_rules.rows, fp8_rules.wgrad
    S, T64, T128, T256 = fp8_rules.STREAM16, fp8_rules.TILE64, fp8_rules.TILE128, fp8_rules.TILE256
    for exact in (0, 1):
        assert [dense(M, 4096, 4096, exact) for M in (1, 16, 17, 512, 1024)] == [S, S, T64, T64, T128]
        assert dense(4096, 4096, 4096, exact) == (T128 if exact else T256)
        assert [rows(n, 8, 4096, exact) for n in (33, 512, 8192)] == [T64, T64, T128]
        assert [wgrad(256, 256, n, exact) for n in (8, 64)] == [T64, T128]
        assert wgrad(256, 256, 256, exact) == (T128 if exact else T256)
    assert [rows(n, 8, 4096, 1) for n in (1, 32)] == [S, S] and rows(32, 8, 4096, 0) == T64


@pytest.mark.parametrize("which", ["lda", "ldb"])
def test_wide_rows_leave_the_256_tile(which):
    """255 rows of a pitch from 2^24 on pass 32 bits, where the 128 x 128 tile's do not."""
    dense, rows, wgrad = fp8_rules.dense, fp8_rules.rows, fp8_rules.wgrad
    for ld, tile in ((2 ** 24 - 16, fp8_rules.TILE256), (2 ** 24, fp8_rules.TILE128), (20 << 20, fp8_rules.TILE128),
                     (2 ** 25 - 16, fp8_rules.TILE128)):
        assert dense(256, 49152, 1, 0, **{which: ld}) == tile
        assert rows(256, 1, 49152, 0, **{which: ld}) == tile
        assert wgrad(256, 256, 192, 0, **{which: ld}) == tile
    assert dense(256, 49152, 2 ** 24 - 16, 0, lda=2 ** 24 - 16, ldb=2 ** 24 - 16) == fp8_rules.TILE128   # (K counts too)


def test_launches_of_up_to_32_bits_of_work_items():
    fits = fp8_rules.lib().grid_fits
    for threads in (256, 512, 1024):
        most = (LIMIT - 1) // threads
        assert fits(most, threads, 1) and fits(1, threads, 1)
        for workgroups, times in ((most + 1, 1), (2 ** 31 - 1, 1), (2 ** 32 // threads * 3, 1), (2 ** 62, 1),
                                  (2 ** 50, 2 ** 14), (2 ** 50, 2 ** 31 - 1)):   # (a product that passes 64 bits)
            assert not fits(workgroups, threads, times), (workgroups, times)
