"""The largest sizes the 8-bit expert layer takes, without a GPU."""
import os

import pytest

from tile_planned_generator_amd import dg

pytestmark = pytest.mark.skipif(not os.path.exists(dg.LIB_PATH),
                                reason="libdg.so not built (run __graft_entry__.build())")
MOST = 2 ** 31 - 4096


@pytest.fixture(scope="module")
def off():
    h = dg.Handle(offline=dg.default_device_desc())
    yield h
    h.close()


@pytest.mark.parametrize("at", [0, 1, 2])
def test_sizes_that_a_tile_would_carry_past_31_bits_are_refused(off, at):
    """The kernels round sizes up to whole tiles, blocks or runs, of 2048 at most, in 32 bits."""
    sizes = [1, 1, 1]
    for v, ok in ((MOST, True), (MOST + 1, False), (2 ** 31 - 1, False), (2 ** 31, False)):
        sizes[at] = v
        if ok:
            off.plan_fp8(*sizes)
            off.moe_sort_workspace(sizes[at], 1, 8)
        else:
            for call in (lambda: off.plan_fp8(*sizes), lambda: off.moe_sort_workspace(sizes[at], 1, 8)):
                with pytest.raises(dg.DGError) as e:
                    call()
                assert e.value.status == dg.DG_ERR_UNSUPPORTED
