"""GPU: calls of the 8-bit expert layer that other tests do not reach, and what they
refuse on a device.  Formulas in 64 bits and bounds as in tests/moe_ref.py."""
import pytest
import torch

from tests import moe_ref as ref
from tests.parity import say
from tests.test_gpu_moe import DEV, F8, check_product, codes, gen, h, scales  # noqa: F401 (h: fixture)
from tile_planned_generator_amd import dg

pytestmark = pytest.mark.gpu


def test_weight_gradients_that_share_elements_are_refused(h):
    """Before anything is enqueued: C keeps what it held."""
    say("[case] wgrad, overlapping experts")
    g = gen(71)
    M, N, R, E = 64, 80, 256, 2
    a, b, sa, sb = codes(g, M, R), codes(g, N, R), scales(g, 2, M), scales(g, 2, N)
    off = torch.tensor([0, 128, 256], dtype=torch.int32, device=DEV)
    flat = torch.full((2 * M * N,), 7.0, device=DEV)
    for stride in (N, M * N - 1):
        with pytest.raises(dg.DGError) as e:
            h.gemm_fp8_wgrad(a, sa, b, sb, off, flat.as_strided((E, M, N), (stride, N, 1)))
        assert e.value.status == dg.DG_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert (flat == 7).all()
    one, side = torch.empty(E, M, N, device=DEV), torch.empty(M, E, N, device=DEV)
    h.gemm_fp8_wgrad(a, sa, b, sb, off, one)
    h.gemm_fp8_wgrad(a, sa, b, sb, off, side.transpose(0, 1))   # the experts' rows side by side
    assert torch.equal(one, side.transpose(0, 1))


def test_rows_20_mib_apart(h):
    """The size takes the 256 x 256 tile, 255 of whose rows would lie past 4 GiB."""
    M, N, K, ld = 256, 49152, 128, 20 << 20
    say(f"[case] gemm_fp8 {M}x{N}x{K}, rows of A {ld} bytes apart")
    g = gen(72)
    a = torch.empty((M - 1) * ld + K, dtype=torch.uint8, device=DEV).view(F8).as_strided((M, K), (ld, 1))
    near = codes(g, M, K)
    a.copy_(near)
    b, sa, sb = codes(g, N, K), scales(g, 1, M), scales(g, 1, N // 128)
    c, want = (torch.empty(M, N, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    h.gemm_fp8(a, sa, b, sb, c)
    h.gemm_fp8(near, sa, b, sb, want)
    da, db = ref.dequant(near.cpu(), sa.cpu()), ref.dequant(b.cpu(), sb.cpu(), 128)
    exact, mag = ref.product(da, db)
    unit = ref.unit_error(da, db)
    check_product(c, exact, mag, K, unit)
    check_product(want, exact, mag, K, unit)


@pytest.mark.parametrize("N", [64, 50])
@pytest.mark.parametrize("type", [torch.float32, torch.bfloat16])
def test_experts_without_k(h, N, type):
    """K = 0: zeros in the experts' rows, whatever N makes of the empty weights' stride."""
    say(f"[case] grouped K = 0, N {N} {type}")
    E, R = 3, 300
    off = torch.tensor([0, 130, 130, 290], dtype=torch.int32, device=DEV)
    a, b = (torch.empty(*s, 0, dtype=torch.uint8, device=DEV) for s in ((R,), (E, N)))
    c = torch.full((R, N), 7.0, dtype=type, device=DEV)
    h.gemm_fp8_grouped(a, torch.empty(0, R, device=DEV), b, torch.empty(E, 0, 1, device=DEV), off, c)
    assert (c[:290] == 0).all() and (c[290:] == 7).all()
