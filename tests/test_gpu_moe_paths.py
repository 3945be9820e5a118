"""GPU: calls of the 8-bit expert layer that other tests do not reach, and what they
refuse on a device.  Formulas in 64 bits and bounds as in tests/moe_ref.py."""
import pytest
import torch

from tests import fp8_rules
from tests import moe_ref as ref
from tests.parity import say
from tests.test_gpu_moe import DEV, F8, TYPES, check_product, codes, gen, h, offsets_of, scales  # noqa: F401 (h: fixture)
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


# ------------------------------------------------------- every kernel of every mode
def experts_operands(g, R, E, N, K):
    """Codes and scales of rows and experts, one row of padding after each expert's weights."""
    kb, nb = -(-K // 128), -(-N // 128)
    b = codes(g, E * (N + 1), K)
    b = b.as_strided((E, N, K), ((N + 1) * b.stride(0), b.stride(0), 1))
    return codes(g, R, K), scales(g, kb, R), b, scales(g, E * kb, nb).view(E, kb, nb)


def check_experts(h, off, R, N, K, types, kernel):
    E, g = len(off) - 1, gen(N + K)
    a, sa, b, sb = experts_operands(g, R, E, N, K)
    for t in types:
        assert fp8_rules.rows(R, E, N, t == torch.float32) == kernel
        c = torch.full((R, N + 3), 7.0, dtype=t, device=DEV)
        s = sa * (1e-5 if t == torch.float16 else 1.0)
        h.gemm_fp8_grouped(a, s, b, sb, off.to(DEV), c[:, :N])
        for e in range(E):
            lo, hi = int(off[e]), int(off[e + 1])
            if lo < hi:
                da, db = ref.dequant(a[lo:hi].cpu(), s[:, lo:hi].cpu()), ref.dequant(b[e].cpu(), sb[e].cpu(), 128)
                want, mag = ref.product(da, db)
                check_product(c[lo:hi, :N], want, mag, K, ref.unit_error(da, db))
        assert (c[int(off[-1]):] == 7).all() and (c[:, N:] == 7).all()


@pytest.mark.parametrize("counts,spare,N,K", [
    ([1] * 16, 40, 100, 300), ([2, 0, 3, 1], 2, 77, 1000), ([20, 0, 1, 3, 0, 0], 0, 130, 129), ([1], 0, 4096, 128),
    ([0, 0, 40, 33, 0, 2] + [0] * 20, 5, 16, 5000)])
def test_experts_with_a_few_exact_rows(h, counts, spare, N, K):
    """The streaming kernel over experts, one with more rows than a tile among them."""
    say(f"[case] streamed experts {counts} {N} {K}")
    off = offsets_of(counts, 1)
    check_experts(h, off, int(off[-1]) + spare, N, K, [torch.float32], fp8_rules.STREAM16)


@pytest.mark.parametrize("type", ["f32", "bf16", "f16"])
def test_experts_on_the_128_tile(h, type):
    """Nine blocks along K, the last one short: stages are refilled and the dies start at different blocks."""
    say(f"[case] experts, 128 x 128 tile, {type}")
    off = offsets_of([1500, 700, 0, 3, 130], 1)
    check_experts(h, off, int(off[-1]) + 9, 2100, 1100, [TYPES[type]], fp8_rules.TILE128)


@pytest.mark.parametrize("type", ["bf16", "f16"])
def test_experts_on_the_256_tile(h, type):
    say(f"[case] experts, 256 x 256 tile, {type}")
    off = offsets_of([0, 3584, 128, 1], 1)
    check_experts(h, off, int(off[-1]) + 9, 4090, 650, [TYPES[type]], fp8_rules.TILE256)


@pytest.mark.parametrize("b_block", [128, 1])
@pytest.mark.parametrize("M,N,K,type,kernel", [
    (2100, 2050, 1100, "f32", fp8_rules.TILE128), (2100, 2050, 1100, "bf16", fp8_rules.TILE128),
    (2050, 2100, 640, "f16", fp8_rules.TILE128), (3601, 3500, 650, "f16", fp8_rules.TILE256),
    (3590, 3605, 1025, "bf16", fp8_rules.TILE256)])
def test_dense_on_the_large_tiles(h, M, N, K, type, kernel, b_block):
    say(f"[case] gemm_fp8 {M}x{N}x{K} {type} b_block {b_block}")
    t = TYPES[type]
    assert fp8_rules.dense(M, N, K, type == "f32") == kernel
    g, kb = gen(M + K), -(-K // 128)
    a, b = codes(g, M, K, (K + 15) // 16 * 16 + 16), codes(g, N, K)
    sa, sb = scales(g, kb, M + 2)[:, :M] * (1e-5 if type == "f16" else 1.0), scales(g, kb, -(-N // b_block))
    da, db = ref.dequant(a.cpu(), sa.cpu()), ref.dequant(b.cpu(), sb.cpu(), b_block)
    want, mag = ref.product(da, db)
    c = torch.full((M, N + 5), 7.0, dtype=t, device=DEV)
    h.gemm_fp8(a, sa, b, sb, c[:, :N], b_block=b_block)
    check_product(c[:, :N], want, mag, K, ref.unit_error(da, db))
    assert (c[:, N:] == 7).all()
    again = torch.empty(M, N, dtype=t, device=DEV)
    h.gemm_fp8(a, sa, b, sb, again, b_block=b_block)
    assert torch.equal(again, c[:, :N])


@pytest.mark.parametrize("M,N,counts,type,kernel", [
    (200, 130, [3, 0, 500, 128], "f16", fp8_rules.TILE64), (1100, 1000, [700, 0, 1, 650], "f32", fp8_rules.TILE128),
    (1100, 1000, [700, 0, 1, 650], "bf16", fp8_rules.TILE128), (1100, 1000, [700, 0, 1, 650], "f16", fp8_rules.TILE128),
    (1990, 2030, [700, 0, 129, 5], "f16", fp8_rules.TILE256)])
def test_weight_gradients_on_every_tile(h, M, N, counts, type, kernel):
    say(f"[case] wgrad {M}x{N} {counts} {type}")
    E, g, t = len(counts), gen(M + N), TYPES[type]
    assert fp8_rules.wgrad(M, N, E, type == "f32") == kernel
    off = offsets_of(counts, 128)
    R = int(off[-1])
    a, b, sa, sb = codes(g, M, R), codes(g, N, R), scales(g, R // 128, M), scales(g, R // 128, N)
    sa = sa * (1e-5 if type == "f16" else 1.0)
    da, db = ref.dequant(a.cpu(), sa.cpu()), ref.dequant(b.cpu(), sb.cpu())
    c = torch.full((E, M + 1, N + 1), 7.0, dtype=t, device=DEV)
    h.gemm_fp8_wgrad(a, sa, b, sb, off.to(DEV), c[:, :M, :N])
    for e in range(E):
        lo, hi = int(off[e]), int(off[e + 1])
        want, mag = ref.product(da[:, lo:hi], db[:, lo:hi])
        check_product(c[e, :M, :N], want, mag, hi - lo, ref.unit_error(da[:, lo:hi], db[:, lo:hi]))
    assert (c[:, M:] == 7).all() and (c[:, :, N:] == 7).all()
