"""GPU: what the fp8 matrix unit, which sums the blocks of 16-bit outputs, keeps of its
products.  Inside each group of 8 consecutive k it cuts every product towards zero at
2^-13 of the group's largest one (the largest sum of the two factors' exponents);
everything else is binary32.  Products with binary32 outputs are exact."""
import math

import pytest
import torch

from tests.parity import say
from tests.test_gpu_moe import DEV, F8, fp8_empty, h  # noqa: F401 (h: fixture)

pytestmark = pytest.mark.gpu
BIG, FAR, GROUP = 8, 40, range(8, 16)   # places along k of the large product and of its opposite


def ones_product(h, a, b, type):
    M, N = a.shape[0], b.shape[0]
    c = torch.empty(M, N, dtype=type, device=DEV)
    one = torch.ones(1, max(M, N), device=DEV)
    h.gemm_fp8(a.to(F8).to(DEV), one[:, :M], b.to(F8).to(DEV), one[:, :N], c, b_block=1)
    return c.double().cpu()


@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("place", [9, 15, 7, 16, 70, 127])
def test_what_a_large_product_hides(h, place, sign):
    """2^12 and, in another group, -2^12 leave the small product alone, or nothing of it."""
    say(f"[case] small product at k = {place}, sign {sign}")
    powers = list(range(8, -10, -1))                  # the small product is sign * 2^(j + 4), 2^(j - 8) of the large one
    a, b = torch.zeros(64, 128), torch.full((64, 128), 16.0)
    for r, j in enumerate(powers):
        a[r, BIG], a[r, FAR], a[r, place] = 256, -256, sign * 2.0 ** j
    want = torch.tensor([sign * 2.0 ** (j + 4) for j in powers], dtype=torch.float64)
    kept = torch.tensor([place not in GROUP or j - 8 >= -13 for j in powers])
    got = ones_product(h, a, b, torch.float16)[:len(powers)]
    assert (got == (want * kept)[:, None]).all()
    assert (ones_product(h, a, b, torch.float32)[:len(powers)] == want[:, None]).all()


def cut_sum(a, b):
    """Sums over k of a b^T (binary64 values with e4m3 factors), every product cut as above."""
    K = a.shape[1]
    pad = -K % 8
    a, b = (torch.nn.functional.pad(t, (0, pad)) for t in (a, b))

    def exponent(t):
        return torch.floor(torch.log2(t.abs().clamp_min(2.0 ** -9)))
    out = torch.empty(a.shape[0], b.shape[0], dtype=torch.float64)
    eb = exponent(b)
    for i in range(a.shape[0]):
        p = (a[i] * b).view(b.shape[0], -1, 8)
        e = torch.where(p != 0, (exponent(a[i]) + eb).view_as(p), -100.0).amax(2, keepdim=True)
        step = torch.exp2(e - 13)
        out[i] = (torch.trunc(p / step) * step).sum((1, 2))
    return out


@pytest.mark.parametrize("spread", [False, True])
def test_the_cut_on_activations(h, spread):
    """The slices of a product cut along K, which are binary32, against the model and
    against the exact sums; `spread`: rows of other magnitudes and a few large columns.

    The binary32 sums add one error of at most a step (2^-23) per group and two per
    block, independent of each other: sqrt(count) steps of the result's norm.  The
    cut itself comes out at 1.4e-5 of it (2.7e-5 with `spread`), several times that."""
    say(f"[case] the cut on activations, spread {spread}")
    M, N, K = 60, 120, 3000
    g = torch.Generator().manual_seed(91)
    x, w = torch.randn(M, K, generator=g), torch.randn(N, K, generator=g)
    if spread:
        x *= torch.exp2(4 * torch.rand(M, 1, generator=g) - 2)
        x *= 1 + 15 * (torch.rand(1, K, generator=g) < 0.01)
    ops = []
    for t in (x, w):
        q, s = fp8_empty(*t.shape), torch.empty(-(-K // 128), t.shape[0], device=DEV)
        h.quant_fp8(t.to(DEV), q, s)
        ops += [q, s]
    a, sa, b, sb = ops
    info = h.plan_fp8(M, N, K)
    assert info.split_k > 1
    ws = torch.empty(info.workspace_bytes // 4, device=DEV)
    h.gemm_fp8(a, sa, b, sb, torch.empty(M, N, dtype=torch.bfloat16, device=DEV), b_block=1, workspace=ws)
    got = ws.view(info.split_k, M, N).double().sum(0).cpu()
    va, vb = a.float().double().cpu(), b.float().double().cpu()
    model, want = torch.zeros(M, N, dtype=torch.float64), torch.zeros(M, N, dtype=torch.float64)
    for k in range(0, K, 128):
        f = sa[k // 128].double().cpu()[:, None] * sb[k // 128].double().cpu()[None]
        model += f * cut_sum(va[:, k:k + 128], vb[:, k:k + 128])
        want += f * (va[:, k:k + 128] @ vb[:, k:k + 128].t())
    sums = math.sqrt(-(-K // 8) + 2 * -(-K // 128)) * 2.0 ** -23
    cut, off = ((model - want).norm() / want.norm()).item(), ((got - model).norm() / want.norm()).item()
    print(f"cut {cut:.3g} of the norm, kernel from the model {off:.3g}, bound {sums:.3g}")
    assert off <= sums
    assert sums < cut <= (4e-5 if spread else 2e-5)
    c = torch.empty(M, N, device=DEV)
    h.gemm_fp8(a, sa, b, sb, c, b_block=1, workspace=ws)
    assert ((c.double().cpu() - want).norm() / want.norm()).item() <= sums
