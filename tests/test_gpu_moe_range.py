"""GPU: the 8-bit expert layer where element and byte offsets pass 32 bits.  Values are
small whole numbers, so every result is exact; the far ends are compared."""
import pytest
import torch

from tests import moe_ref as ref
from tests.parity import say
from tests.test_gpu_moe import DEV, F8, gen, h  # noqa: F401 (h: fixture)
from tile_planned_generator_amd import dg

pytestmark = pytest.mark.gpu
ROWS, H = 1 << 21, 2056     # 4.3e9 elements


@pytest.fixture(scope="module")
def rows():
    torch.cuda.init()
    x = torch.zeros(ROWS, H, dtype=torch.bfloat16, device=DEV)
    x[-300:] = torch.randint(-7, 8, (300, H), generator=gen(1)).to(torch.bfloat16).to(DEV)
    x[0] = 3
    yield x
    del x
    torch.cuda.empty_cache()


def test_movement(h, rows):
    say(f"[case] movement, {ROWS} x {H}")
    g, T, k = gen(2), 50, 2
    pick = (ROWS - 1 - torch.randperm(300, generator=g)[:T * k]).int()
    pick[0], pick[1] = 0, -1
    want = rows[pick.clamp_min(0).long().to(DEV)]
    want[1] = 0
    y = torch.empty(T * k, H, dtype=torch.bfloat16, device=DEV)
    h.moe_gather(rows, pick.to(DEV), y, topk=1)
    assert torch.equal(y, want)
    w = 2.0 ** torch.randint(-1, 2, (T, k), generator=g)
    o = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    dst = pick.view(T, k).to(DEV)
    h.moe_combine(rows, dst, o, weights=w.to(DEV))
    assert torch.equal(o, (want.view(T, k, H).double() * w.to(DEV)[..., None]).sum(1).to(torch.bfloat16))
    # the gradient: every row of 2^21 is written
    do = torch.randint(-7, 8, (T, H), generator=g).to(torch.bfloat16).to(DEV)
    src = torch.full((ROWS,), -1, dtype=torch.int32)
    flat = pick.tolist()
    for p, r in enumerate(flat):
        if r >= 0:
            src[r] = p
    dy = torch.full((ROWS, H), 7.0, dtype=torch.bfloat16, device=DEV)
    dw = torch.empty(T, k, device=DEV)
    h.moe_combine_grad(do, rows, dst, src.to(DEV), dy, dw, weights=w.to(DEV))
    live = [p for p in range(T * k) if flat[p] >= 0]
    at = torch.tensor([flat[p] for p in live], device=DEV)
    grad = (do[torch.tensor(live, device=DEV) // k].double() * w.view(-1)[live].to(DEV)[:, None]).to(torch.bfloat16)
    assert torch.equal(dy[at], grad)
    dy[at] = 0
    assert not any(part.any() for part in dy.split(1 << 18))
    terms = want[live].double() * do[torch.tensor(live, device=DEV) // k].double()
    assert torch.equal(dw.double().view(-1)[live], terms.sum(1))


@pytest.mark.parametrize("transpose", [False, True])
def test_quantiser(h, rows, transpose):
    say(f"[case] quantiser, {ROWS} x {H}, transpose {transpose}")
    m, n = (H, ROWS) if transpose else (ROWS, H)
    q = torch.full((m, n), 0x7f, dtype=torch.uint8, device=DEV).view(F8)
    s = torch.full((-(-n // 128), m), -1.0, device=DEV)
    h.quant_fp8(rows, q, s, transpose=transpose)
    tail = rows[-384:].double().cpu()
    wc, ws = ref.quant_rows(tail.t().contiguous() if transpose else tail)
    if transpose:
        assert torch.equal(q[:, -384:].double().cpu(), wc) and torch.equal(s[-3:].double().cpu(), ws)
    else:
        assert torch.equal(q[-384:].double().cpu(), wc) and torch.equal(s[:, -384:].double().cpu(), ws)


def test_experts(h):
    """80 experts of 8192 x 8192: 5.4e9 weights, and as many elements of their gradients."""
    E, N, K, R = 80, 8192, 8192, 80 * 128
    say(f"[case] {E} experts of {N} x {K}")
    g = gen(3)
    off = torch.arange(E + 1, dtype=torch.int32, device=DEV) * 128
    b = torch.zeros(E, N, K, dtype=torch.uint8, device=DEV).view(F8)
    last = torch.randint(-3, 4, (N, K), generator=g).float()
    b[-1] = last.to(F8).to(DEV)
    x = torch.randint(-3, 4, (R, K), generator=g).float()
    c = torch.full((R, N), 7.0, device=DEV)
    h.gemm_fp8_grouped(x.to(F8).to(DEV), torch.ones(K // 128, R, device=DEV), b,
                       torch.ones(E, K // 128, N // 128, device=DEV), off, c)
    want = x[-128:].to(DEV) @ last.t().contiguous().to(DEV)     # whole numbers below 2^24
    assert torch.equal(c[-128:], want) and not c[:-128].any()
    del b, c
    dy = torch.randint(-3, 4, (N, R), generator=g).float()
    for t in (torch.float32, torch.bfloat16):
        dw = torch.full((E, N, K), 7.0, dtype=t, device=DEV)
        h.gemm_fp8_wgrad(dy.to(F8).to(DEV), torch.ones(R // 128, N, device=DEV), x.t().contiguous().to(F8).to(DEV),
                         torch.ones(R // 128, K, device=DEV), off, dw)
        for e in (0, E // 2, E - 1):
            seg = slice(e * 128, (e + 1) * 128)
            assert torch.equal(dw[e], (dy[:, seg].to(DEV) @ x[seg].to(DEV)).to(t))
        del dw
    torch.cuda.empty_cache()


def test_the_largest_launch(h):
    """A wave moves a row's piece: 2^26 of them pass one launch's 2^32 work-items, and are refused."""
    most, H = (1 << 26) - 4, 2
    say(f"[case] gather of {most} rows")
    x = torch.arange(12, dtype=torch.bfloat16, device=DEV).view(6, H)
    src = torch.randint(-1, 6, (most + 4,), generator=torch.Generator(device=DEV).manual_seed(5), dtype=torch.int32, device=DEV)
    y = torch.full((most + 4, H), 7.0, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(dg.DGError) as e:
        h.moe_gather(x, src, y, topk=1)
    assert e.value.status == dg.DG_ERR_UNSUPPORTED
    torch.cuda.synchronize()
    assert (y == 7).all()
    h.moe_gather(x, src[:most], y[:most], topk=1)
    want = torch.cat([torch.zeros(1, H, dtype=torch.bfloat16, device=DEV), x])[src[:most].long() + 1]
    assert torch.equal(y[:most], want) and (y[most:] == 7).all()
