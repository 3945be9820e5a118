"""GPU: calls that allocate their own workspace on a stream that is not the current
one, while the memory they could wrongly take is in use: by work enqueued before
them on the current stream, or by allocations made there right after them."""
import pytest
import torch

from tests.parity import say
from tests.test_gpu_moe import DEV, codes, gen, h, scales  # noqa: F401 (h: fixture)
from tile_planned_generator_amd import dg

pytestmark = pytest.mark.gpu


def gemm(h):
    """A product cut along K: (its call, its output, the size of its workspace)."""
    g, (M, N, K) = gen(81), (100, 200, 3000)
    a, b, sa, sb = codes(g, M, K), codes(g, N, K), scales(g, 24, M), scales(g, 24, 2)
    out = torch.zeros(M, N, device=DEV)
    return (lambda s: h.gemm_fp8(a, sa, b, sb, out, stream=s)), out, h.plan_fp8(M, N, K).workspace_bytes


def sort(h):
    ids = torch.randint(-1, 64, (5000, 2), generator=gen(82), dtype=torch.int32).to(DEV)
    out = torch.zeros(65 + 20000, dtype=torch.int32, device=DEV)
    return (lambda s: h.moe_sort(ids, out[:65], out[65:10065], out[10065:].view(5000, 2), stream=s)), out, \
        h.moe_sort_workspace(5000, 2, 64)


def planned(h):
    """A planned product cut along K (dg_gemm)."""
    g, (M, N, K) = gen(83), (192, 160, 512)
    a, b = (torch.randn(*s, generator=g).half().to(DEV) for s in ((M, K), (K, N)))
    out, opts = torch.zeros(M, N, dtype=torch.float16, device=DEV), dg.dg_plan_opts(force_split_k=2, force_path=dg.DG_PATH_TILED)
    return (lambda s: h.gemm(a, b, out, opts=opts, stream=s)), out, \
        h.plan(M, N, K, opts=opts).workspace_bytes


class Busy:
    """Some tens of milliseconds of work on the current stream."""

    def __init__(self):
        self.x = torch.randn(4096, 4096, device=DEV)
        self.y = [torch.empty_like(self.x) for _ in range(2)]
        self()
        torch.cuda.synchronize()

    def __call__(self):
        for i in range(24):
            torch.mm(self.x, self.x, out=self.y[i & 1])


@pytest.fixture(scope="module")
def busy():
    torch.cuda.init()
    return Busy()


def result(call, out):
    call(None)
    torch.cuda.synchronize()
    want = out.clone()
    out.zero_()
    torch.cuda.synchronize()
    return want


@pytest.mark.parametrize("make", [gemm, sort, planned])
def test_memory_that_earlier_work_still_reads(h, busy, make):
    say(f"[case] own workspace, memory in use: {make.__name__}")
    call, out, need = make(h)
    assert need > 0
    want, side = result(call, out), torch.cuda.Stream()
    held = [torch.full((need,), 7, dtype=torch.uint8, device=DEV) for _ in range(8)]
    copies = [torch.zeros_like(t) for t in held]
    torch.cuda.synchronize()
    busy()
    for c, t in zip(copies, held):
        c.copy_(t)        # enqueued behind the work; then the memory goes back to this stream's allocations
    del held, t
    call(side.cuda_stream)
    torch.cuda.synchronize()
    assert all((c == 7).all() for c in copies) and torch.equal(out, want)


@pytest.mark.parametrize("make", [gemm, sort, planned])
@pytest.mark.parametrize("default", [False, True])
def test_memory_that_is_handed_out_after_the_call(h, busy, make, default):
    """`default`: the call names stream 0 while another stream is current."""
    say(f"[case] own workspace, memory handed out: {make.__name__}, {'stream 0' if default else 'side stream'}")
    call, out, need = make(h)
    want, side = result(call, out), torch.cuda.Stream()
    runs, current = (torch.cuda.default_stream(), side) if default else (side, torch.cuda.default_stream())
    with torch.cuda.stream(runs):
        busy()
    with torch.cuda.stream(current):
        call(0 if default else side.cuda_stream)
        filled = [torch.full((need,), 255, dtype=torch.uint8, device=DEV) for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(out, want) and all((t == 255).all() for t in filled)
