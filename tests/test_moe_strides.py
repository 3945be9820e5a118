"""What the 8-bit expert layer's wrapper passes on as strides and refuses, without a
GPU: the library's calls are replaced by recorders, so nothing is launched."""
import os

import pytest
import torch

from tile_planned_generator_amd import dg

pytestmark = pytest.mark.skipif(not os.path.exists(dg.LIB_PATH),
                                reason="libdg.so not built (run __graft_entry__.build())")
E, R, N, K = 4, 12, 8, 256
KB, NB = 2, 1


@pytest.fixture()
def calls(monkeypatch):
    """(a handle without a device, the argument lists that reached the library)"""
    seen = []
    for name in ("dg_gemm_fp8_grouped", "dg_gemm_fp8_wgrad"):
        monkeypatch.setattr(dg, name, lambda *a: seen.append(a) or dg.DG_OK)
    monkeypatch.setattr(dg, "_stream", lambda *a: 0)
    h = dg.Handle(offline=dg.default_device_desc())
    yield h, seen
    h.close()


def f8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


def i32(n):
    return torch.zeros(n, dtype=torch.int32)


def grouped(h, B, SB, experts=E):
    h.gemm_fp8_grouped(f8(R, K), torch.zeros(KB, R), B, SB, i32(experts + 1), torch.zeros(R, N))


@pytest.mark.parametrize("which", ["B", "SB", "both"])
def test_operands_expanded_over_the_experts_are_refused(calls, which):
    """Their expert stride is 0, which the library takes for tightly packed."""
    h, seen = calls
    B, SB = f8(E, N, K), torch.zeros(E, KB, NB)
    if which in ("B", "both"):
        B = f8(1, N, K).expand(E, N, K)
    if which in ("SB", "both"):
        SB = torch.ones(1, KB, NB).expand(E, KB, NB)
    with pytest.raises(ValueError, match="expert"):
        grouped(h, B, SB)
    assert not seen


def test_one_expert_and_other_strides_are_passed_on(calls):
    h, seen = calls
    grouped(h, f8(N, K).expand(1, N, K), torch.zeros(KB, NB).expand(1, KB, NB), experts=1)
    grouped(h, f8(E, N + 3, K)[:, :N], torch.zeros(KB, E, NB).transpose(0, 1))
    packed, other = seen
    # (ldb, the experts' stride of B; ldb_scale, the experts' stride of the scales; 0 and N K mean the same for one expert)
    assert packed[10] == K and packed[11] in (0, N * K) and packed[14] in (0, KB * NB)
    assert other[10] == K and other[11] == (N + 3) * K and other[13] == E * NB and other[14] == NB
