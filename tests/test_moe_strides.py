"""What the 8-bit expert layer's wrapper passes on as strides and refuses, without a
GPU: the library's calls are replaced by recorders, so nothing is launched."""
import os

import pytest
import torch

from tests import fp8_rules
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


def wgrad(h, C_out):
    h.gemm_fp8_wgrad(f8(N, 256), torch.zeros(2, N), f8(K, 256), torch.zeros(2, K), i32(E + 1), C_out)


def test_a_gradient_expanded_over_the_experts_is_refused(calls):
    """All experts but the first would be written past the tensor's end."""
    h, seen = calls
    with pytest.raises(ValueError, match="expert"):
        wgrad(h, torch.zeros(1, N, K).expand(E, N, K))
    assert not seen
    wgrad(h, torch.zeros(E, N, K))
    wgrad(h, torch.zeros(N, E, K).transpose(0, 1))   # rows of the experts side by side
    assert [(a[-3], a[-2]) for a in seen] == [(K, N * K), (E * K, K)]


@pytest.mark.parametrize("M,N,ld,stride,experts,ok", [
    (8, 256, 256, 8 * 256, 4, True), (8, 256, 300, 7 * 300 + 256, 4, True), (8, 256, 300, 7 * 300 + 255, 4, False),
    (8, 256, 256, 256, 4, False), (8, 256, 4 * 256, 256, 4, True), (8, 256, 4 * 256 - 1, 256, 4, False),
    (8, 256, 1 << 20, 255, 4, False), (1, 256, 256, 256, 9, True), (1, 256, 256, 255, 9, False), (8, 256, 256, 1, 1, True),
    (0, 256, 256, 1, 4, True), (2 ** 31 - 1, 1, 2 ** 62, 2 ** 61, 4, False), (2, 1, 2 ** 62, 2 ** 61, 3, False),
    (2, 1, 2 ** 62, 2 ** 60, 4, True)])
def test_when_the_experts_gradients_share_no_element(M, N, ld, stride, experts, ok):
    assert bool(fp8_rules.lib().experts_disjoint(M, N, ld, stride, experts)) == ok
    if M * experts < 100:   # the definition, on the smaller pitches
        starts = [e * stride + m * ld for e in range(experts) for m in range(M)]
        starts.sort()
        assert all(b - a >= N for a, b in zip(starts, starts[1:])) == ok
