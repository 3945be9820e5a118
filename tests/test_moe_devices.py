"""Operands of the 8-bit expert layer that are not on the handle's GPU are refused
before the library is called, whether the call names a stream or not (no GPU is
needed: the library's calls are replaced by recorders)."""
import os
import types

import pytest
import torch

from tile_planned_generator_amd import dg

pytestmark = pytest.mark.skipif(not os.path.exists(dg.LIB_PATH),
                                reason="libdg.so not built (run __graft_entry__.build())")
CALLS = ["dg_quant_fp8", "dg_gemm_fp8", "dg_gemm_fp8_grouped", "dg_gemm_fp8_wgrad", "dg_moe_sort", "dg_moe_gather",
         "dg_moe_combine", "dg_moe_combine_grad"]
E, T, TOPK, N, K = 2, 4, 2, 64, 128


def u8(*shape):
    return torch.zeros(*shape, dtype=torch.uint8)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def z(*shape):
    return torch.zeros(*shape)


CALLED = {
    "quant_fp8": lambda h, **s: h.quant_fp8(z(T, K), u8(T, K), z(1, T), **s),
    "gemm_fp8": lambda h, **s: h.gemm_fp8(u8(T, K), z(1, T), u8(N, K), z(1, 1), z(T, N), **s),
    "gemm_fp8_with_a_workspace": lambda h, **s: h.gemm_fp8(u8(100, 3000 + 8)[:, :3000], z(24, 100), u8(200, 3008)[:, :3000],
                                                           z(24, 2), z(100, 200), **s),
    "gemm_fp8_grouped": lambda h, **s: h.gemm_fp8_grouped(u8(T, K), z(1, T), u8(E, N, K), z(E, 1, 1), i32(E + 1), z(T, N), **s),
    "gemm_fp8_wgrad": lambda h, **s: h.gemm_fp8_wgrad(u8(N, K), z(1, N), u8(N, K), z(1, N), i32(E + 1), z(E, N, N), **s),
    "moe_sort": lambda h, **s: h.moe_sort(i32(T, TOPK), i32(E + 1), i32(T * TOPK), i32(T, TOPK), **s),
    "moe_sort_with_a_workspace": lambda h, **s: h.moe_sort(i32(5000, 2), i32(E + 1), i32(10000), i32(5000, 2), **s),
    "moe_gather": lambda h, **s: h.moe_gather(z(T, K), i32(8), z(8, K), topk=TOPK, **s),
    "moe_combine": lambda h, **s: h.moe_combine(z(8, K), i32(T, TOPK), z(T, K), **s),
    "moe_combine_grad": lambda h, **s: h.moe_combine_grad(z(T, K), z(8, K), i32(T, TOPK), i32(8), z(8, K), z(T, TOPK), **s),
}


@pytest.fixture()
def calls(monkeypatch):
    seen = []
    for name in CALLS:
        monkeypatch.setattr(dg, name, lambda *a: seen.append(a) or dg.DG_OK)
    h = dg.Handle(offline=dg.default_device_desc())
    yield h, seen
    h.close()


@pytest.mark.parametrize("stream", [None, 0, 4096])
@pytest.mark.parametrize("name", CALLED)
def test_host_operands_are_refused(calls, name, stream):
    h, seen = calls
    with pytest.raises(ValueError, match="GPU"):
        CALLED[name](h, stream=stream)
    assert not seen


def test_operands_of_another_gpu_are_refused():
    h = types.SimpleNamespace(index=0)
    for stream in (0, 4096):
        assert dg._stream(h, torch.device("cuda", 0), stream) == stream
        with pytest.raises(ValueError, match="cuda:1"):
            dg._stream(h, torch.device("cuda", 1), stream)


def test_a_handle_knows_its_device(calls):
    assert calls[0].index is None   # (offline: the library refuses to launch)
