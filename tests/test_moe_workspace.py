"""Whose memory the workspace of a call is that allocates its own: that of the stream
the call runs on (no GPU is needed: torch's allocator and streams are stood in for).

Memory of another stream may still be read or written by work enqueued there, and
goes back to that stream's next allocation as soon as the call has returned."""
import contextlib
import ctypes as C
import types

import pytest
import torch

from tile_planned_generator_amd import dg

CURRENT, SIDE = 11, 22


class Stand:
    """torch, as far as a workspace needs it: `current` is the stream that owns what is allocated."""
    uint8 = "uint8"

    def __init__(self):
        self.current = CURRENT
        self.owners = []
        self.cuda = types.SimpleNamespace(stream=self.stream, ExternalStream=lambda s, device: ("external", s, device),
                                          default_stream=lambda device: ("external", 0, device))

    @contextlib.contextmanager
    def stream(self, s):
        before, self.current = self.current, s[1]
        yield
        self.current = before

    def empty(self, n, dtype, device):
        self.owners.append((self.current, n, device))
        return types.SimpleNamespace(record_stream=lambda s: None)


@pytest.mark.parametrize("stream,owner", [(None, CURRENT), (CURRENT, CURRENT), (SIDE, SIDE), (0, 0), (C.c_void_p(SIDE), SIDE),
                                          (C.c_void_p(0), 0)])
def test_the_workspace_is_the_calls_streams(monkeypatch, stream, owner):
    ty, stand = dg._types(), Stand()
    monkeypatch.setattr(ty, "torch", stand)
    monkeypatch.setattr(ty, "current_stream", lambda index: stand.current)
    ty.space(4096, types.SimpleNamespace(index=0), stream)
    assert [(s, n) for s, n, _ in stand.owners] == [(owner, 4096)] and stand.current == CURRENT


def test_planned_products_ask_for_their_streams_memory(monkeypatch):
    """The planned products (dg_gemm, dg_gemm_mx) take their own workspace in the same way."""
    asked = []
    monkeypatch.setattr(dg._Types, "space", lambda self, n, device, stream: asked.append((n, stream)) or
                        torch.empty(n, dtype=torch.uint8))
    for name in ("dg_gemm", "dg_gemm_mx"):
        monkeypatch.setattr(dg, name, lambda *a: dg.DG_OK)
    h = dg.Handle(offline=dg.default_device_desc())
    split = dg.dg_plan_opts(force_split_k=2, force_path=dg.DG_PATH_TILED)
    half, u8 = dict(dtype=torch.float16), dict(dtype=torch.uint8)
    one = h.gemm(torch.zeros(192, 512, **half), torch.zeros(512, 160, **half), torch.zeros(192, 160, **half),
                 opts=split, stream=SIDE)
    two = h.gemm_mx(torch.zeros(96, 1536, **u8), torch.zeros(48, 96, **u8), torch.zeros(160, 768, **u8),
                    torch.zeros(48, 160, **u8), torch.zeros(96, 160, **half), opts=split, stream=SIDE)
    h.close()
    assert one.workspace_bytes > 0 and two.workspace_bytes > 0
    assert asked == [(one.workspace_bytes, SIDE), (two.workspace_bytes, SIDE)]
