"""Whose memory the workspace of a call is that allocates its own: that of the stream
the call runs on (no GPU is needed: torch's allocator and streams are stood in for).

Memory of another stream may still be read or written by work enqueued there, and
goes back to that stream's next allocation as soon as the call has returned."""
import contextlib
import types

import pytest

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


@pytest.mark.parametrize("stream,owner", [(None, CURRENT), (CURRENT, CURRENT), (SIDE, SIDE), (0, 0)])
def test_the_workspace_is_the_calls_streams(monkeypatch, stream, owner):
    ty, stand = dg._types(), Stand()
    monkeypatch.setattr(ty, "torch", stand)
    monkeypatch.setattr(ty, "current_stream", lambda index: stand.current)
    ty.space(4096, types.SimpleNamespace(index=0), stream)
    assert [(s, n) for s, n, _ in stand.owners] == [(owner, 4096)] and stand.current == CURRENT
