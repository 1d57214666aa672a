"""CPU: where the binding takes the cached attention's workspace from."""
import pytest

from streaming_speaker_diarization_b200 import binding as b

torch = pytest.importorskip("torch")


@pytest.fixture
def taken(monkeypatch):
    """The stream that was current at each allocation, with torch's streams replaced by plain values."""
    at, got = ["current"], []

    class On:
        def __init__(self, stream):
            self.stream = stream

        def __enter__(self):
            at.append(self.stream)

        def __exit__(self, *_):
            at.pop()

    real = torch.empty
    monkeypatch.setattr(torch.cuda, "stream", On)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda s, device=None: ("external", s, device))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: ("default", device))
    monkeypatch.setattr(torch, "empty", lambda *a, **kw: got.append(at[-1]) or real(*a, **kw))
    return got


def test_a_workspace_comes_from_the_pool_of_the_stream_that_uses_it(taken):
    """The allocator orders a block's uses by the stream it was taken on, so it is taken on the stream of the call."""
    q = torch.zeros(1)
    for stream in (None, 0x7f1234567890, 0, 1):
        assert b._scratch(48, q, stream).numel() == 48
    cpu = q.device
    assert taken == ["current", ("external", 0x7f1234567890, cpu), ("default", cpu), ("default", cpu)]
