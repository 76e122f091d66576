"""Whose memory a call of the soft-assignment operators uses, no GPU needed:
the library is a fake that notes the pointers it is given."""

import pytest
import torch

import means_clustering_flashassign_b200 as km
from test_soft_checks import FakeCuda, fake_q, q_cpu


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream, self.device = handle, torch.device("cuda:0")


class FakeLibrary:
    """The library, but for the launches of km_scores: where their status words are."""

    def __init__(self, lib):
        self._lib, self.words = lib, []

    def __getattr__(self, name):
        return getattr(self._lib, name)

    def km_scores(self, *args):
        self.words.append(args[-3])
        return 0


@pytest.fixture
def calls(monkeypatch):
    fake = FakeLibrary(km.library())
    real, kept, capturing = torch.empty, [], []

    def empty(*a, device=None, **k):
        kept.append(real(*a, **k))      # nothing is freed: no address is given out twice
        return kept[-1]

    class On:
        def __init__(self, device, stream):
            self.raw = 0 if stream is None else stream.cuda_stream

        def __enter__(self):
            return self.raw

        def __exit__(self, *a):
            pass

    monkeypatch.setattr(km, "library", lambda: fake)
    monkeypatch.setattr(km, "_on", On)
    monkeypatch.setattr(km, "_status_words", {})
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: bool(capturing))

    def call(handle, captured=False):
        capturing[:] = [1] if captured else []
        out = FakeCuda(torch.zeros(6, 4))
        km.scores(fake_q(*q_cpu(6, 40)), fake_q(*q_cpu(4, 40)), out=out, stream=FakeStream(handle))
        return fake.words[-1]
    return call


def test_streams_do_not_share_a_status_word(calls):
    """Memory is in order on the stream that it was allocated on alone: work
    queued there before may still use it when another stream's call clears it."""
    a = calls(0x10)
    assert calls(0x20) != a
    assert calls(0x10) == a             # kept from call to call


def test_a_graph_has_a_status_word_of_its_own(calls):
    """A graph may be replayed on another stream than the one it was captured on."""
    a = calls(0x10)
    b = calls(0x10, captured=True)
    assert b != a and calls(0x10, captured=True) not in (a, b)
    assert calls(0x10) == a
