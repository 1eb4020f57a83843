"""A workspace that a call allocates by itself comes from the memory of the
stream that the call runs on (no GPU needed)."""
import contextlib

import pytest
import torch

import paged_kv_cache_311_gb300 as pkv


class Stream:
    """As torch.cuda.Stream and ExternalStream look from outside."""

    def __init__(self, handle=77, device=None):
        self.cuda_stream = handle


@pytest.mark.parametrize("given", [Stream(), 77, "torch"])
def test_scratch_is_allocated_on_the_calls_stream(monkeypatch, given):
    entered, inside = [], []

    @contextlib.contextmanager
    def on(stream):
        entered.append(stream.cuda_stream)
        yield
        entered.pop()

    empty = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, **k: (inside.append(list(entered)), empty(*a, **k))[1])
    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "ExternalStream", Stream)
    if given == "torch":
        monkeypatch.setattr(torch.cuda, "Stream", Stream)
        given = Stream()
    t = pkv._scratch(256, torch.zeros(1), given)
    assert t.numel() == 256 and t.dtype == torch.uint8
    assert inside == [[77]] and not entered


def test_scratch_without_a_stream_is_the_current_ones(monkeypatch):
    monkeypatch.setattr(torch.cuda, "stream", None)   # not entered
    assert pkv._scratch(16, torch.zeros(1), None).numel() == 16
