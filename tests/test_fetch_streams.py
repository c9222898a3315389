"""Which stream's memory the fetch's outputs are (CPU only: allocator and entry point are
stand-ins that record what they are asked)."""
import contextlib
from types import SimpleNamespace
from unittest import mock

import pytest
import torch

import zero_partitioned_optimizer_amd as Z
from zero_partitioned_optimizer_amd import _binding as B


@pytest.fixture
def seen(monkeypatch):
    """Streams that tensors were allocated on, that they were recorded on and that the
    copies went to; the current stream is 7."""
    current = [SimpleNamespace(cuda_stream=7)]
    got = SimpleNamespace(made=[], used=[], copies=[])

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def empty(*size, **kw):
        got.made.append(current[-1].cuda_stream)
        t = mock.MagicMock()
        t.record_stream.side_effect = lambda s: got.used.append(s.cuda_stream)
        return t

    def plan(shards, S, offsets, numels, outs):
        def run(stream=None):
            got.copies.append(B._stream(stream))
            return outs
        return run

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[-1])
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, *a: SimpleNamespace(cuda_stream=h))
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(B, "GatherPlan", plan)
    return got


def shards():
    return [SimpleNamespace(dtype=torch.bfloat16, device="cuda:0", get_device=lambda: 0)] * 2


@pytest.mark.parametrize("stream", [SimpleNamespace(cuda_stream=9), 9], ids=["stream", "handle"])
def test_outputs_belong_to_the_copies_stream(seen, stream):
    """Memory from the current stream's pool may still be in use there when the copies on
    another stream write it, and goes back to that pool while this stream reads it."""
    assert len(Z.zero_gather_tensors(shards(), 64, [0, 8, 16], [8, 8, 4], stream=stream)) == 3
    assert seen.copies == [9] and seen.made == [9, 9, 9]
    assert seen.used == [7, 7, 7]               # a caller may read them on its own stream


def test_outputs_of_the_current_stream(seen):
    Z.zero_gather_tensors(shards(), 64, [0], [8])
    Z.zero_gather_tensors(shards(), 64, [0], [8], stream=7)
    assert seen.copies == [7, 7] and seen.made == [7, 7] and seen.used == []


def test_layer_fetch_on_a_stream(seen):
    layer = Z.FlatLinear([0, 16], [12, 4], 0, 1, 3, 4)
    layer.fetch(shards(), 64, stream=SimpleNamespace(cuda_stream=9))
    assert seen.copies == [9] and seen.made == [9, 9] and seen.used == [7, 7]
    layer.release()
    layer.fetch(shards(), 64)
    assert seen.copies == [9, 7] and seen.made == [9, 9, 7, 7]
