"""A captured graph keeps the layer's buffers that it uses (CPU: the capture is a stand-in)."""
import gc
import weakref

import pytest
import torch

from moe_gqa_query_b200 import layer as mod


@pytest.fixture
def layer(monkeypatch):
    capturing = [False]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    self = object.__new__(mod.GQELayer)
    self.device, self._bufs, self._captured = torch.device("cpu"), {}, {}
    return self, capturing


def test_a_buffer_lives_on_when_a_captured_call_used_it(layer):
    """Two captured steps of different shapes, or a captured one and an eager one: each name has one
    current buffer, and replays of the first graph still write into its own."""
    self, capturing = layer
    for made_in_capture in (False, True):
        capturing[0] = made_in_capture
        ref = weakref.ref(self._buf("t_q", (2, 8, 64)))
        ws = weakref.ref(self._ws("t_ws", 1000))
        capturing[0] = True
        self._buf("t_q", (2, 8, 64)), self._ws("t_ws", 1000)
        capturing[0] = False
        assert self._buf("t_q", (2, 4, 64)) is not ref()
        self._ws("t_ws", 5000)
        gc.collect()
        assert ref() is not None and ws() is not None


def test_a_buffer_of_eager_calls_alone_is_released(layer):
    self, _ = layer
    ref = weakref.ref(self._buf("t_q", (2, 8, 64)))
    self._buf("t_q", (2, 4, 64))
    gc.collect()
    assert ref() is None
