"""The feed-forward operators' Python face: streams, devices, handles' lifetimes and imports, with stand-ins for
the GPU's side."""
import contextlib
from types import SimpleNamespace

import pytest
import torch

from shot_allreduce_ranks_gb300 import build


@pytest.fixture(scope="module")
def ff():
    build.build()
    from shot_allreduce_ranks_gb300 import feed_forward
    return feed_forward


def on(index):
    return SimpleNamespace(device=torch.device("cuda", index), cuda_stream=70 + index)


def handle(ff, index=0, train=True):
    h = ff.GatedFFN.__new__(ff.GatedFFN)
    h.device, h.train, h._h, h._constants = torch.device("cuda", index), train, 99, (99,)
    return h


@pytest.fixture
def devices(monkeypatch):
    """Which device is current, as `torch.cuda.device` sets it."""
    now = [0]

    @contextlib.contextmanager
    def device(d):
        before, now[0] = now[0], torch.device("cuda", d).index if isinstance(d, int) else d.index
        yield
        now[0] = before

    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    return now


def test_a_stream_of_another_device_is_refused(ff, monkeypatch, devices):
    def used(stream):
        raise AssertionError("the stream was used")

    monkeypatch.setattr(torch.cuda, "stream", used)
    x, s = on(0), on(1)
    ffn = handle(ff)
    ffn._h = None  # nothing to free
    for call in (lambda: ffn.forward(x, x, x, stream=s), lambda: ffn.backward(x, x, x, x, x, x, stream=s),
                 lambda: ff.dropout(x, 0.5, 1, stream=s), lambda: ff.dropout_backward(x, 0.5, 1, stream=s),
                 lambda: ff.quantize_rows(x, stream=s), lambda: ff.linear_i8(x, x, x, x, stream=s)):
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            call()


def test_the_status_is_read_on_the_streams_device(ff, monkeypatch, devices):
    read = []
    lib = SimpleNamespace(ar_ops_get_device_status=lambda s: read.append((devices[0], s)) or 0)
    monkeypatch.setattr(ff, "load", lambda: lib)
    assert ff.ops_device_status(on(1)) == 0
    assert read == [(1, 71)]
