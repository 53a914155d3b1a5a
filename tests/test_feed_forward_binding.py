"""The feed-forward operators' Python face: streams, devices, handles' lifetimes and imports, with stand-ins for
the GPU's side."""
import contextlib
import os
import subprocess
import sys
from types import SimpleNamespace

import pytest
import torch

from shot_allreduce_ranks_gb300 import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


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


@pytest.fixture
def destroyed(ff, monkeypatch, devices):
    calls = []
    monkeypatch.setattr(ff, "load", lambda: SimpleNamespace(ar_ffn_destroy=lambda h: calls.append((devices[0], h)) or 0))
    return calls


def test_a_handle_dropped_during_a_capture_is_freed_after_it(ff, monkeypatch, destroyed):
    capturing = [True]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    a, b = handle(ff, 1), handle(ff, 0)
    del a
    assert destroyed == []
    with pytest.raises(RuntimeError, match="captured"):
        b.close()
    assert destroyed == [] and b._h == 99
    capturing[0] = False
    b.close()
    assert sorted(destroyed) == [(0, 99), (1, 99)]
    b.close()
    assert len(destroyed) == 2


def test_a_handle_without_a_workspace_is_freed_at_any_time(ff, monkeypatch, destroyed):
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: True)
    a = handle(ff, 0, train=False)
    del a
    assert destroyed == [(0, 99)]


def test_a_captured_handle_is_freed_by_close_alone(ff, monkeypatch, destroyed):
    capturing = [True]
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing[0])
    monkeypatch.setattr(ff, "_ops", SimpleNamespace(ffn_backward=lambda *a: None))
    a, b = handle(ff), handle(ff)
    for h in (a, b):
        h.backward(*[None] * 6)
    capturing[0] = False
    del a
    assert destroyed == []
    b.close()
    assert destroyed == [(0, 99)]


def test_a_star_import_does_not_need_the_library():
    code = ("import shot_allreduce_ranks_gb300._lib as lib\n"
            "lib.PKG = '/nonexistent'\n"
            "from shot_allreduce_ranks_gb300 import *\n"
            "assert AllReduce and GatedFFN and dropout\n"
            "try:\n"
            "    dropout(None, 0.5, 1)\n"
            "except RuntimeError as e:\n"
            "    assert 'not built' in str(e), e\n"
            "else:\n"
            "    raise SystemExit('a missing binding went unnoticed')\n")
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
