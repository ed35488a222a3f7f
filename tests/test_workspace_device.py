"""A workspace on another device than the current one: it is zeroed and its status is read on the
stream where that device's calls run.  One device is enough here: what the library is handed is
looked at, nothing is run."""

import contextlib
import types

import pytest

torch = pytest.importorskip("torch")

import paged_kv_cache_sa_b200 as sa


class Buffer:
    is_cuda = True
    device = torch.device("cuda", 1)

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 4096


@pytest.fixture
def handed(monkeypatch):
    now, got = [0], []

    @contextlib.contextmanager
    def device(d):
        before, now[0] = now[0], torch.device(d).index
        yield
        now[0] = before

    def current_stream(d=None):
        return types.SimpleNamespace(cuda_stream=1000 + (now[0] if d is None
                                                         else torch.device(d).index))

    def record(*args):
        got.append((now[0], args[-1].value))
        return 0
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", current_stream)
    monkeypatch.setattr(sa, "lib", types.SimpleNamespace(sa_workspace_init=record,
                                                         sa_workspace_status=record))
    monkeypatch.setattr(sa, "_empty", lambda *a: Buffer())
    return got


def test_zeroed_and_read_on_its_own_device(handed):
    ws = sa.Workspace(256, device="cuda:1")
    ws.status()
    assert handed == [(1, 1001), (1, 1001)]


def test_a_given_stream_is_used(handed):
    stream = types.SimpleNamespace(cuda_stream=77)
    sa.Workspace(256, device="cuda:1", stream=stream).status(stream)
    assert handed == [(1, 77), (1, 77)]
