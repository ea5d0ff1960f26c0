"""The cache operators' binding: devices, copies and concurrent use of a
configuration (no GPU needed)."""
import contextlib
import copy
import dataclasses
import pickle
import sys

import pytest

import long_context_prefill_last_b200 as crisp

torch = pytest.importorskip("torch")


class OnDevice:
    """A tensor's face on a device that is not there."""

    def __init__(self, t, index):
        self.t, self.device = t, torch.device("cuda", index)

    def get_device(self):
        return self.device.index

    def __getattr__(self, name):
        return getattr(self.t, name)


class Machine:
    """A stand-in for the library and for torch's current device and streams (stream number 100 + device)."""

    def __init__(self, monkeypatch):
        self.current, self.calls = 0, []
        stream = type("Stream", (), {})

        def current_stream(device=None):
            s = stream()
            s.cuda_stream = 100 + (self.current if device is None else torch.device("cuda", device).index)
            return s

        @contextlib.contextmanager
        def device(index):
            before, self.current = self.current, index
            yield
            self.current = before

        def status(cfg, stream, out):
            self.calls.append((self.current, getattr(stream, "value", stream)))
            return 0

        monkeypatch.setattr(torch.cuda, "current_stream", current_stream)
        monkeypatch.setattr(torch.cuda, "device", device)
        monkeypatch.setattr(crisp, "lib", lambda: type("L", (), {"crisp_cache_device_status": staticmethod(status)}))


def test_device_status_runs_on_the_workspace_s_device(monkeypatch):
    m = Machine(monkeypatch)
    cfg = crisp.CacheConfig(batch=1, n_q=1, n_k=16, h_q=2, h_kv=1)
    cfg.workspace = OnDevice(torch.zeros(256, dtype=torch.uint8), 1)
    assert crisp.cache_device_status(cfg) == 0
    assert m.calls == [(1, 101)] and m.current == 0
    own = type("Stream", (), {"cuda_stream": 77})()
    crisp.cache_device_status(cfg, own)
    assert m.calls[-1] == (1, 77)


def test_device_status_without_a_device_workspace_is_refused():
    cfg = crisp.CacheConfig(batch=1, n_q=1, n_k=16, h_q=2, h_kv=1)
    with pytest.raises(crisp.CrispError):
        crisp.cache_device_status(cfg)
    cfg.workspace = torch.zeros(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        crisp.cache_device_status(cfg)


NAMES = ("k",)


def used():
    cfg = crisp.CacheConfig(batch=1, n_q=1, n_k=16, h_q=2, h_kv=2, window=5)
    cfg._ref(NAMES, [torch.zeros(1, 2, 16, 128)])
    return cfg


@pytest.mark.parametrize("make", [copy.copy, copy.deepcopy, lambda c: pickle.loads(pickle.dumps(c)),
                                  dataclasses.replace], ids=["copy", "deepcopy", "pickle", "replace"])
def test_a_used_configuration_can_be_copied(make):
    cfg = used()
    other = make(cfg)
    assert other == cfg and other.window == 5
    t = [torch.zeros(1, 2, 16, 128)]
    ref = cfg._ref(NAMES, t)
    assert other._ref(NAMES, t)._obj is not ref._obj
    other.window = 9
    assert other._ref(NAMES, t)._obj.window == 9 and cfg._ref(NAMES, t) is ref and ref._obj.window == 5


def test_two_threads_calls_get_their_own_structures():
    """Another call on the same configuration, between any two lines of this one."""
    dense, sparse = [torch.zeros(1, 2, 16, 128)], [torch.zeros(1, 16, 2, 128).transpose(1, 2)]
    cfg = used()
    cfg.window = 6

    def interrupt(frame, event, arg):
        if frame.f_code.co_name != "_ref":
            return None
        if event == "line":
            sys.settrace(None)
            cfg._ref(NAMES, sparse)
            sys.settrace(interrupt)
        return interrupt

    sys.settrace(interrupt)
    try:
        ref = cfg._ref(NAMES, dense)
    finally:
        sys.settrace(None)
    assert ref._obj.k.head == dense[0].stride(1)


def test_a_workspace_resized_in_place_is_noticed():
    cfg = crisp.CacheConfig(batch=1, n_q=1, n_k=16, h_q=2, h_kv=2)
    cfg.workspace = torch.zeros(256, dtype=torch.uint8)
    t = [torch.zeros(1, 2, 16, 128)]
    assert cfg._ref(NAMES, t)._obj.workspace_bytes == 256
    cfg.workspace.resize_(1 << 20)
    c = cfg._ref(NAMES, t)._obj
    assert c.workspace == cfg.workspace.data_ptr() and c.workspace_bytes == 1 << 20
