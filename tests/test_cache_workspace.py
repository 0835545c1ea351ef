"""The workspaces of the smaller cache's calls through the binding, on host memory (CPU only: nothing is launched)."""
import types

import pytest
import torch

from mla_attention_gb300 import _cache, _lib, _step
from tests.test_step_binding import Shaped, bf16, i32


class OnGpu(torch.Tensor):
    """Host memory that says it is GPU 0's."""

    def get_device(self):
        return 0


class On:
    """torch.cuda.stream: which is current."""

    now = "current"

    def __init__(self, stream):
        self.stream = stream

    def __enter__(self):
        self.was, On.now = On.now, self.stream

    def __exit__(self, *_):
        On.now = self.was


@pytest.fixture
def calls(monkeypatch):
    """The C calls stand-ins record what they get; buffers are host memory."""
    got, zeros = {}, torch.zeros

    def call(name):
        return lambda *a: got.__setitem__(name, a) or 0

    names = ("mla_decode_fp4", "mla_key_weights")
    fake = types.SimpleNamespace(**{n: call(n) for n in names}, **{n + "_workspace_size": lambda *a: 9000 for n in names})
    monkeypatch.setattr(_lib, "lib", lambda: fake)
    monkeypatch.setattr(_step, "_functions", {})
    for name in ("_ws_cache", "_scratch_cache", "_status_cache"):
        monkeypatch.setattr(_lib, name, {}, raising=False)
    monkeypatch.setattr(_lib, "_ws_outgrown", [])
    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, **k: zeros(*a, **k).as_subclass(OnGpu))
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: types.SimpleNamespace(synchronize=lambda: None))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda dev=None: 0)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, dev=None: handle)
    monkeypatch.setattr(torch.cuda, "stream", On)
    return got


def _decode(stream=0):
    _cache.mla_decode_fp4(bf16(2, 2, 128, 576), Shaped(torch.uint8, 8, 16, 416), 1.0, i32(2, 4), i32(2), 0.1, out=bf16(2, 2, 128, 512),
                          lse=Shaped(torch.float32, 2, 2, 128), stream=stream)


def _weights():
    _cache.mla_key_weights(bf16(2, 2, 128, 576), Shaped(torch.float32, 2, 2, 128), Shaped(torch.uint8, 8, 16, 416), i32(2, 4), i32(2), 0.1,
                           Shaped(torch.float32, 2, 64), stream=0)


@pytest.mark.parametrize("call,name", [(_decode, "mla_decode_fp4"), (_weights, "mla_key_weights")])
def test_scratch_is_not_the_attentions(calls, call, name):
    """The attention's kernels give up their waits while the word at the start of their workspace is set; these calls record
    lengths that were cut, which is no reason to."""
    attention = _lib.workspace(20000, torch.device("cuda", 0))
    call()
    assert calls[name][-2] >= 9000 or calls[name][-3] >= 9000
    assert attention.data_ptr() not in calls[name]
    call()
    scratch = _lib._scratch_cache[("cuda", 0)]
    assert scratch.data_ptr() in calls[name] and not any(w is scratch for w in _lib._ws_cache.values())


def test_what_the_scratch_records_is_told(calls, monkeypatch):
    from tests.test_workspace import Words
    _decode()
    scratch = _lib._scratch_cache[("cuda", 0)]
    own = _lib.workspace(256, torch.device("cuda", 0))
    words = Words({own.data_ptr(): 0, scratch.data_ptr(): 0x207B})
    monkeypatch.setattr(_lib, "lib", lambda: words)
    monkeypatch.setattr(torch.Tensor, "device", property(lambda t: torch.device("cuda", 0)))
    with pytest.raises(_lib.MLAError) as e:
        _lib.check_device_status(device="cuda:0", stream=0)
    assert e.value.status == 5 and "0x207b" in str(e.value)
    assert _lib.check_device_status(device="cuda:0", stream=0) == 0


@pytest.mark.parametrize("capturing", [False, True])
def test_a_new_buffer_is_filled_before_the_call_that_asked_for_it(calls, monkeypatch, capturing):
    """The call may be on another stream than the current one, on which the zeros are written; a capture cannot wait."""
    waited = []
    stream = types.SimpleNamespace(synchronize=lambda: waited.append(dict(calls)))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: stream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: capturing)
    _decode()
    assert waited == ([] if capturing else [{}])         # once, before the call
    _decode()
    _lib.workspace(100, torch.device("cuda", 0))
    assert len(waited) == (0 if capturing else 2)


@pytest.mark.parametrize("stream", [0, 1 << 40])
def test_a_new_buffer_is_filled_on_the_streams_of_the_call(calls, monkeypatch, stream):
    """In a capture with several streams the zeros come before the call's kernels, not beside them at each replay."""
    zeros, on = torch.zeros, []
    monkeypatch.setattr(torch, "zeros", lambda *a, **k: on.append(On.now) or zeros(*a, **k))
    _decode(stream)
    assert on == [stream] and On.now == "current"
