"""The binding's cached workspaces and status words, on host memory (CPU only)."""
import pytest
import torch

from mla_attention_gb300 import _lib, workspace

CPU = torch.device("cpu")


@pytest.fixture(autouse=True)
def own_caches(monkeypatch):
    monkeypatch.setattr(_lib, "_ws_cache", {})
    monkeypatch.setattr(_lib, "_ws_outgrown", [])


def test_a_need_that_creeps_upward_keeps_less_than_twice_the_buffer():
    for need in range(1000, 600_000, 500):       # a batch that grows by one request a step
        ws = workspace(need, CPU)
        assert ws.numel() >= need
    held = ws.numel() + sum(w.numel() for w in _lib._ws_outgrown)
    assert ws.numel() <= 2 * 600_000 and held < 2 * ws.numel()


def test_outgrown_buffers_stay_and_a_large_enough_one_is_kept():
    """A captured graph may hold their addresses."""
    first = workspace(1000, CPU)
    assert workspace(10, CPU) is first and not workspace(1000, CPU).any()
    second = workspace(5000, CPU)
    assert second.numel() == 5000 and any(w is first for w in _lib._ws_outgrown)
    assert workspace(256, CPU) is second


def test_where_twice_the_size_does_not_fit_the_need_is_enough(monkeypatch):
    zeros, first = torch.zeros, workspace(1000, CPU)

    def small(n, **k):
        if n > 1500:
            raise torch.cuda.OutOfMemoryError("no")
        return zeros(n, **k)

    monkeypatch.setattr(torch, "zeros", small)
    assert workspace(1200, CPU).numel() == 1200 and first.numel() == 1000


class Words:
    """The C calls that read a status word, over words on the host."""

    def __init__(self, codes):
        self.codes, self.last = codes, b""       # by address

    def mla_check_device_status(self, ptr, stream, detail):
        code, self.codes[ptr.value] = self.codes.get(ptr.value, 0), 0
        detail._obj.value = code
        self.last = b"" if code == 0 else b"site 0x%x" % code
        return 0 if code == 0 else 4 if code < 0x2000 else 5

    def mla_last_error_string(self):
        return self.last


@pytest.mark.parametrize("own,step,status,told", [(0, 0, 0, []), (0x1011, 0, 4, ["0x1011"]), (0, 0x2071, 5, ["0x2071"]),
                                                  (0x1011, 0x2071, 4, ["0x1011", "0x2071"])])
def test_a_status_check_tells_of_every_fault_that_it_clears(monkeypatch, own, step, status, told):
    a, b = torch.zeros(256, dtype=torch.uint8), torch.zeros(256, dtype=torch.uint8)
    words = Words({a.data_ptr(): own, b.data_ptr(): step})
    monkeypatch.setattr(_lib, "lib", lambda: words)
    monkeypatch.setattr(_lib, "workspace", lambda n, device: a)
    monkeypatch.setattr(_lib, "_status_cache", {0: b})
    if not status:
        assert _lib.check_device_status(device="cuda:0", stream=0) == 0
        return
    with pytest.raises(_lib.MLAError) as e:
        _lib.check_device_status(device="cuda:0", stream=0)
    assert e.value.status == status and all(t in str(e.value) for t in told)
    assert _lib.check_device_status(device="cuda:0", stream=0) == 0 and not any(words.codes.values())


def test_a_fault_in_an_outgrown_workspace_is_reported(monkeypatch):
    """A graph captured before the workspace grew reports in the old one, and its kernels give up their waits until it is cleared."""
    old, new = workspace(256, CPU), workspace(9000, CPU)
    words = Words({old.data_ptr(): 0x1011, new.data_ptr(): 0})
    monkeypatch.setattr(_lib, "lib", lambda: words)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    with pytest.raises(_lib.MLAError) as e:
        _lib.check_device_status(device=CPU, stream=0)
    assert e.value.status == 4
    assert _lib.check_device_status(device=CPU, stream=0) == 0 and not any(words.codes.values())
