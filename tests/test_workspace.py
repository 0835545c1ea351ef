"""The binding's cached workspaces, on host memory (CPU only)."""
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
