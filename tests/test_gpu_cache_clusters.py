"""The smaller cache's calls where their grids change shape (requests that share clusters of sixteen CTAs, of fewer, of one; wide
rows; keys that do not fit a CTA), as a process's first calls captured into a graph, and with a wait that cannot finish."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle.cache_oracle as co
import tests.test_gpu_cache as cases
from mla_attention_gb300 import (MLAError, check_device_status, inject_stall, mla_compact_rows, mla_decode_fp4, mla_key_weights,
                                 mla_select_keys, set_spin_limit)
from tests.helpers import dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B", [1, 2, 19, 20, 38, 39, 76, 77, 152, 153])
@pytest.mark.parametrize("row", [416, 1152])
def test_compact_by_requests(B, row):
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 400, (B,), generator=g).tolist()
    lens[0] = 1500
    cases._check_compact(lens, row, 16, [int(n * 0.7) for n in lens], B)


@pytest.mark.parametrize("row,B", [(65536, 2), (1920 * 16, 1), (1921 * 16, 3), (128, 1), (144, 40)])
def test_compact_wide_rows(row, B):
    cases._check_compact([60, 13, 33][:min(B, 3)] + [5] * (B - 3), row, 4, [40, 6, 33][:min(B, 3)] + [2] * (B - 3), row, weights=B != 2)


@pytest.mark.parametrize("n,keep", [(40000, 39000), (40000, 17), (200, 199)])
def test_compact_one_long_request(n, keep):
    cases._check_compact([n], 48, 64, [keep], n + keep)


@pytest.mark.parametrize("fmt", cases.FORMATS)
@pytest.mark.parametrize("s,H", [(129, 1), (2, 80), (7, 23), (3, 85), (2, 128), (257, 1), (17, 16), (3, 100)])
def test_weights_around_two_chunks(fmt, s, H):
    """Query rows around 128 and 256 (129, 160, 161, 255, 256, 257, 272, 300), keys around 128, 256 and a range of 2048."""
    cases._check_weights(fmt, [0, 1, 127, 129, 255, 256, 257, 2048, 2300, 600], H, s=s, page=16, seed=s + H)


@pytest.mark.parametrize("fmt", ["e4m3", "fp4"])
def test_weights_of_many_chunks_repeat_bit_for_bit(fmt):
    cache, table, keys = cases._paged(fmt, [5000, 300, 2049], 64, 4, poison=False)
    q, L = cases._query(3, 12, 128, 4).to(dev()), cases._i32([5000, 300, 2049])
    lse = torch.full((3, 12, 128), 5.0, device=dev())
    first = None
    for _ in range(10):
        w = torch.zeros((3, 5000), device=dev())
        mla_key_weights(q, lse, cache, table, L, 0.07, w, decay=0.0)
        cases._done()
        first = w if first is None else first
        assert torch.equal(w, first)


@pytest.mark.parametrize("B", [1, 19, 20, 38, 39, 76, 77, 152, 153])
def test_select_by_requests(B):
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 3000, (B,), generator=g).tolist()
    lens[0] = 3000
    w = torch.randint(0, 40, (B, 3000), generator=g).float()           # many equal ones, over several CTAs
    cases._check_select(w, lens, [n // 3 for n in lens], 1000, 3, 9)


def test_select_keys_that_one_cta_cannot_hold():
    B, W = 160, 26000
    w = torch.zeros((B, W))
    w[5] = torch.rand(W, generator=torch.Generator().manual_seed(6)) - 0.5
    w[7] = torch.randint(0, 3, (W,), generator=torch.Generator().manual_seed(7)).float()
    lens, keep = [0] * B, [0] * B
    lens[5], keep[5] = 26000, 25000
    lens[7], keep[7] = 25999, 900
    cases._check_select(w, lens, keep, 25000, 4, 100)


@pytest.mark.parametrize("B", [1, 30, 200])
@pytest.mark.parametrize("swap", [False, True])
def test_select_counts_in_place(B, swap):
    """count in the place of lens and dropped in that of keep, or the other way round: read by all before they are written."""
    g = torch.Generator().manual_seed(B)
    w = torch.rand((B, 3000), generator=g)
    lens = torch.randint(0, 3000, (B,), generator=g)
    keep = torch.randint(0, 3000, (B,), generator=g)
    lens[0], keep[0] = 3000, 1700
    ref = co.select_keys(w.double().numpy(), lens.tolist(), keep.tolist(), 3000, 3, 9)
    d, first = w.to(dev()), [lens.int().to(dev()), keep.int().to(dev())]
    for _ in range(20):
        L, K = (t.clone() for t in first)
        idx, count, dropped = mla_select_keys(d, L, K, 3000, first=3, recent=9, count=K if swap else L, dropped=L if swap else K)
        cases._done()
        for a, b in zip((idx, count, dropped), ref):
            np.testing.assert_array_equal(a.cpu().numpy(), b)


FIRST = """
import sys
sys.path.insert(0, %r)
import torch
import tests.test_gpu_cache as cases
from mla_attention_gb300 import check_device_status, mla_compact_rows, mla_decode_fp4, mla_key_weights, mla_select_keys
d = torch.device("cuda", 0)
cache, table, keys = cases._paged("fp4", [300, 77], 16, 3, poison=False)
q, L, keep = cases._query(2, 1, 16, 3).to(d), cases._i32([300, 77]), cases._i32([64, 20])
w = torch.zeros((2, 320), device=d)
def step():
    out, lse = mla_decode_fp4(q, cache, 1.0, table, L, 0.07)
    mla_key_weights(q, lse, cache, table, L, 0.07, w, decay=0.0)
    idx, count, dropped = mla_select_keys(w, L, keep, 64, first=1, recent=8)
    mla_compact_rows(cache, table, idx, count, weights=w)
    return out, lse, idx, count, dropped
first = cache.clone()
mla_select_keys(w[:, :8], cases._i32([8, 8]), cases._i32([4, 4]), 4)    # the status word, which a capture cannot make
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    held = step()
graph.replay()
torch.cuda.synchronize()
check_device_status()
got = [t.clone() for t in (*held, cache, w)]
cache.copy_(first)
for a, b in zip(got, (*step(), cache, w)):
    assert torch.equal(a, b)
check_device_status()
print("first calls ok")
"""


def test_first_launches_of_a_process_are_captured():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST % root], capture_output=True, text=True, timeout=300, cwd=root)
    assert r.returncode == 0 and "first calls ok" in r.stdout, r.stdout[-2000:] + r.stderr[-2000:]


def _expect_timeout(run):
    check_device_status()
    set_spin_limit(4096)
    inject_stall(True)
    try:
        run()
        torch.cuda.synchronize()
    finally:
        inject_stall(False)
        set_spin_limit(0)
    with pytest.raises(MLAError) as e:
        check_device_status()
    assert e.value.status == 4
    check_device_status()   # the word was cleared


@pytest.mark.parametrize("fmt", cases.FORMATS)
def test_key_weights_timeout(fmt):
    cache, table, keys = cases._paged(fmt, [700, 70], 16, 1, poison=False)
    q, L, w = cases._query(2, 1, 16, 1).to(dev()), cases._i32([700, 70]), torch.zeros((2, 704), device=dev())
    lse = torch.full((2, 1, 16), 9.0, device=dev())
    run = lambda: mla_key_weights(q, lse, cache, table, L, 0.07, w, decay=0.0)    # noqa: E731
    _expect_timeout(run)
    run()
    torch.cuda.synchronize()
    check_device_status()
    assert torch.isfinite(w).all() and (w[0, :700] > 0).all()


def test_decode_timeout():
    cache, table, keys = cases._paged("fp4", [700, 70], 16, 2, poison=False)
    q, L = cases._query(2, 1, 16, 2).to(dev()), cases._i32([700, 70])
    run = lambda: mla_decode_fp4(q, cache, 1.0, table, L, 0.07)    # noqa: E731
    want, _ = run()
    _expect_timeout(run)
    out, _ = run()
    torch.cuda.synchronize()
    check_device_status()
    assert torch.equal(out, want)


def test_compact_timeout_moves_nothing():
    cache = torch.randint(0, 256, (64, 16, 416), dtype=torch.uint8, device=dev())
    table, idx = torch.arange(64, dtype=torch.int32, device=dev()).reshape(1, 64), torch.arange(1, 1001, 2, dtype=torch.int32, device=dev())[None]
    before = cache.clone()
    _expect_timeout(lambda: mla_compact_rows(cache, table, idx, cases._i32([500])))
    assert torch.equal(cache, before)
    mla_compact_rows(cache, table, idx, cases._i32([500]))
    torch.cuda.synchronize()
    check_device_status()
    rows = before.reshape(1024, 416)
    assert np.array_equal(cache.reshape(1024, 416)[:500].cpu().numpy(), rows[1:1001:2].cpu().numpy())
