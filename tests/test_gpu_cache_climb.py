"""mla_decode_fp4 where a row's running maximum rises behind the first tile of a share, so that O is scaled while more is to be
added to it.  One key of each row stands out by 5.4 to 6.5 nats (2^8 is 5.545): what came before it, the other keys of its tile and
the key itself all stay a visible part of the result."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import oracle.cache_oracle as co
import tests.test_gpu_cache as cases
from mla_attention_gb300 import build, mla_decode_fp4
from tests.helpers import dev, to_np

pytestmark = pytest.mark.gpu

SCALE, COLUMNS, Q = 192 ** -0.5, 8, 13.875
# the key that stands out for the rows of each column: in either half of a tile, first and last of a half, in tiles 1 to 11
PEAKS = [[130, 197, 320, 575, 576, 700, 1152, 1407], [128, 191, 192, 255, 390, 480, 645, 699]]
LENS = [1500, 700]


def _climbing(climb, H, s, sign, seed):
    """Cache, table, keys and queries: row (i, h) has the climb at PEAKS[request][(i + h) % COLUMNS]."""
    page = 64
    cache, table, keys = cases._paged("fp4", LENS, page, seed)
    raw = cache.cpu()
    top = float(torch.tensor(climb / (SCALE * Q)).bfloat16())
    for b, n in enumerate(LENS):
        pe = torch.zeros((n, COLUMNS))
        for j, at in enumerate(PEAKS[b]):
            pe[at, j] = top
        bits = pe.bfloat16().view(torch.uint8).reshape(n, 2 * COLUMNS)
        for j in range(n):
            raw[table[b][j // page].item(), j % page, 288:288 + 2 * COLUMNS] = bits[j]
        keys[b][:, 512:512 + COLUMNS] = pe.double().numpy()
    q = cases._query(2, s, H, seed, 0.02)
    q[..., 512:512 + COLUMNS] = 0
    for i in range(s):
        for h in range(H):
            q[:, i, h, 512 + (i + h) % COLUMNS] = sign * Q
    return raw.to(dev()), table, keys, q


def _check_climb(climb, H, s, splits, sign, seed=70, repeats=20):
    cache, table, keys, q = _climbing(climb, H, s, sign, seed)
    qn, scale = to_np(q), sign * SCALE
    ro, rl = co.decode(qn, keys, scale)
    bo, bl = cases._decode_bounds(qn, keys, scale, None, ro, rl)
    d, L = q.to(dev()), cases._i32(LENS)
    first = None
    for _ in range(repeats):
        out, lse = mla_decode_fp4(d, cache, 1.0, table, L, scale, num_splits=splits)
        cases._done()
        if first is None:
            first = out, lse
            cases._within(lse, rl, bl, "lse")
            cases._within(out, ro, bo, "out")
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])


@pytest.mark.parametrize("climb", [5.4, 5.7, 6.5])
@pytest.mark.parametrize("splits", [1, 2, 5])
@pytest.mark.parametrize("sign", [1, -1])
def test_climb(climb, splits, sign):
    """Rows in both CTAs of a pair, each with its climb in a tile of its own."""
    _check_climb(climb, 128, 1, splits, sign)


@pytest.mark.parametrize("H,s", [(1, 1), (20, 1), (64, 1), (65, 1), (40, 2), (64, 2), (128, 2)])
def test_climb_rows(H, s):
    _check_climb(6.0, H, s, 1, 1, seed=71, repeats=5)


def test_climb_in_every_tile():
    """The maximum rises by 6.2 nats in the second half of each tile: O is scaled behind every one."""
    n, page, H = 1500, 64, 128
    cache, table, keys = cases._paged("fp4", [n], page, 72)
    raw = cache.cpu()
    level = torch.tensor([6.2 * ((j + 64) // 128) for j in range(n)]) / (SCALE * Q)
    bits = level.bfloat16().view(torch.uint8).reshape(n, 2)
    for j in range(n):
        raw[table[0][j // page].item(), j % page, 288:290] = bits[j]
    keys[0][:, 512] = level.bfloat16().double().numpy()
    q = cases._query(1, 1, H, 72, 0.02)
    q[..., 512] = Q
    qn = to_np(q)
    ro, rl = co.decode(qn, keys, SCALE)
    out, lse = mla_decode_fp4(q.to(dev()), raw.to(dev()), 1.0, table, cases._i32([n]), SCALE, num_splits=1)
    cases._done()
    bo, bl = cases._decode_bounds(qn, keys, SCALE, None, ro, rl)
    cases._within(lse, rl, bl, "lse")
    cases._within(out, ro, bo, "out")


def test_the_climbs_are_visible():
    """What a lost half tile, a lost O or a scaling too many would change is far above the bounds (in the oracle, on the host)."""
    cache, table, keys, q = _climbing(6.0, 8, 1, 1, 70)
    qn = to_np(q)
    ro, rl = co.decode(qn, keys, SCALE)
    bo, _ = cases._decode_bounds(qn, keys, SCALE, None, ro, rl)
    for b in range(2):
        for h in range(8):
            at = PEAKS[b][h]
            tile, w = at // 128 * 128, np.exp(SCALE * (keys[b] @ qn[b, 0, h]) - rl[b, 0, h])
            assert (w[at] > 0.1 and w[:tile].sum() > 0.05)
            for part in (slice(0, tile), slice(tile, tile + 64), slice(tile + 64, tile + 128)):
                part = np.arange(len(w))[part]
                if len(part) and (at in part or part[0] == 0):
                    lost = np.abs(w[part] @ keys[b][part, :512])
                    assert (lost > bo[b, 0, h]).mean() > 0.8, (b, h, part[:1])


def test_climb_through_the_guarded_build():
    path = build.build(guard=True)
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, os.path.join(here, "guarded_cache_climb_cases.py"), path], capture_output=True, text=True,
                       timeout=900, cwd=os.path.dirname(here))
    assert r.returncode == 0 and "guarded ok" in r.stdout, (r.stdout[-3000:] + r.stderr[-3000:])
