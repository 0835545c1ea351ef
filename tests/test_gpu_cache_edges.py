"""The smaller cache's operators at values that ordinary inputs do not have: long tails behind one heavy key, NaN and infinite keys
in hidden places, rows whose page is none together with their weights.  Tolerances as in test_gpu_cache.py."""
import numpy as np
import pytest
import torch

import oracle.cache_oracle as co
import tests.test_gpu_cache as cases
from mla_attention_gb300 import mla_decode_fp4
from tests.helpers import dev, to_np

pytestmark = pytest.mark.gpu

SCALE = 192 ** -0.5


def _rows(cache, table, b, js):
    """Pages and rows of keys js of request b."""
    page = cache.shape[1]
    return table[b].cpu()[torch.as_tensor(js) // page].long(), torch.as_tensor(js) % page


def _put_pe(raw, table, b, j, column, value):
    """RoPE column `column` of key j of request b in a 4-bit cache on the host."""
    pg, r = _rows(raw, table, b, [j])
    raw[pg[0], r[0], 288 + 2 * column:290 + 2 * column] = torch.tensor([value]).bfloat16().view(torch.uint8)


# ---------------------------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("below", [12.0, 18.5, 20.0])
def test_decode_a_heavy_key_and_a_long_tail(below):
    """A first key without a value and 20000 others, e^-below of its weight each, whose values are all positive: all of the result is theirs.
    A weight keeps an error of 2^-32 of the largest, so 2^-5 of itself at e^-18.5 (2^-26.7)."""
    n, page, H = 20001, 64, 3
    cache, table, keys = cases._paged("fp4", [n], page, 90)
    raw = cache.cpu()
    pg, r = _rows(raw, table, 0, list(range(n)))
    raw[pg, r, :256] &= 0x77                       # no signs
    raw[pg[0], r[0], :256] = 0
    top = float(torch.tensor(below / (SCALE * 8.0)).bfloat16())
    raw[pg, r, 288:290] = 0
    _put_pe(raw, table, 0, 0, 0, top)
    keys = [co.fp4_values(raw[pg, r].numpy())]
    q = cases._query(1, 1, H, 90, 0.01)
    q[..., 512] = 8.0
    qn = to_np(q)
    ro, rl = co.decode(qn, keys, SCALE)
    out, lse = mla_decode_fp4(q.to(dev()), raw.to(dev()), 1.0, table, cases._i32([n]), SCALE, num_splits=1)
    cases._done()
    bo, bl = np.zeros(ro.shape), np.zeros(rl.shape)
    v = keys[0][:, :512]
    for h in range(H):
        size = SCALE * (np.abs(keys[0]) @ np.abs(qn[0, 0, h])).max()
        ds = cases.SCORE * size + SCALE * 2.0 ** -25 * np.abs(keys[0]).sum(1).max()
        w = np.exp(SCALE * (keys[0] @ qn[0, 0, h]) - rl[0, 0, h])
        # 20000 fp32 sums besides, sixteen at a time, of values of one sign: 1250 additions at 2^-23
        bo[0, 0, h] = cases.BF16 * ro[0, 0, h] + (2 * ds + cases.F16 + cases.EXP + 1250 * 2.0 ** -23) * (w @ v) + 2.0 ** -32 * v.sum(0) * w.max()
        bl[0, 0, h] = 2 * ds + cases.EXP + 2.0 ** -21 * abs(rl[0, 0, h]) + 1250 * 2.0 ** -23
    assert (bo < 0.1 * ro + 1e-9).mean() > 0.9 if below < 19 else True
    cases._within(lse, rl, bl, "lse")
    cases._within(out, ro, bo, "out")


@pytest.mark.parametrize("s,H,scale", [(3, 16, 0.07), (3, 16, -0.07), (10, 16, 0.07), (2, 128, 0.07), (130, 1, 0.07)])
@pytest.mark.parametrize("nan", [0x7F, 0xFF])
def test_decode_a_nan_reaches_the_tokens_that_see_it_alone(s, H, scale, nan):
    """A NaN scale in a request's last key, in the last but one, and in one that all tokens see."""
    lens, page = [200, 200, 200, 200], 16
    cache, table, keys = cases._paged("fp4", lens, page, 91)
    raw = cache.cpu()
    for b, j in ((0, 199), (1, 198), (2, 200 - s)):
        pg, r = _rows(raw, table, b, [j])
        raw[pg[0], r[0], 256 + 7 * b] = nan
    q = cases._query(4, s, H, 91)
    ro, rl = co.decode(to_np(q), keys, scale)
    out, lse = mla_decode_fp4(q.to(dev()), raw.to(dev()), 1.0, table, cases._i32(lens), scale)
    cases._done()
    bo, bl = cases._decode_bounds(to_np(q), keys, scale, None, ro, rl)
    for b, seen in ((0, s - 1), (1, s - 2), (2, 0), (3, s)):       # tokens from `seen` on see the NaN
        cases._within(out[b, :seen], ro[b, :seen], bo[b, :seen], "out")
        cases._within(lse[b, :seen], rl[b, :seen], bl[b, :seen], "lse")
        assert torch.isnan(out[b, seen:]).all() and torch.isnan(lse[b, seen:]).all()
