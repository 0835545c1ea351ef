"""The smaller cache's operators at values that ordinary inputs do not have: long tails behind one heavy key, NaN and infinite keys
in hidden places, rows whose page is none together with their weights.  Tolerances as in test_gpu_cache.py."""
import numpy as np
import pytest
import torch

import oracle.cache_oracle as co
import tests.test_gpu_cache as cases
from mla_attention_gb300 import mla_compact_rows, mla_decode_ex, mla_decode_fp4, mla_key_weights, mla_prefill
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


@pytest.mark.parametrize("scale", [2e5, 1e6, 4e6, -4e6, 1.5e7])
def test_decode_scores_whose_steps_are_large(scale):
    """Scores of 2^24 to 2^30, where fp32 has steps of 2 to 128: a weight may be off by many powers of two, but it is a number, and the
    output lies among the values; that of a key far above all others is the output."""
    lens, H = [300, 129, 64, 1000], 64
    cache, table, keys = cases._paged("fp4", lens, 64, 97)
    q = cases._query(len(lens), 1, H, 97)
    qn = to_np(q)
    for splits in (0, 1, 3):
        out, lse = mla_decode_fp4(q.to(dev()), cache, 1.0, table, cases._i32(lens), scale, num_splits=splits)
        cases._done()
        o, e, plain = to_np(out), to_np(lse), 0
        assert np.isfinite(o).all() and np.isfinite(e).all()
        for b, k in enumerate(keys):
            raw = np.sign(scale) * (k @ qn[b, 0].T)                   # [keys, H]
            error = cases.SCORE * (np.abs(k) @ np.abs(qn[b, 0]).T).max(0) + 2.0 ** -22 * np.abs(raw).max(0)
            v = k[:, :512]
            assert (o[b, 0] <= v.max(0) + cases.BF16 * np.abs(v).max(0)).all() and (o[b, 0] >= v.min(0) - cases.BF16 * np.abs(v).max(0)).all()
            top, second = np.sort(raw, 0)[-1], np.sort(raw, 0)[-2]
            clear = top - second > 2 * error + 1e2 / abs(scale)
            plain += clear.sum()
            best = v[raw.argmax(0)]
            assert (np.abs(o[b, 0] - best) <= cases.BF16 * np.abs(best))[clear].all()
            assert (np.abs(e[b, 0] - abs(scale) * top) <= abs(scale) * 2 * error + 10).all()
        assert plain > 200


# ---------------------------------------------------------------------------------------------
# the keys' weights
# ---------------------------------------------------------------------------------------------
def _with_bf16(cache, table, fmt, keys, b, j, column, value):
    """The cache with RoPE column `column` of a key set, bf16 in both formats."""
    raw = cache.cpu()
    if fmt == "fp4":
        _put_pe(raw, table, b, j, column, value)
    else:
        pg, r = _rows(raw, table, b, [j])
        raw[pg[0], r[0], 512 + column] = value
    keys[b][j, 512 + column] = value
    return raw.to(dev())


@pytest.mark.parametrize("fmt", ["bf16", "fp4"])
@pytest.mark.parametrize("s,H", [(1, 16), (1, 32), (1, 40), (1, 128), (3, 16), (2, 80), (3, 100), (9, 64)])
def test_weights_of_an_infinite_key(fmt, s, H):
    """A key with scores of -inf in every row has the weight 0, whatever the number of rows."""
    lens, n = [300, 70], 60
    cache, table, keys = cases._paged(fmt, lens, 64, 92)
    q = cases._query(2, s, H, 92)
    q[..., 512] = q[..., 512].abs() + 0.5
    qn = to_np(q)
    cache = _with_bf16(cache, table, fmt, keys, 0, n, 0, -float("inf"))
    cache = _with_bf16(cache, table, fmt, keys, 1, n, 0, -float("inf"))
    _, rl = co.decode(qn, [np.delete(k, n, 0) for k in keys], 0.07)
    w = torch.ones((2, 300), device=dev())
    mla_key_weights(q.to(dev()), torch.tensor(rl, dtype=torch.float32).to(dev()), cache, table, cases._i32(lens), 0.07, w, decay=0.5)
    cases._done()
    assert w[0, n] == 0.5 and w[1, n] == 0.5 and torch.isfinite(w).all()
    ref = co.key_weights(qn, rl, keys, 0.07, np.ones((2, 300)), 0.5)
    finite = [np.nan_to_num(k, neginf=0.0) for k in keys]
    cases._within(w, ref, cases._weight_bounds(qn, rl, finite, 0.07, ref), "weights")


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "fp4"])
@pytest.mark.parametrize("s,H", [(1, 16), (1, 32), (1, 128), (2, 128), (3, 100), (5, 64)])
def test_weights_rows_with_an_infinite_lse_add_nothing(fmt, s, H):
    """-inf and +inf add nothing over a NaN key either; a NaN key shows in its weight where a row of a finite one sees it."""
    lens, n = [300, 300], 61
    cache, table, keys = cases._paged(fmt, lens, 64, 93)
    raw = cache.cpu().view(torch.uint8)
    for b in range(2):
        pg, r = _rows(raw, table, b, [n])
        raw[pg[0], r[0], 256 if fmt == "fp4" else 0] = 0x7F
        if fmt == "bf16":
            raw[pg[0], r[0], 0], raw[pg[0], r[0], 1] = 0xC0, 0x7F
    cache = raw.to(dev()).view(cache.dtype)
    q = cases._query(2, s, H, 93)
    qn = to_np(q)
    _, rl = co.decode(qn, [np.delete(k, n, 0) for k in keys], 0.07)
    rl[0] = -np.inf
    rl[0, :, 1::2] = np.inf
    rl[1, :, ::3] = -np.inf
    w = torch.ones((2, 300), device=dev())
    mla_key_weights(q.to(dev()), torch.tensor(rl, dtype=torch.float32).to(dev()), cache, table, cases._i32(lens), 0.07, w)
    cases._done()
    assert (w[0] == 1).all()
    assert torch.isnan(w[1, n])
    w[1, n], ref = 1, co.key_weights(qn, rl, keys, 0.07, np.ones((2, 300)), 1.0)
    ref[1, n] = 1
    cases._within(w, ref, cases._weight_bounds(qn, rl, keys, 0.07, ref), "weights")


def test_weights_of_a_score_that_gave_an_infinite_lse():
    """A key with a score of +inf, and the log-sum-exp of +inf that it leads to: the row adds nothing, to that key neither."""
    lens, n = [150], 33
    cache, table, keys = cases._paged("bf16", lens, 64, 94)
    q = cases._query(1, 1, 32, 94)
    q[..., 512] = torch.where(torch.arange(32) % 2 == 0, 1.0, -1.0).bfloat16()
    qn = to_np(q)
    cache = _with_bf16(cache, table, "bf16", keys, 0, n, 0, float("inf"))
    _, rl = co.decode(qn, [np.delete(k, n, 0) for k in keys], 0.07)
    rl[:, :, ::2] = np.inf
    w = torch.zeros((1, 150), device=dev())
    mla_key_weights(q.to(dev()), torch.tensor(rl, dtype=torch.float32).to(dev()), cache, table, cases._i32(lens), 0.07, w)
    cases._done()
    assert w[0, n] == 0
    odd = co.key_weights(qn[:, :, 1::2], rl[:, :, 1::2], keys, 0.07, np.zeros((1, 150)), 1.0)
    finite = [np.nan_to_num(k, posinf=0.0) for k in keys]
    cases._within(w, odd, cases._weight_bounds(qn, rl, finite, 0.07, odd), "weights")


# ---------------------------------------------------------------------------------------------
# the moves
# ---------------------------------------------------------------------------------------------
def test_compact_weights_stay_with_rows_whose_page_is_none():
    """Rows that are not moved, since they or their places have no page, keep their weights."""
    page, lens = 4, 12
    cache = torch.arange(8 * page * 16, dtype=torch.int32).reshape(8, page, 16).to(torch.uint8)
    w0 = torch.rand((3, lens), generator=torch.Generator().manual_seed(95))
    table = cases._i32([[0, 8, 2], [-1, 4, 5], [6, 7, 1]])           # the second page of request 0, the first of request 1 are none
    idx = [[5, 6, 8, 9, 10, 11], [4, 5, 6, 8, 9, 11], [1, 2, 3, 5, 8, 11]]
    for K in (6, 300):
        wide = torch.full((3, K), -1, dtype=torch.int32)
        wide[:, :6] = torch.tensor(idx, dtype=torch.int32)
        d, w = cache.to(dev()), w0.to(dev())
        mla_compact_rows(d, table, wide.to(dev()), cases._i32([6, 6, 6]), weights=w)
        assert "0x7d" in cases._faults()
        ref, rw = cache.clone(), w0.clone()
        host = table.cpu()
        for b in range(3):
            for i, j in enumerate(idx[b]):
                src, dst = int(host[b, j // page]), int(host[b, i // page])
                if 0 <= src < 8 and 0 <= dst < 8:
                    ref[dst, i % page] = ref[src, j % page]
                    rw[b, i] = rw[b, j]
        assert torch.equal(d.cpu(), ref) and torch.equal(w.cpu(), rw)


# ---------------------------------------------------------------------------------------------
# status words
# ---------------------------------------------------------------------------------------------
def test_what_is_recorded_ends_no_attention_call():
    """A length that decode and weights cut, not asked for yet: the attention calls that follow are as ever."""
    lens, page = [300, 77], 16
    cache, table, _ = cases._paged("bf16", lens, page, 96, poison=False)
    small, small_table, _ = cases._paged("fp4", lens, page, 96, poison=False)
    q = cases._query(2, 2, 128, 96).to(dev())
    L, bad = cases._i32(lens), cases._i32([1 << 20, 77])
    x, kv = torch.randn((1000, 16, 576), device=dev()).bfloat16(), torch.randn((1000, 576), device=dev()).bfloat16()

    def attention():
        return (*mla_decode_ex(q, cache, table, L, 0.07), *mla_prefill(x, kv, 0.07))

    want = attention()
    cases._done()
    w = torch.zeros((2, 320), device=dev())
    mla_decode_fp4(q, small, 1.0, small_table, bad, 0.07)
    mla_key_weights(q, torch.zeros((2, 2, 128), device=dev()), cache, table, bad, 0.07, w)
    for _ in range(3):
        for a, b in zip(attention(), want):
            assert torch.equal(a, b)
    assert "0x7b" in cases._faults()
    cases._done()
