"""The smaller cache's operators (mla_kv_append_fp4, mla_decode_fp4, mla_key_weights, mla_select_keys, mla_compact_rows) against
the fp64 oracle, at the sizes, masks and strides where they can go wrong, and together as a server uses them.

Tolerances count roundings.  A score is a sum of 576 exact products, sixteen at a time on the tensor cores: 36 additions, each off by
at most 2^-23 of the sum of sizes, so SCORE = 2^-17 of that sum; q in f16 adds 2^-25 a column.  A weight of the softmax is off by that
much, by 2^-20 of itself (exponential, its argument) and, on the way to its product with V, by 2^-11 of itself and
2^-25 of the largest (f16).  An output in bf16 is off by 2^-8 of itself."""
import numpy as np
import pytest
import torch

import oracle.cache_oracle as co
from mla_attention_gb300 import (MLAError, check_device_status, mla_compact_rows, mla_decode_ex, mla_decode_fp4, mla_decode_fp8,
                                 mla_key_weights, mla_kv_append, mla_kv_append_fp4, mla_prefill, mla_select_keys, mla_slot_map)
from tests.helpers import assert_lse_close, assert_out_close, dev, to_np

pytestmark = pytest.mark.gpu

BF16, SCORE, EXP, F16 = 2.0 ** -8, 2.0 ** -17, 2.0 ** -20, 2.0 ** -11


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=dev())


def _within(gpu, ref, bound, what):
    g, r = to_np(gpu), np.asarray(ref, np.float64)
    assert g.shape == r.shape, (what, g.shape, r.shape)
    fine = np.isfinite(r)
    assert (np.isnan(g) == np.isnan(r)).all() and (g[~fine & ~np.isnan(r)] == r[~fine & ~np.isnan(r)]).all(), f"{what}: special values"
    err = np.abs(np.where(fine, g, 0) - np.where(fine, r, 0))
    worst = float((err - np.where(fine, bound, 0)).max()) if err.size else 0.0
    assert worst <= 0, f"{what}: worst excess {worst:.3e}, largest error {float(err.max()):.3e}"


def _done():
    torch.cuda.synchronize()
    check_device_status()


def _faults(status=5):
    torch.cuda.synchronize()
    with pytest.raises(MLAError) as e:
        check_device_status()
    assert e.value.status == status
    return str(e.value)


# ---------------------------------------------------------------------------------------------
# paged caches
# ---------------------------------------------------------------------------------------------
FORMATS = ["bf16", "e4m3", "fp4"]


def _values_to_cache(fmt, rows, g):
    """[n, 576] random rows of a format as stored."""
    n = rows.shape[0]
    if fmt == "bf16":
        return rows.bfloat16()
    if fmt == "e4m3":
        return (rows * 8).to(torch.float8_e4m3fn)
    code, scale = co.quantise_fp4(rows[:, :512].double().numpy(), 1.0)
    bits = rows[:, 512:].bfloat16().view(torch.int16).numpy().astype(np.int64) & 0xFFFF
    return torch.from_numpy(co.fp4_rows(code, scale, bits)).reshape(n, 416)


def _read(fmt, stored):
    """What stored rows stand for, fp64 numpy, without the cache's scale."""
    if fmt == "fp4":
        return co.fp4_values(stored.cpu().numpy())
    return stored.cpu().float().double().numpy()


def _paged(fmt, lens, page, seed, spare=2, poison=True, scale=1.0, row_scale=1.0):
    """A paged cache with requests of these lengths: (cache, block table) on the GPU and each request's keys.  Unused rows
    hold NaN (every byte 0xFF), entries of the table behind a request's pages an invalid page."""
    g = torch.Generator().manual_seed(seed)
    held = [-(-n // page) for n in lens]
    pages = sum(held) + spare
    ids = torch.randperm(pages, generator=g).tolist()
    width = max(held + [1]) + 1
    table = torch.full((len(lens), width), -7, dtype=torch.int32)
    row = {"bf16": 576, "e4m3": 576, "fp4": 416}[fmt]
    dtype = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "fp4": torch.uint8}[fmt]
    raw = torch.full((pages, page, row * dtype.itemsize), 0xFF if poison else 0, dtype=torch.uint8)
    cache = raw.view(dtype)
    keys = []
    for b, n in enumerate(lens):
        mine = [ids.pop() for _ in range(held[b])]
        table[b, :held[b]] = torch.tensor(mine, dtype=torch.int32)
        stored = _values_to_cache(fmt, torch.randn((n, 576), generator=g) * row_scale, g).contiguous()
        sv = stored.view(torch.uint8).reshape(n, row * dtype.itemsize)
        for k, pg in enumerate(mine):
            part = sv[k * page:(k + 1) * page]
            raw[pg, :len(part)] = part
        keys.append(_read(fmt, stored).reshape(n, 576) * scale)
    return cache.to(dev()), table.to(dev()), keys


def _query(B, s, H, seed, size=1.0):
    g = torch.Generator().manual_seed(seed + 1000)
    return (torch.randn((B, s, H, 576), generator=g) * size).bfloat16()


def _decode_bounds(q, keys, scale, sinks, out, lse):
    B, s, H, _ = q.shape
    bo, bl = np.zeros(out.shape), np.zeros(lse.shape)
    for b in range(B):
        for i in range(s):
            k = keys[b][:max(0, len(keys[b]) - s + 1 + i)]
            if len(k) == 0:
                continue
            for h in range(H):
                size = abs(scale) * (np.abs(k) @ np.abs(q[b, i, h])).max()
                ds = SCORE * size + abs(scale) * 2.0 ** -25 * np.abs(k).sum(1).max()
                if sinks is not None and np.isfinite(sinks[h]):
                    ds += 2.0 ** -22 * abs(sinks[h])
                w = np.exp(scale * (k @ q[b, i, h]) - lse[b, i, h])
                v = np.abs(k[:, :512])
                bo[b, i, h] = BF16 * np.abs(out[b, i, h]) + (2 * ds + F16 + EXP) * (w @ v) + 2.0 ** -25 * v.sum(0) * w.max() + 1e-30
                bl[b, i, h] = 2 * ds + EXP + 2.0 ** -21 * abs(lse[b, i, h]) if np.isfinite(lse[b, i, h]) else 0
    return bo, bl


def _check_decode(lens, H, s=1, page=64, seed=1, scale=192 ** -0.5, kv_scale=1.0, sinks=None, splits=0, q_size=1.0, row_scale=1.0, **kw):
    cache, table, keys = _paged("fp4", lens, page, seed, scale=kv_scale, row_scale=row_scale)
    q = _query(len(lens), s, H, seed, q_size)
    sk = None if sinks is None else np.asarray(sinks, np.float32)
    qn = to_np(q)
    ro, rl = co.decode(qn, keys, scale, sk)
    out, lse = mla_decode_fp4(q.to(dev()), cache, kv_scale, table, _i32(lens), scale,
                              sinks=None if sk is None else torch.tensor(sk).to(dev()), num_splits=splits, **kw)
    _done()
    bo, bl = _decode_bounds(qn, keys, scale, sk, ro, rl)
    _within(lse, rl, bl, "lse")
    _within(out, ro, bo, "out")
    return out, lse


# ---------------------------------------------------------------------------------------------
# decode
# ---------------------------------------------------------------------------------------------
EDGES = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 300]


@pytest.mark.parametrize("H", [1, 3, 16, 64, 65, 128])
def test_decode_lengths(H):
    _check_decode(EDGES, H, seed=H)


@pytest.mark.parametrize("page", [1, 7, 16, 32, 48, 128, 192, 1000])
def test_decode_page_sizes(page):
    _check_decode([0, 1, 130, 257, 31], 16, page=page, seed=page)


@pytest.mark.parametrize("s,H", [(2, 16), (3, 5), (4, 128), (7, 40), (16, 8), (130, 1), (2, 127), (5, 64)])
def test_decode_several_tokens(s, H):
    """Causal among a request's tokens; the first ones of a short request see no key."""
    _check_decode([0, 1, 3, s, 64, 129, 200], H, s=s, seed=s * 200 + H)


@pytest.mark.parametrize("splits", [1, 2, 5, 76, 300])
def test_decode_splits(splits):
    _check_decode([700, 1, 0, 129, 1025], 16, splits=splits, seed=7)


def test_decode_sinks():
    sinks = [0.0, 3.0, -np.inf, 12.0, -40.0, 1.5, 2.5, 90.0]
    _check_decode([0, 1, 200, 77], 8, s=2, sinks=sinks, seed=8)


@pytest.mark.parametrize("scale,kv_scale", [(0.0, 1.0), (-0.05, 1.0), (0.07, 0.375), (0.0002, 300.0), (1e4, 2.0 ** -20)])
def test_decode_scales(scale, kv_scale):
    _check_decode([200, 65, 1], 16, scale=scale, kv_scale=kv_scale, seed=9)


@pytest.mark.parametrize("sign", [1, -1])
def test_decode_scores_that_climb(sign):
    """Scores that grow by 12 a tile, so that the running maximum moves all along; through a RoPE column, so V stays of order one."""
    lens, page, H = [1500, 700], 64, 20
    cache, table, keys = _paged("fp4", lens, page, 10)
    raw = cache.cpu()
    for b, n in enumerate(lens):
        ramp = (torch.arange(n) * (12.0 / 64)).bfloat16()
        bits = ramp.view(torch.uint8).reshape(n, 2)
        for j in range(n):
            raw[table[b][j // page].item(), j % page, 288:290] = bits[j]
        keys[b][:, 512] = ramp.double().numpy()
    q = _query(2, 1, H, 10)
    q[..., 512] = sign * 13.875
    qn = to_np(q)
    scale = 192 ** -0.5
    ro, rl = co.decode(qn, keys, scale)
    out, lse = mla_decode_fp4(q.to(dev()), raw.to(dev()), 1.0, table, _i32(lens), scale)
    _done()
    bo, bl = _decode_bounds(qn, keys, scale, None, ro, rl)
    _within(lse, rl, bl, "lse")
    _within(out, ro, bo, "out")


def test_decode_long_request_and_many_short_ones():
    _check_decode([9000] + [5] * 30, 2, page=128, seed=11)


def test_decode_more_requests_than_splits():
    _check_decode([3, 70, 1] * 120, 4, page=16, seed=12)


def test_decode_one_hot_rows_are_the_rows_of_the_table():
    """q = 0 makes all scores equal: out * n is the sum of the rows, exact in f16 products of ones."""
    lens, page = [130, 64], 16
    cache, table, _ = _paged("fp4", lens, page, 13)
    raw = cache.cpu()
    for b, n in enumerate(lens):
        for j in range(n):
            r = raw[table[b][j // page].item(), j % page]
            r[:] = 0
            c = (j * 3) % 512
            r[c // 2] = 2 << (4 * (c % 2))               # 1.0
            r[256 + c // 16] = 0x38                      # scale 1.0
    q = torch.zeros((2, 1, 4, 576), dtype=torch.bfloat16)
    out, lse = mla_decode_fp4(q.to(dev()), raw.to(dev()), 1.0, table, _i32(lens), 1.0)
    _done()
    for b, n in enumerate(lens):
        hist = np.bincount((np.arange(n) * 3) % 512, minlength=512)
        got = to_np(out[b, 0])
        assert (np.rint(got * n) == hist).all() and (np.abs(got * n - hist) <= hist * 2.0 ** -7).all()
        np.testing.assert_allclose(to_np(lse[b]), np.log(n), rtol=1e-6)


def test_decode_single_token_shapes_and_given_outputs():
    cache, table, keys = _paged("fp4", [100, 33], 32, 14)
    q = _query(2, 1, 16, 14).to(dev())
    four, lse4 = mla_decode_fp4(q, cache, 1.0, table, _i32([100, 33]), 0.07)
    three, lse3 = mla_decode_fp4(q[:, 0], cache, 1.0, table, _i32([100, 33]), 0.07)
    out, lse = torch.empty_like(three), torch.empty_like(lse3)
    got = mla_decode_fp4(q[:, 0], cache, 1.0, table, _i32([100, 33]), 0.07, out=out, lse=lse)
    _done()
    assert three.shape == (2, 16, 512) and lse3.shape == (2, 16) and got[0] is out and got[1] is lse
    assert torch.equal(four[:, 0], three) and torch.equal(lse4[:, 0], lse3) and torch.equal(out, three) and torch.equal(lse, lse3)


def test_decode_repeats_bit_for_bit():
    cache, table, _ = _paged("fp4", [3000, 17, 900], 64, 15)
    q = _query(3, 2, 64, 15).to(dev())
    first = mla_decode_fp4(q, cache, 1.0, table, _i32([3000, 17, 900]), 0.07)
    for _ in range(3):
        again = mla_decode_fp4(q, cache, 1.0, table, _i32([3000, 17, 900]), 0.07)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    _done()


def test_decode_nan_and_infinite_keys_stay_in_their_request():
    lens, page = [70, 70, 70], 16
    cache, table, keys = _paged("fp4", lens, page, 16)
    raw = cache.cpu()
    raw[table[1][2].item(), 3, 256] = 0x7F               # a NaN scale in key 35 of request 1
    q = _query(3, 2, 8, 16)
    out, lse = mla_decode_fp4(q.to(dev()), raw.to(dev()), 1.0, table, _i32(lens), 0.07)
    _done()
    ro, rl = co.decode(to_np(q), keys, 0.07)
    bo, bl = _decode_bounds(to_np(q), keys, 0.07, None, ro, rl)
    for b in (0, 2):
        _within(out[b], ro[b], bo[b], "out")
        _within(lse[b], rl[b], bl[b], "lse")
    assert torch.isnan(lse[1]).all() and torch.isnan(out[1]).all()


def test_decode_bad_pages_and_lengths_are_recorded():
    cache, table, keys = _paged("fp4", [40, 40], 16, 17)
    q = _query(2, 1, 8, 17)
    bad = table.clone()
    bad[1, 1] = cache.shape[0]
    out, lse = mla_decode_fp4(q.to(dev()), cache, 1.0, bad, _i32([40, 40]), 0.07)
    assert "0x7a" in _faults()
    keys[1][16:32] = 0
    ro, rl = co.decode(to_np(q), keys, 0.07)
    bo, bl = _decode_bounds(to_np(q), keys, 0.07, None, ro, rl)
    _within(out, ro, bo, "out")
    _within(lse, rl, bl, "lse")
    full = torch.stack([table[0, :2], table[1, :2]]).contiguous()
    out, lse = mla_decode_fp4(q.to(dev()), cache, 1.0, full, _i32([33, -1]), 0.07)
    assert "0x7b" in _faults()
    ro, rl = co.decode(to_np(q), [keys[0][:32], keys[0][:0]], 0.07)
    bo, bl = _decode_bounds(to_np(q), [keys[0][:32], keys[0][:0]], 0.07, None, ro, rl)
    _within(out, ro, bo, "out")
    _within(lse, rl, bl, "lse")
    out, lse = mla_decode_fp4(q.to(dev()), cache, 1.0, table, _i32([40, 0]), 0.07)    # and the next call is as ever
    _done()


def _far_rows(row_bytes, above):
    """Rows so that their bytes pass `above`, in a fresh allocation (None where the card is too full)."""
    rows = above // row_bytes + 4096
    if torch.cuda.mem_get_info()[0] < 2 * rows * row_bytes:
        pytest.skip("not enough memory")
    return rows


@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_behind_two_to_the_32_bytes(fmt):
    """Pages at the far end of a cache of more than 2^32 bytes: decode (4-bit), weights and moves read and write there."""
    lens, page, H = [200, 77], 64, 8
    cache, table, keys = _paged(fmt, lens, page, 18)
    row = cache.shape[2] * cache.element_size()
    pages = _far_rows(row, 1 << 32) // page
    big = torch.full((pages, page, row), 0xFF, dtype=torch.uint8, device=dev())
    n = cache.shape[0]
    big[pages - n:] = cache.view(torch.uint8)
    far = table + (pages - n)
    big = big.view(cache.dtype)
    q = _query(2, 1, H, 18)
    ro, rl = co.decode(to_np(q), keys, 0.07)
    if fmt == "fp4":
        out, lse = mla_decode_fp4(q.to(dev()), big, 1.0, far, _i32(lens), 0.07)
        _done()
        bo, bl = _decode_bounds(to_np(q), keys, 0.07, None, ro, rl)
        _within(out, ro, bo, "out")
        _within(lse, rl, bl, "lse")
    w = torch.zeros((2, 256), device=dev())
    mla_key_weights(q.to(dev()), torch.tensor(rl, dtype=torch.float32).to(dev()), big, far, _i32(lens), 0.07, w, decay=0.0)
    _done()
    _within(w, co.key_weights(to_np(q), rl, keys, 0.07, np.zeros((2, 256)), 0.0), _weight_bounds(to_np(q), rl, keys, 0.07, to_np(w)), "weights")
    idx, count, _ = mla_select_keys(w, _i32(lens), _i32([50, 50]), 50, first=1, recent=8)
    before = big[pages - n:].clone()
    mla_compact_rows(big, far, idx, count)
    _done()
    ref, _ = co.compact_rows(before.view(torch.uint8).cpu().numpy(), table.cpu().numpy(), idx.cpu().numpy(), count.cpu().numpy())
    np.testing.assert_array_equal(big[pages - n:].view(torch.uint8).cpu().numpy(), ref)


# ---------------------------------------------------------------------------------------------
# the keys' weights
# ---------------------------------------------------------------------------------------------
def _weight_bounds(q, lse, keys, scale, w):
    bound = np.abs(w) * 2.0 ** -17 + 1e-30
    B, s, H, _ = q.shape
    for b in range(B):
        for i in range(s):
            k = keys[b][:max(0, len(keys[b]) - s + 1 + i)]
            for h in range(H):
                if len(k) and np.isfinite(lse[b, i, h]):
                    ds = abs(scale) * (SCORE * (np.abs(k) @ np.abs(q[b, i, h])) + 2.0 ** -25 * np.abs(k).sum(1))
                    p = np.exp(scale * (k @ q[b, i, h]) - lse[b, i, h])
                    bound[b, :len(k)] += p * (2 * ds + EXP + 2.0 ** -21 * abs(lse[b, i, h])) + 2.0 ** -120
    return bound


def _check_weights(fmt, lens, H, s=1, page=64, seed=1, scale=192 ** -0.5, decay=1.0, width_more=3, sinks=None, kv_scale=None):
    kv_scale = {"bf16": 1.0, "e4m3": 0.125, "fp4": 1.0}[fmt] if kv_scale is None else kv_scale
    cache, table, keys = _paged(fmt, lens, page, seed, scale=kv_scale)
    q = _query(len(lens), s, H, seed)
    qn = to_np(q)
    _, rl = co.decode(qn, keys, scale, sinks)
    rl = rl.astype(np.float32).astype(np.float64)
    g = torch.Generator().manual_seed(seed + 5)
    width = max(lens) + width_more
    old = torch.rand((len(lens), width + 5), generator=g)
    w = old.to(dev())[:, :width]
    got = mla_key_weights(q.to(dev()), torch.tensor(rl, dtype=torch.float32).to(dev()), cache, table, _i32(lens), scale, w, kv_scale=kv_scale,
                          decay=decay)
    _done()
    assert got is w
    ref = co.key_weights(qn, rl, keys, scale, to_np(old)[:, :width], decay)
    _within(w, ref, _weight_bounds(qn, rl, keys, scale, ref), "weights")
    for b, n in enumerate(lens):                       # the others are left as they were
        assert torch.equal(w[b, n:].cpu(), old[b, n:width])
    return w


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("H", [1, 16, 65, 128])
def test_weights_lengths(fmt, H):
    _check_weights(fmt, EDGES, H, seed=20 + H)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("page", [1, 7, 16, 32, 128, 192])
def test_weights_page_sizes(fmt, page):
    _check_weights(fmt, [0, 1, 130, 257, 31], 5, page=page, seed=40 + page, decay=0.5)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("s,H", [(2, 16), (4, 128), (3, 5), (32, 40), (130, 1), (9, 128)])
def test_weights_several_tokens(fmt, s, H):
    _check_weights(fmt, [0, 1, 3, s, 64, 129, 200], H, s=s, seed=60 + s)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("scale,decay", [(0.0, 1.0), (-0.05, 0.0), (0.07, 0.25)])
def test_weights_scales(fmt, scale, decay):
    _check_weights(fmt, [200, 65, 1], 16, scale=scale, decay=decay, seed=80)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("lens,s", [([60000], 1), ([30000, 5, 21000], 2), ([20500], 200)])
def test_weights_long(fmt, lens, s):
    """Several tiles for each CTA, with one chunk of query rows and with more."""
    _check_weights(fmt, lens, 1, s=s, seed=70)


def test_weights_with_sinks_and_many_requests():
    _check_weights("bf16", [3, 70, 1, 0] * 60, 4, page=16, seed=81, sinks=np.array([0.0, 2.0, -np.inf, 8.0]))


def test_weights_without_decay_do_not_read_the_old_ones():
    cache, table, keys = _paged("bf16", [70], 64, 82)
    q = _query(1, 1, 4, 82).to(dev())
    _, rl = co.decode(to_np(q), keys, 0.07)
    lse = torch.tensor(rl, dtype=torch.float32).to(dev())
    w = torch.full((1, 80), float("nan"), device=dev())
    mla_key_weights(q, lse, cache, table, _i32([70]), 0.07, w, decay=0.0)
    _done()
    assert torch.isfinite(w[0, :70]).all() and torch.isnan(w[0, 70:]).all()
    np.testing.assert_allclose(float(w[0, :70].sum()), 4, rtol=1e-4)


def test_weights_special_lse():
    """-inf and +inf add nothing, a NaN shows."""
    cache, table, keys = _paged("bf16", [70], 64, 83)
    q = _query(1, 1, 3, 83).to(dev())
    _, rl = co.decode(to_np(q), keys, 0.07)
    lse = torch.tensor(rl, dtype=torch.float32).to(dev())
    lse[0, 0, 0], lse[0, 0, 1] = float("-inf"), float("inf")
    w = torch.zeros((1, 70), device=dev())
    mla_key_weights(q, lse, cache, table, _i32([70]), 0.07, w)
    _done()
    np.testing.assert_allclose(float(w.sum()), 1, rtol=1e-4)
    lse[0, 0, 2] = float("nan")
    mla_key_weights(q, lse, cache, table, _i32([70]), 0.07, w)
    _done()
    assert torch.isnan(w).all()


def test_weights_bad_pages_and_lengths_are_recorded():
    cache, table, keys = _paged("bf16", [40, 40], 16, 84)
    q = _query(2, 1, 8, 84).to(dev())
    lse = torch.zeros((2, 1, 8), device=dev())
    bad = table.clone()
    bad[1, 1] = -1
    w = torch.zeros((2, 48), device=dev())
    mla_key_weights(q, lse, cache, bad, _i32([40, 40]), 0.07, w)
    assert "0x7a" in _faults()
    np.testing.assert_allclose(to_np(w[1, 16:32]), 8, rtol=1e-5)      # keys of zeros: a score of 0 in each of 8 heads
    w = torch.zeros((2, 30), device=dev())
    mla_key_weights(q, lse, cache, table, _i32([40, 20]), 0.07, w)
    assert "0x7b" in _faults()
    assert (w[0] > 0).all() and (w[1, :20] > 0).all() and (w[1, 20:] == 0).all()


# ---------------------------------------------------------------------------------------------
# the rows that stay
# ---------------------------------------------------------------------------------------------
def _check_select(w, lens, keep, K, first, recent, pad=0):
    B, W = w.shape
    wide = torch.full((B, W + pad), 9e9)
    wide[:, :W] = w
    ref = co.select_keys(w.double().numpy(), lens, keep, K, first, recent)
    d = wide.to(dev())[:, :W]
    for _ in range(2):
        got = mla_select_keys(d, _i32(lens), _i32(keep), K, first=first, recent=recent)
        if ref[3]:
            assert "0x7c" in _faults()
        else:
            _done()
        for name, a, b in zip(("idx", "count", "dropped"), got, ref):
            np.testing.assert_array_equal(to_np(a), b, err_msg=name)


@pytest.mark.parametrize("kind", ["normal", "heavy", "equal", "few", "zeros", "special", "signs"])
@pytest.mark.parametrize("first,recent", [(0, 0), (4, 32), (0, 1), (1000, 5), (3, 5000)])
def test_select_kinds(kind, first, recent):
    g = torch.Generator().manual_seed(len(kind) + first)
    W = 1203
    w = torch.rand((9, W), generator=g)
    if kind == "heavy":
        w = torch.exp(6 * torch.randn((9, W), generator=g))
    elif kind == "equal":
        w[:] = 0.25
    elif kind == "few":
        w = torch.randint(0, 3, (9, W), generator=g).float()
    elif kind == "zeros":
        w[w < 0.9] = 0
        w[w < 0.92] = -0.0
    elif kind == "special":
        w[w < 0.1], w[w > 0.9] = float("nan"), float("inf")
        w[(w > 0.4) & (w < 0.5)] = -float("inf")
        w[(w > 0.5) & (w < 0.6)] = 1e-45
    elif kind == "signs":
        w -= 0.5
    _check_select(w, [0, 1, 31, 32, 33, 1024, 1025, 1203, 700], [5, 1, 30, 40, 32, 512, 1, 1202, 0], 1210, first, recent)


@pytest.mark.parametrize("lens", [[1], [2], [4096], [40000], [150001], [70000, 3, 129, 33000]])
@pytest.mark.parametrize("share", [0.01, 0.5, 0.99])
def test_select_lengths(lens, share):
    g = torch.Generator().manual_seed(sum(lens))
    w = torch.exp(2 * torch.randn((len(lens), max(lens)), generator=g))
    keep = [max(1, int(n * share)) for n in lens]
    _check_select(w, lens, keep, max(keep), 2, 7, pad=3)


def test_select_many_requests():
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 200, (1500,), generator=g).tolist()
    keep = torch.randint(0, 150, (1500,), generator=g).tolist()
    _check_select(torch.rand((1500, 200), generator=g), lens, keep, 150, 1, 4)


def test_select_refuses_bad_requests_alone():
    w = torch.rand((6, 50), generator=torch.Generator().manual_seed(4))
    _check_select(w, [50, 51, -1, 20, 40, 30], [9, 9, 9, -1, 12, 30], 11, 1, 2)


def test_select_empty():
    idx, count, dropped = mla_select_keys(torch.zeros((0, 8), device=dev()), _i32([]), _i32([]), 4)
    assert idx.shape == (0, 4) and count.shape == (0,)
    idx, count, dropped = mla_select_keys(torch.zeros((2, 8), device=dev()), _i32([8, 0]), _i32([0, 5]), 0)
    _done()
    assert idx.shape == (2, 0) and count.tolist() == [0, 0] and dropped.tolist() == [-8, 0]


# ---------------------------------------------------------------------------------------------
# the moves
# ---------------------------------------------------------------------------------------------
def _check_compact(lens, row, page, keeps, seed, weights=True, dtype=torch.uint8):
    g = torch.Generator().manual_seed(seed)
    held = [-(-n // page) for n in lens]
    pages = sum(held) + 3
    ids = torch.randperm(pages, generator=g).tolist()
    table = torch.full((len(lens), max(held + [1])), -1, dtype=torch.int32)
    for b, n in enumerate(held):
        table[b, :n] = torch.tensor([ids.pop() for _ in range(n)], dtype=torch.int32)
    cache = torch.randint(0, 256, (pages, page, row), generator=g, dtype=torch.uint8)
    K = max(keeps) + 2
    idx = torch.full((len(lens), K), -1, dtype=torch.int32)
    for b, (n, k) in enumerate(zip(lens, keeps)):
        idx[b, :k] = torch.sort(torch.randperm(n, generator=g)[:k]).values.int()
    W = max(lens) + 1
    w = torch.rand((len(lens), W), generator=g) if weights else None
    ref, rw = co.compact_rows(cache.numpy(), table.numpy(), idx.numpy(), keeps, None if w is None else w.numpy())
    d = cache.to(dev()).view(dtype) if dtype is not torch.uint8 else cache.to(dev())
    dw = None if w is None else w.to(dev())
    mla_compact_rows(d, table.to(dev()), idx.to(dev()), _i32(keeps), weights=dw)
    _done()
    np.testing.assert_array_equal(d.view(torch.uint8).cpu().numpy(), ref)
    if w is not None:
        np.testing.assert_array_equal(dw.cpu().numpy(), rw)


@pytest.mark.parametrize("row,dtype", [(1152, torch.bfloat16), (576, torch.float8_e4m3fn), (416, torch.uint8), (16, torch.uint8), (48, torch.uint8),
                                       (4096, torch.float32)])
@pytest.mark.parametrize("page", [1, 7, 16, 64])
def test_compact(row, dtype, page):
    lens = [0, 1, 2, 130, 257, 300, 64, 999]
    _check_compact(lens, row, page, [0, 1, 1, 70, 257, 1, 32, 700], row + page, dtype=dtype)


@pytest.mark.parametrize("keep", [1, 2999, 3000, 1500, 127, 128, 129])
def test_compact_long(keep):
    _check_compact([3000, 20], 416, 64, [keep, 10], keep, weights=False)


def test_compact_of_many_requests():
    g = torch.Generator().manual_seed(5)
    lens = torch.randint(0, 90, (400,), generator=g).tolist()
    _check_compact(lens, 416, 16, [n // 2 for n in lens], 6)


def test_compact_skips_and_records_bad_entries():
    cache = torch.arange(8 * 4 * 16, dtype=torch.int32).reshape(8, 4, 16).to(torch.uint8)
    table = _i32([[0, 1, 2], [3, 4, 5]])
    idx = _i32([[0, 2, 1, 3, 9], [1, 12, 7, 8, 9]])
    for count, moved in (([5, 0], [(0, 1, 2), (0, 4, 9)]), ([0, 2], [(1, 0, 1)]), ([6, 0], []), ([-1, 0], [])):
        d = cache.to(dev())
        mla_compact_rows(d, table, idx, _i32(count))
        assert "0x7d" in _faults()
        ref = cache.clone()
        for b, i, j in moved:                    # entry 2 lies below its place and entry 1, 3 at its own
            ref[table[b][i // 4], i % 4] = cache[table[b][j // 4], j % 4]
        assert torch.equal(d.cpu(), ref), count
    bad = _i32([[0, 8, 2], [3, 4, 5]])
    d = cache.to(dev())
    mla_compact_rows(d, bad, _i32([[5, 6, 8], [0, 1, 2]]), _i32([3, 3]))
    assert "0x7d" in _faults()
    ref = cache.clone()
    ref[0, 2] = cache[2, 0]
    assert torch.equal(d.cpu(), ref)


# ---------------------------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------------------------
def _append_inputs(T, H, seed, size=1.0, max_pos=512):
    g = torch.Generator().manual_seed(seed)
    kv = (torch.randn((T, 576), generator=g) * size).bfloat16()
    w = (1 + 0.3 * torch.randn(512, generator=g)).bfloat16()
    ang = torch.arange(max_pos, dtype=torch.float64)[:, None] * 10000.0 ** (-2.0 * torch.arange(32, dtype=torch.float64) / 64)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float()
    pos = torch.randint(0, max_pos, (T,), generator=g, dtype=torch.int32)
    q = torch.randn((T, H, 64), generator=g).bfloat16() if H else None
    return kv, w, cs, pos, q, g


def _check_append(kv, w, cs, pos, q, g, kv_scale=1.0, eps=1e-6, neox=False, page=16, rows_out=True, holes=()):
    T, kv_scale = len(kv), float(np.float32(kv_scale))
    pages = -(-T // page) + 2
    slots = torch.randperm(pages * page, generator=g)[:T].int()
    pos, slots = pos.clone(), slots.clone()
    for t in holes:
        pos[t] = -1
    cache = torch.randint(0, 256, (pages, page, 416), generator=g, dtype=torch.uint8)
    live = [t for t in range(T) if pos[t] >= 0]
    code, scale, pe, rows, rq = co.kv_append_fp4(to_np(kv[live, :512]), to_np(kv[live, 512:]), pos[live].numpy(), cs.numpy(), kv_scale,
                                                 None if w is None else to_np(w), eps, None if q is None else to_np(q[live]), neox)
    d = cache.to(dev())
    x = kv.to(dev())
    kv_out = torch.full((T, 576), 7.0, dtype=torch.bfloat16, device=dev()) if rows_out else None
    got_q, got_rows = mla_kv_append_fp4(x[:, :512], x[:, 512:], slots.to(dev()), pos.to(dev()), cs.to(dev()), d, kv_scale,
                                        norm_weight=None if w is None else w.to(dev()), eps=eps, q_pe=None if q is None else q.to(dev()),
                                        kv_out=kv_out, is_neox=neox)
    _done()
    new = d.cpu().reshape(-1, 416).numpy()
    at = slots[live].long().numpy()
    want = co.fp4_rows(code, scale, np.zeros((len(live), 64), np.int64))
    np.testing.assert_array_equal(new[at, 256:288], want[:, 256:288], err_msg="scales")
    nan = np.repeat(np.isnan(scale), 16, 1)[:, 0::2]
    for shift in (0, 4):                        # the codes of 0 and -0 stand for the same value
        a, b = (new[at, :256] >> shift) & 15, (want[:, :256] >> shift) & 15
        np.testing.assert_array_equal(np.where(nan | (a == 8), 0, a), np.where(nan | (b == 8), 0, b), err_msg="codes")
    got_pe = torch.from_numpy(np.ascontiguousarray(new[at, 288:])).view(torch.bfloat16)
    turned = (np.abs(to_np(kv[live, 512:])) + 1e-30).max(1, keepdims=True) / kv_scale
    _within(got_pe, pe, BF16 * np.abs(pe) + 2.0 ** -21 * turned + 2.0 ** -134, "pe")
    others = np.setdiff1d(np.arange(pages * page), at)
    np.testing.assert_array_equal(new[others], cache.reshape(-1, 416).numpy()[others])
    if q is not None:
        _within(got_q[live, :, 512:], rq, BF16 * np.abs(rq) + 2.0 ** -21 * np.abs(to_np(q[live])).max(), "q")
    if rows_out:
        lat_size = np.abs(rows)
        lat_size[:, 512:] += turned * kv_scale
        _within(got_rows[live], rows, BF16 * np.abs(rows) + 2.0 ** -18 * lat_size + 2.0 ** -134, "rows")
        for t in holes:
            assert (got_rows[t] == 7).all()


@pytest.mark.parametrize("T,H", [(1, 1), (2, 128), (3, 17), (64, 16), (257, 0), (33, 5)])
@pytest.mark.parametrize("neox", [False, True])
def test_append(T, H, neox):
    _check_append(*_append_inputs(T, H, T + H), neox=neox, holes=(0,) if T > 2 else ())


@pytest.mark.parametrize("kv_scale", [1.0, 0.75, 0.02, 2.0 ** -100, 2.0 ** 100, 3e-5])
@pytest.mark.parametrize("norm", [True, False])
def test_append_scales(kv_scale, norm):
    kv, w, cs, pos, q, g = _append_inputs(120, 2, 5)
    _check_append(kv, w if norm else None, cs, pos, q, g, kv_scale=kv_scale)


@pytest.mark.parametrize("norm", [True, False])
def test_append_ties_and_borders(norm):
    """Values that are quotients of few bits: most lie on a border between two codes or two scales, or next to it."""
    kv, w, cs, pos, q, g = _append_inputs(400, 0, 6)
    kv[:, :512] = (torch.randint(-96, 97, (400, 512), generator=g) / 16.0).bfloat16()
    kv[::3, :512] = (torch.randint(-12, 13, (134, 512), generator=g) / 2.0).bfloat16()
    w[:] = 1.0
    if norm:                                   # a row of mean square one keeps its values (eps = 0)
        kv[::2, :512] = torch.where(torch.rand((200, 512), generator=g) < 0.5, 1.0, -1.0).bfloat16()
        w = (torch.randint(1, 97, (512,), generator=g) / 16.0).bfloat16()
    _check_append(kv, w if norm else None, cs, pos, q, g, eps=0.0)
    _check_append(kv, w if norm else None, cs, pos, q, g, eps=0.0, kv_scale=0.375)


def test_append_many_random_rows_have_the_exact_codes():
    kv, w, cs, pos, q, g = _append_inputs(6000, 0, 7)
    _check_append(kv, w, cs, pos, q, g, rows_out=False)


@pytest.mark.parametrize("size", [2.0 ** -130, 2.0 ** -60, 2.0 ** 60, 2.0 ** 120])
def test_append_rows_far_from_one(size):
    kv, w, cs, pos, q, g = _append_inputs(40, 0, 8)
    kv[:, :512] = (kv[:, :512].double() * size).bfloat16()
    _check_append(kv, w, cs, pos, q, g, eps=0.0)


def test_append_special_values():
    kv, _, cs, pos, q, g = _append_inputs(12, 0, 9)
    kv[0, 5], kv[1, 100], kv[2, :512], kv[3, 31] = float("nan"), float("inf"), 0.0, -float("inf")
    kv[4, 16:32] = 0.0
    kv[4, 20] = -0.0
    _check_append(kv, None, cs, pos, q, g, rows_out=False)


def test_append_in_place_rows_and_strided_views():
    kv, w, cs, pos, q, g = _append_inputs(65, 3, 10)
    wide = torch.zeros((65, 640), dtype=torch.bfloat16)
    wide[:, :576] = kv
    x = wide.to(dev())
    a, b = torch.zeros((5, 16, 416), dtype=torch.uint8, device=dev()), torch.zeros((5, 16, 416), dtype=torch.uint8, device=dev())
    slots = torch.randperm(80, generator=g)[:65].int().to(dev())
    rows = torch.empty((65, 576), dtype=torch.bfloat16, device=dev())
    common = (slots, pos.to(dev()), cs.to(dev()))
    mla_kv_append_fp4(x[:, :512], x[:, 512:576], *common, a, norm_weight=w.to(dev()), kv_out=rows)
    mla_kv_append_fp4(x[:, :512], x[:, 512:576], *common, b, norm_weight=w.to(dev()), kv_out=x[:, :576])
    _done()
    assert torch.equal(a, b) and torch.equal(rows, x[:, :576])


def test_append_in_place_no_norm_rows_with_ties():
    """A row that has to be decided again is decided from what was read, not from what was written in its place."""
    kv, _, cs, pos, _, g = _append_inputs(64, 0, 11)
    kv[:, :512] = (torch.randint(-96, 97, (64, 512), generator=g) / 16.0).bfloat16()
    w = (torch.randint(1, 33, (512,), generator=g) / 16.0).bfloat16().to(dev())
    a, b = torch.zeros((5, 16, 416), dtype=torch.uint8, device=dev()), torch.zeros((5, 16, 416), dtype=torch.uint8, device=dev())
    slots = torch.arange(64, dtype=torch.int32, device=dev())
    x = kv.to(dev())
    mla_kv_append_fp4(x[:, :512], x[:, 512:], slots, pos.to(dev()), cs.to(dev()), a, norm_weight=w, eps=0.0)
    mla_kv_append_fp4(x[:, :512], x[:, 512:], slots, pos.to(dev()), cs.to(dev()), b, norm_weight=w, eps=0.0, kv_out=x)
    _done()
    assert torch.equal(a, b)


def test_append_bad_positions_and_slots_are_recorded():
    kv, w, cs, pos, q, g = _append_inputs(4, 0, 12)
    x, cache = kv.to(dev()), torch.zeros((1, 4, 416), dtype=torch.uint8, device=dev())
    mla_kv_append_fp4(x[:, :512], x[:, 512:], _i32([0, 1, 4, -1]), _i32([512, 3, 3, 3]), cs.to(dev()), cache)
    assert "0x7" in _faults()
    assert (cache[0, 0] == 0).all() and (cache[0, 1] != 0).any() and (cache[0, 2:] == 0).all()


def test_append_holds_the_bf16_append_to_four_bits():
    """The same rows as mla_kv_append's, through the same slots, in 4 bits."""
    kv, w, cs, pos, q, g = _append_inputs(100, 4, 13)
    x = kv.to(dev())
    slots = torch.randperm(112, generator=g)[:100].int().to(dev())
    c16 = torch.zeros((7, 16, 576), dtype=torch.bfloat16, device=dev())
    c4 = torch.zeros((7, 16, 416), dtype=torch.uint8, device=dev())
    args = dict(norm_weight=w.to(dev()), q_pe=q.to(dev()))
    q16, _ = mla_kv_append(x[:, :512], x[:, 512:], slots, pos.to(dev()), cs.to(dev()), c16, **args)
    q4, _ = mla_kv_append_fp4(x[:, :512], x[:, 512:], slots, pos.to(dev()), cs.to(dev()), c4, **args)
    _done()
    assert torch.equal(q16[..., 512:], q4[..., 512:])
    a, b = to_np(c16).reshape(-1, 576), co.fp4_values(c4.cpu().numpy()).reshape(-1, 576)
    np.testing.assert_array_equal(a[:, 512:], b[:, 512:])
    top = np.abs(a[:, :512]).reshape(len(a), -1, 16).max(2).repeat(16, 1)
    # half a step between 4 and 6, a scale off by 2^-4 of itself that may cut the largest, bf16
    assert (np.abs(a[:, :512] - b[:, :512]) <= top / 6 * (1 + 2.0 ** -4) * 1.0 + top * (2.0 ** -4 + BF16) + 6 * 2.0 ** -9).all()


# ---------------------------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------------------------
def _serve(steps=6, stream=None):
    """Requests that grow by a token a step over a 4-bit cache; after each step the keys' weights are added up and, every
    other step, requests over their budget lose rows and give pages back.  Returns all that the steps gave."""
    g = torch.Generator().manual_seed(21)
    d, page, H, B = dev(), 16, 8, 3
    max_pages, pages, K = 8, 22, 40
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device=d)
    pool, state = torch.arange(pages, dtype=torch.int32, device=d), _i32([0, pages])
    cache = torch.zeros((pages, page, 416), dtype=torch.uint8, device=d)
    weights = torch.zeros((B, max_pages * page), device=d)
    ang = torch.arange(256, dtype=torch.float64)[:, None] * 10000.0 ** (-2.0 * torch.arange(32, dtype=torch.float64) / 64)
    cs = torch.cat([ang.cos(), ang.sin()], 1).float().to(d)
    w = (1 + 0.2 * torch.randn(512, generator=g)).bfloat16().to(d)
    lens, gone = _i32([0] * B), _i32([0] * B)
    keep = _i32([40, 30, 35])
    got = []
    kw = dict(stream=stream)
    for step in range(steps):
        new = [50, 21, 44] if step == 0 else [1, 1, 1]
        T = sum(new)
        kv = torch.randn((T, 576), generator=g).bfloat16().to(d)
        q = torch.randn((B, H, 576), generator=g).bfloat16().to(d)
        q_pe = q[:, :, 512:].contiguous()
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        pos, slots, cu, lens, state = mla_slot_map(lens, _i32(new), table, pool, state, page, T, **kw)
        torch.cuda.synchronize()
        seen = pos + torch.repeat_interleave(gone, torch.tensor(new, device=d)).int()     # positions go on past what was dropped
        mla_kv_append_fp4(kv[:, :512], kv[:, 512:], slots, seen, cs, cache, norm_weight=w, **kw)
        out, lse = mla_decode_fp4(q, cache, 1.0, table, lens, 0.07, **kw)
        mla_key_weights(q, lse, cache, table, lens, 0.07, weights, decay=0.5, **kw)
        torch.cuda.synchronize()
        got += [out.clone(), lse.clone(), weights.clone()]
        if step % 2 == 0:
            idx, count, dropped = mla_select_keys(weights, lens, keep, K, first=2, recent=4, **kw)
            mla_compact_rows(cache, table, idx, count, weights=weights, **kw)
            torch.cuda.synchronize()
            gone = (gone - dropped).int()
            # the weights behind the kept rows start anew with the tokens that come there
            weights.masked_fill_(torch.arange(weights.shape[1], device=d)[None] >= count[:, None], 0)
            torch.cuda.synchronize()
            _, _, _, lens, state = mla_slot_map(lens, dropped, table, pool, state, page, 0, **kw)
            torch.cuda.synchronize()
            assert lens.tolist() == count.tolist()
            got += [idx.clone(), lens.clone(), state.clone()]
    check_device_status()
    return got, (cache, table, lens, weights, q, out, lse)


def test_served_steps_with_evictions():
    got, (cache, table, lens, weights, q, out, lse) = _serve(steps=6)
    # the last step against the oracle over what the cache then held
    n = [int(v) for v in lens]
    raw = cache.cpu().numpy()
    keys = [co.fp4_values(co.held_rows(raw, table.cpu().numpy(), n, b)) for b in range(3)]
    qn = to_np(q)[:, None]
    ro, rl = co.decode(qn, keys, 0.07)
    bo, bl = _decode_bounds(qn, keys, 0.07, None, ro, rl)
    _within(out[:, None], ro, bo, "out")
    _within(lse[:, None], rl, bl, "lse")
    other = _serve(steps=6, stream=torch.cuda.Stream())[0]
    assert len(got) == len(other)
    for a, b in zip(got, other):
        assert torch.equal(a, b)


def test_captured_steps_replay():
    """Decode, weights, selection and moves in one captured graph, replayed with new lengths and queries in the same places."""
    lens, page, H, K = [300, 77, 130], 16, 16, 64
    cache, table, keys = _paged("fp4", lens, page, 30, poison=False)
    d = dev()
    q = _query(3, 1, H, 30).to(d)
    L, keep = _i32(lens), _i32([64, 64, 50])
    w = torch.zeros((3, 320), device=d)
    first = cache.clone()

    def step():
        out, lse = mla_decode_fp4(q, cache, 1.0, table, L, 0.07)
        mla_key_weights(q, lse, cache, table, L, 0.07, w, decay=0.5)
        idx, count, dropped = mla_select_keys(w, L, keep, K, first=1, recent=8)
        mla_compact_rows(cache, table, idx, count, weights=w)
        return out, lse, idx, count, dropped

    step()
    torch.cuda.synchronize()
    cache.copy_(first)
    w.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for lengths, seed in (([300, 77, 130], 31), ([299, 1, 0], 32), ([16, 77, 64], 33)):
        new_q = _query(3, 1, H, seed).to(d)
        ref = []
        for run in range(2):
            cache.copy_(first)
            w.zero_()
            L.copy_(_i32(lengths))
            q.copy_(new_q)
            if run == 0:
                ref = [t.clone() for t in (*step(), cache, w)]
            else:
                graph.replay()
        _done()
        for a, b in zip(ref, (*held, cache, w)):
            assert torch.equal(a, b)


def test_kept_rows_of_every_format_decode_as_the_chosen_ones():
    """After a move, decode over the kept rows is attention over the chosen rows."""
    lens, page, H = [150, 90], 16, 8
    for fmt, kv_scale in (("bf16", 1.0), ("e4m3", 0.125), ("fp4", 1.0)):
        cache, table, keys = _paged(fmt, lens, page, 40, scale=kv_scale)
        table = torch.where(table < 0, 0, table)
        q = _query(2, 1, H, 40).to(dev())
        _, rl = co.decode(to_np(q), keys, 0.07)
        w = torch.zeros((2, 160), device=dev())
        mla_key_weights(q, torch.tensor(rl, dtype=torch.float32).to(dev()), cache, table, _i32(lens), 0.07, w, kv_scale=kv_scale)
        idx, count, dropped = mla_select_keys(w, _i32(lens), _i32([60, 64]), 64, first=2, recent=8)
        mla_compact_rows(cache, table, idx, count, weights=w)
        if fmt == "bf16":
            out, lse = mla_decode_ex(q, cache, table, count, 0.07)
        elif fmt == "e4m3":
            out, lse = mla_decode_fp8(q, cache, kv_scale, table, count, 0.07)
        else:
            out, lse = mla_decode_fp4(q, cache, kv_scale, table, count, 0.07)
        _done()
        chosen = [keys[b][idx[b, :int(count[b])].cpu().numpy()] for b in range(2)]
        ro, rl = co.decode(to_np(q), chosen, 0.07)
        assert_out_close(out, ro)
        assert_lse_close(lse, rl)


def test_weights_of_a_prompt_choose_what_the_prefill_attended_to():
    """The weights that a prompt's last tokens give, from the prefill's own log-sum-exp, add up to its query rows."""
    T, H, s = 200, 16, 8
    g = torch.Generator().manual_seed(50)
    q, kv = torch.randn((T, H, 576), generator=g).bfloat16().to(dev()), torch.randn((T, 576), generator=g).bfloat16().to(dev())
    out, lse = mla_prefill(q, kv, 0.07)
    cache = torch.zeros((4, 64, 576), dtype=torch.bfloat16, device=dev())
    cache.view(-1, 576)[:T] = kv
    w = torch.zeros((1, 256), device=dev())
    mla_key_weights(q[None, T - s:], lse.t()[None, T - s:].contiguous(), cache, _i32([[0, 1, 2, 3]]), _i32([T]), 0.07, w)
    _done()
    np.testing.assert_allclose(float(w.sum()), s * H, rtol=2e-4)


def test_two_streams_at_once():
    """The same calls on two streams with their own workspaces give what each gives alone."""
    lens, page, H = [900, 300], 64, 32
    cache, table, _ = _paged("fp4", lens, page, 60)
    L = _i32(lens)
    qs = [_query(2, 1, H, s).to(dev()) for s in (60, 61)]
    alone = [mla_decode_fp4(q, cache, 1.0, table, L, 0.07) for q in qs]
    from mla_attention_gb300 import lib
    size = lib().mla_decode_fp4_workspace_size(2, 1, H, 0)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    spaces = [torch.zeros(size, dtype=torch.uint8, device=dev()) for _ in qs]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i, (q, st, ws) in enumerate(zip(qs, streams, spaces)):
            got[i] = mla_decode_fp4(q, cache, 1.0, table, L, 0.07, ws=ws, stream=st)
    torch.cuda.synchronize()
    for (a, b), (c, e) in zip(alone, got):
        assert torch.equal(a, c) and torch.equal(b, e)
    for ws in spaces:
        check_device_status(ws)
