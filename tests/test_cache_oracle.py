"""Pins of the smaller cache's oracle: hand-worked cases, torch's conversions, identities (CPU only)."""
import numpy as np
import pytest
import torch

import oracle.cache_oracle as co
import oracle.mla_oracle as mo


def test_e2m1_by_hand():
    v = [0.0, 0.25, 0.2500001, 0.75, 0.74, 1.25, 1.75, 2.5, 2.51, 3.5, 5.0, 5.01, 7.0, np.inf, -0.1, -0.75, -5.0]
    assert co.round_e2m1(v).tolist() == [0, 0, 1, 2, 1, 2, 4, 4, 5, 6, 6, 7, 7, 7, 8, 10, 14]


def test_quantise_by_hand():
    lat = np.zeros((1, 512))
    lat[0, :16] = [12, 6, 3, 2, 1, 0.5, -0.5, -12] + [0] * 8           # scale 2
    lat[0, 16:18] = [2.0 ** -12, -2.0 ** -10]                          # below the smallest scale
    lat[0, 32] = 1e9                                                   # beyond the largest
    lat[0, 48] = np.nan
    code, scale = co.quantise_fp4(lat, 1.0)
    assert scale[0, :3].tolist() == [2.0, 2.0 ** -9, 448.0] and np.isnan(scale[0, 3]) and (scale[0, 4:] == 2.0 ** -9).all()
    assert code[0, :8].tolist() == [7, 5, 3, 2, 1, 0, 8, 15]           # 0.25 of the scale: a tie, to even
    assert code[0, 16:18].tolist() == [0, 9] and code[0, 32] == 7
    twice, scale2 = co.quantise_fp4(lat * 0.375, 0.375)
    np.testing.assert_array_equal(code[0, :48], twice[0, :48])
    np.testing.assert_array_equal(scale, scale2)


def test_rows_there_and_back():
    g = np.random.default_rng(1)
    lat = g.normal(size=(9, 512))
    code, scale = co.quantise_fp4(lat, 1.0)
    pe = torch.randn(9, 64).bfloat16()
    rows = co.fp4_rows(code, scale, pe.view(torch.int16).numpy().astype(np.int64) & 0xFFFF)
    got = co.fp4_values(rows)
    np.testing.assert_array_equal(got[:, 512:], pe.double().numpy())
    value = np.where(code >= 8, -1, 1) * co.E2M1[code & 7] * np.repeat(scale, 16, 1)
    np.testing.assert_array_equal(got[:, :512], value)
    # a value is at most half a step of 2 (of the largest codes) and the scale's own rounding away
    assert (np.abs(value - lat) <= np.repeat(scale, 16, 1) * (1 + 6 / 16)).all()
    np.testing.assert_array_equal(rows[:, 256:288], torch.tensor(scale).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_every_scale_byte_matches_torch():
    rows = np.zeros((256, 416), np.uint8)
    rows[:, 256] = np.arange(256)
    rows[:, 0] = 0x92                                                  # codes 1.0 and -0.5
    ref = torch.arange(256, dtype=torch.int16).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    got = co.fp4_values(rows)
    np.testing.assert_array_equal(got[:, 0], ref)
    np.testing.assert_array_equal(got[:, 1], -0.5 * ref)


def test_decode_is_the_attention_of_the_held_rows():
    g = np.random.default_rng(2)
    cache = g.integers(0, 120, size=(5, 4, 416)).astype(np.uint8)
    cache[..., 288:] = np.ascontiguousarray(torch.randn(5, 4, 64).bfloat16().view(torch.uint8).numpy())
    table, lens = np.array([[3, 0, 4], [1, 2, -1]]), [9, 6]
    keys = [co.fp4_values(co.held_rows(cache, table, lens, b)) for b in range(2)]
    assert keys[0].shape == (9, 576)
    q = g.normal(size=(2, 1, 3, 576))
    out, lse = co.decode(q, keys, 0.05)
    bf = torch.zeros(5, 4, 576, dtype=torch.float64)
    bf[:] = torch.tensor(co.fp4_values(cache))
    ro, rl = mo.mla_decode(torch.tensor(q[:, 0]), bf, torch.tensor(table), torch.tensor(lens), 0.05)
    np.testing.assert_allclose(out[:, 0], ro, rtol=1e-12, atol=1e-12)
    np.testing.assert_allclose(lse[:, 0], rl, rtol=1e-12)
    none, empty = co.decode(q[:1], [np.zeros((0, 576))], 0.05, sinks=np.array([0.5, -np.inf, 2.0]))
    assert (none == 0).all() and empty[0, 0].tolist() == [0.5, -np.inf, 2.0]


def test_weights_of_a_step_add_up_to_the_query_rows():
    g = np.random.default_rng(3)
    q, keys = g.normal(size=(2, 3, 4, 576)), [g.normal(size=(7, 576)), g.normal(size=(2, 576))]
    _, lse = co.decode(q, keys, 0.1)
    w = co.key_weights(q, lse, keys, 0.1, np.full((2, 8), 5.0), 0.0)
    np.testing.assert_allclose(w[0, :7].sum(), 12, rtol=1e-12)          # every row's weights add up to one
    np.testing.assert_allclose(w[1, :2].sum(), 8, rtol=1e-12)           # its first token sees no key
    assert (w[0, 7:] == 5).all() and (w[1, 2:] == 5).all()
    twice = co.key_weights(q, lse, keys, 0.1, w, 0.5)
    np.testing.assert_allclose(twice[0, :7], 1.5 * w[0, :7], rtol=1e-12)


def test_select_by_hand():
    w = np.array([[5, 1, 1, 9, 1, np.nan, 0, 2, 3, 3.0]])
    idx, count, dropped, bad = co.select_keys(w, [10], [5], 6, 1, 2)
    assert idx.tolist() == [[0, 3, 5, 8, 9, -1]] and count.tolist() == [5] and dropped.tolist() == [-5] and not bad
    assert co.select_keys(w, [7], [5], 5, 0, 0)[0].tolist() == [[0, 1, 2, 3, 5]]          # three of weight 1: the lowest
    assert co.select_keys(w, [10], [3], 3, 4, 2)[0].tolist() == [[0, 8, 9]]               # the last before the first
    assert co.select_keys(w, [10], [2], 2, 4, 8)[0].tolist() == [[8, 9]]
    assert co.select_keys(w, [4], [9], 5, 0, 0)[0].tolist() == [[0, 1, 2, 3, -1]]
    assert co.select_keys(w, [11], [5], 5, 0, 0)[3] == [0] and co.select_keys(w, [9], [8], 7, 0, 0)[3] == [0]


def test_compact_by_hand():
    cache = np.arange(12).reshape(3, 2, 2)
    new, w = co.compact_rows(cache, [[2, 0, 1]], [[0, 2, 4, -1]], [3], np.array([[1.0, 2, 3, 4, 5, 6]]))
    # rows 0, 2, 4 are (page, place) (2, 0), (0, 0), (1, 0)
    assert new[2].tolist() == [[8, 9], [0, 1]] and new[0].tolist() == [[4, 5], [2, 3]] and new[1].tolist() == cache[1].tolist()
    assert w.tolist() == [[1, 3, 5, 4, 5, 6]]


def test_kept_rows_decode_as_before_over_them():
    """Eviction, then attention over what stayed = attention over the chosen rows."""
    g = np.random.default_rng(4)
    cache = g.normal(size=(4, 4, 576))
    table, lens = np.array([[2, 0, 3, 1]]), [14]
    keys = co.held_rows(cache, table, lens, 0)
    idx, count, _, _ = co.select_keys(g.random((1, 16)), lens, [6], 6, 1, 2)
    new, _ = co.compact_rows(cache, table, idx, count)
    np.testing.assert_array_equal(co.held_rows(new, table, count, 0), keys[idx[0]])


@pytest.mark.parametrize("name", co.__all__)
def test_every_function_is_pinned(name):
    with open(__file__) as f:
        text = f.read()
    if name == "kv_append_fp4":        # the rows of kv_append (pinned with the serving step) through quantise_fp4
        c, p = np.ones((1, 512)), np.ones((1, 64))
        cs = np.concatenate([np.ones((1, 32)), np.zeros((1, 32))], 1)
        code, scale, pe, rows, q = co.kv_append_fp4(c, p, [0], cs, 0.5)
        assert (code == 7).all() and (scale == co.round_e4m3(2 / 6)).all() and (pe == 2).all() and (rows == 1).all() and q is None
    else:
        assert f"co.{name}(" in text
