"""Pins of the serving-step oracle: hand-worked cases, torch's own e4m3 conversion, invariants (CPU only)."""
import numpy as np
import pytest
import torch

import oracle.step_oracle as so


def test_e4m3_matches_torch_on_every_bfloat16_pattern():
    v = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).float()
    v = v[torch.isfinite(v)]
    ref = v.clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(so.round_e4m3(v.double().numpy()), ref)
    assert np.isnan(so.round_e4m3(np.nan)) and so.round_e4m3(np.inf) == 448


def test_slot_map_by_hand():
    # page size 4: request 0 grows 3 -> 5 (one new page), 1 shrinks 9 -> 4 (two pages back), 2 starts with 2 tokens
    table = [[7, -1, -1], [3, 5, 6], [-1, -1, -1]]
    pool = [2, 9, 0, 1, -1, -1, -1, -1, 4, 8]           # ring: head 8 -> 4, 8, 2, 9, 0, 1
    pos, slots, cu, lens, state, tab, ring, why = so.slot_map([3, 9, 0], [2, -5, 2], table, pool, [8, 6], 4, 5)
    assert pos.tolist() == [3, 4, 0, 1, -1]
    assert slots.tolist() == [7 * 4 + 3, 4 * 4, 8 * 4, 8 * 4 + 1, -1]
    assert cu.tolist() == [0, 2, 2, 4] and lens.tolist() == [5, 4, 2] and state.tolist() == [0, 6]
    assert tab[0, 1] == 4 and tab[2, 0] == 8 and ring[4:6].tolist() == [5, 6] and not why


def test_slot_map_refusals_by_hand():
    full = so.slot_map([4, 0, 2], [1, 3, 1], [[0], [-1], [1]], [2, 3, -1, -1], [0, 2], 4, 8)
    assert full[-1] == {0x70} and full[3].tolist() == [4, 3, 3]            # request 0 has no room in its table
    none = so.slot_map([0, 0, 1], [5, 1, 1], [[-1, -1]] * 2 + [[0, -1]], [1, 2, 3, -1], [0, 1], 4, 8)
    assert none[-1] == {0x71} and none[3].tolist() == [0, 0, 2] and none[4].tolist() == [0, 1]
    assert none[1].tolist() == [-1] * 6 + [1, -1]


def test_norm_by_hand():
    y, h, s, q = so.rms_norm([[3.0, 4.0]], [1.0, 2.0], 0.0, residual=[[0.0, 0.0]], group=0)
    r = np.sqrt(12.5)
    np.testing.assert_allclose(y, [[3 / r, 8 / r]], rtol=1e-15)
    np.testing.assert_allclose(s, [[8 / r / 448]], rtol=1e-15)
    assert q.tolist() == [[round(3 / 8 * 448 / 16) * 16.0, 448.0]]
    assert so.rms_norm([[0.0, 0.0]], [1.0, 1.0], 1e-6, group=0)[2][0, 0] == 2.0 ** -126


def test_append_rows_by_hand():
    cs = np.zeros((2, 64))
    cs[0, :32], cs[1, 32:] = 1, 1                                       # position 1 turns by 90 degrees
    pe = np.arange(64.0)[None]
    rows, q = so.kv_append(np.full((1, 512), 2.0), pe, [1], cs, np.full(512, 3.0), 0.0, q_pe=pe[:, None], neox=False)
    assert (rows[0, :512] == 3).all()
    np.testing.assert_array_equal(rows[0, 512:].reshape(32, 2), np.stack([-pe[0, 1::2], pe[0, 0::2]], 1))
    np.testing.assert_array_equal(q[0, 0], rows[0, 512:])
    rows, _ = so.kv_append(np.ones((1, 512)), pe, [1], cs, neox=True)
    np.testing.assert_array_equal(rows[0, 512:], np.concatenate([-pe[0, 32:], pe[0, :32]]))


def test_w4_by_hand():
    w4 = np.zeros((1, 1, 32), np.uint8)
    w4[0, 0, 0], w4[0, 0, 31] = 0x2F, 0xF0                              # codes 15, 2 at k = 0, 1; 0, 15 at 62, 63
    w = so.unpack_w4(w4, [[[2.0, 0.5]]])
    assert w[0, 0, :3].tolist() == [14, -12, -16] and w[0, 0, 61:].tolist() == [-4, -4, 3.5]
    x = np.zeros((1, 1, 64))
    x[0, 0, 0], x[0, 0, 63] = 1, 2
    assert so.bmm_w4(x, w4, [[[2.0, 0.5]]])[0][0, 0, 0] == 14 + 7


@pytest.mark.parametrize("seed", range(3))
def test_slot_map_loses_and_doubles_no_page(seed):
    rng = np.random.default_rng(seed)
    B, page, P = 7, 4, 40
    lens, table, ring, state = np.zeros(B, int), np.full((B, 9), -1), rng.permutation(P), np.array([0, P])
    for _ in range(60):
        new = np.where(rng.random(B) < 0.2, -lens, rng.integers(-3, 9, B))
        _, _, _, lens, state, table, ring, _ = so.slot_map(lens, new, table, ring, state, page, 64)
        held = [int(p) for b in range(B) for p in table[b, :-(-lens[b] // page)]]
        free = [int(ring[(state[0] + i) % P]) for i in range(state[1])]
        assert sorted(held + free) == list(range(P))
