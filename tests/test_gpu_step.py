"""The serving step's operators (mla_slot_map, mla_rms_norm, mla_kv_append, mla_bmm_w4) against the
fp64 oracle, at the sizes, strides and masks where they can go wrong, and together as a step uses them.

Tolerances count roundings: an output in bf16 is off by half a step (2^-8 of the value), in e4m3 by
2^-4 of the value or half the smallest step; on top comes the fp32 arithmetic, a relative
2^-16 (256 roundings of 2^-24, more than any sum of positive terms here takes) or, where terms
cancel, its error bound over the sum of their absolute values."""
import numpy as np
import pytest
import torch

import oracle.mla_oracle as mo
import oracle.step_oracle as so
from mla_attention_gb300 import (MLAError, check_device_status, inputs as gen, mla_absorb_q, mla_bmm_w4, mla_decode,
                                 mla_decode_fp8, mla_kv_append, mla_project_out, mla_rms_norm, mla_rope_append,
                                 mla_slot_map)
from tests.helpers import assert_lse_close, assert_out_close, dev, to_np

pytestmark = pytest.mark.gpu

BF16, E4M3, ARITH = 2.0 ** -8, 2.0 ** -4, 2.0 ** -16


def _within(gpu, ref, bound, what):
    g, r = to_np(gpu), np.asarray(ref, np.float64)
    assert g.shape == r.shape, (what, g.shape, r.shape)
    assert (np.isnan(g) == np.isnan(r)).all(), f"{what}: NaN pattern"
    err = np.where(np.isnan(r), 0, np.abs(g - r))
    worst = float(np.where(np.isnan(r), 0, err - bound).max()) if err.size else 0.0
    assert worst <= 0, f"{what}: worst excess {worst:.3e}, largest error {float(err.max()):.3e}"


def _bf16(gpu, ref, what, more=0.0):
    _within(gpu, ref, np.abs(ref) * (BF16 + ARITH) + more + 2.0 ** -126, what)


def _done():
    torch.cuda.synchronize()
    check_device_status()


# ---------------------------------------------------------------------------------------------
# slot map
# ---------------------------------------------------------------------------------------------
def _pages(lens, page, max_pages, spare, g):
    """Tables of requests of these lengths and the ring of the other pages, in random order."""
    have = [-(-n // page) for n in lens]
    P = sum(have) + spare
    ids = torch.randperm(P, generator=g).tolist()
    table = torch.full((len(lens), max_pages), -1, dtype=torch.int32)
    for b, n in enumerate(have):
        table[b, :n] = torch.tensor([ids.pop() for _ in range(n)], dtype=torch.int32)
    head = int(torch.randint(0, max(P, 1), (1,), generator=g))
    ring = torch.full((P,), -1, dtype=torch.int32)
    for i, v in enumerate(ids):
        ring[(head + i) % P] = v
    return table, ring, torch.tensor([head if P else 0, len(ids)], dtype=torch.int32)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32)


def _check_slot_map(lens, new, table, ring, state, page, N, in_place=False):
    d = dev()
    ref = so.slot_map(lens, new, table.numpy(), ring.numpy(), state.numpy(), page, N)
    L, T, R, S = _i32(lens).to(d), table.to(d).clone(), ring.to(d).clone(), state.to(d).clone()
    kw = dict(lens_out=L, pool_state_out=S) if in_place else {}
    for again in range(1 if in_place else 2):   # unchanged inputs: a repeated call writes the same
        got = mla_slot_map(L, _i32(new).to(d), T, R, S, page, N, **kw)
        torch.cuda.synchronize()
        if ref[7]:
            with pytest.raises(MLAError) as e:
                check_device_status()
            assert e.value.status == 5
        else:
            check_device_status()
        for name, a, b in zip(("positions", "slots", "cu_tokens", "lens", "pool_state", "table", "pool"),
                              (*got, T, R), ref):
            np.testing.assert_array_equal(to_np(a), b, err_msg=f"{name} (call {again})")
    return ref[7]


@pytest.mark.parametrize("B,page,N_more,seed", [(1, 64, 0, 1), (3, 1, 2, 2), (65, 16, 7, 3), (1023, 64, 0, 4), (1024, 16, 5, 5),
                                                (1025, 32, 1, 6), (2600, 16, 100, 7), (257, 48, 9000, 8)])
def test_slot_map_random_steps(B, page, N_more, seed):
    g = torch.Generator().manual_seed(seed)
    lens = torch.randint(0, 20 * page, (B,), generator=g).tolist()
    new = torch.randint(-3 * page, 4 * page, (B,), generator=g)
    kind = torch.rand(B, generator=g)
    new = torch.where(kind < 0.5, 1, torch.where(kind < 0.6, 0, torch.where(kind < 0.7, -_i32(lens), new))).tolist()
    table, ring, state = _pages(lens, page, 26, 5 * B + 3, g)
    N = sum(max(n, 0) for n in new) + N_more
    _check_slot_map(lens, new, table, ring, state, page, N)
    _check_slot_map(lens, new, table, ring, state, page, N, in_place=True)


def test_slot_map_one_long_prompt_among_single_tokens():
    g = torch.Generator().manual_seed(11)
    lens = [5] * 40 + [0] + [64] * 40
    new = [1] * 40 + [70001] + [1] * 40
    table, ring, state = _pages(lens, 16, 4400, 4500, g)
    _check_slot_map(lens, new, table, ring, state, 16, 70081 + 33)


@pytest.mark.parametrize("lens,new,N", [([], [], 0), ([], [], 5), ([0], [0], 0), ([0, 0], [0, 0], 3), ([7], [-9], 0), ([0], [1], 1)])
def test_slot_map_empty(lens, new, N):
    table, ring, state = _pages(lens, 4, 3, 3, torch.Generator().manual_seed(12))
    _check_slot_map(lens, new, table, ring, state, 4, N)


def test_slot_map_no_pages_at_all():
    table, ring, state = torch.zeros((2, 0), dtype=torch.int32), torch.zeros(0, dtype=torch.int32), _i32([0, 0])
    _check_slot_map([0, 0], [0, 0], table, ring, state, 16, 2)
    assert _check_slot_map([0, 0], [0, 1], table, ring, state, 16, 2) == {0x70}


@pytest.mark.parametrize("B", [6, 1500])
def test_slot_map_refusals_keep_the_request(B):
    """Each reason alone and all at once; refused requests keep length and pages, the others go on."""
    g = torch.Generator().manual_seed(13)
    page = 4
    base = torch.randint(1, 20, (B,), generator=g).tolist()
    grow = torch.randint(0, 6, (B,), generator=g).tolist()

    def case(lens=None, new=None, spare=6 * B, N=6 * B, state=None, ring=None, table=None, status=0):
        lens, new = list(lens or base), list(new or grow)
        t, r, s = _pages([max(0, min(n, 40)) for n in lens], page, 10, spare, g)
        why = _check_slot_map(lens, new, t if table is None else table(t), r if ring is None else ring(r),
                              s if state is None else _i32(state(len(r))), page, N)
        if B > 1000:                                        # six random requests may all fit
            assert bool(why) == bool(status) and status in (0, *why)

    def at(v, i, x):
        return v[:i] + [x] + v[i + 1:]

    case()
    case(spare=B // 3, status=0x71)
    case(N=B, status=0x72)
    case(lens=at(base, 2, -1), status=0x70)
    case(lens=at(base, 1, 41), status=0x70)
    case(new=at(grow, 3, 2 ** 31 - 1), N=6 * B, status=0x70)
    case(new=at(grow, 3, -2 ** 31))
    case(state=lambda P: [-1, 3], status=0x74)
    case(state=lambda P: [0, P + 1], status=0x74)
    case(state=lambda P: [P, 1], status=0x74)
    case(new=[-20] * B, state=lambda P: [1, P], status=0x73)
    case(ring=lambda r: torch.where(r >= 0, r + 10 ** 6, r), status=0x75)
    case(new=[-20] * B, table=lambda t: torch.where(t >= 0, -7, t), status=0x75)
    case(new=[1] * B, spare=B // 4, N=B - 2, lens=at(base, 0, -3), status=0x70)


@pytest.mark.parametrize("lens,new,state,N,why", [
    ([4, 0, 2], [9, 3, 1], [0, 2], 13, 0x70), ([-1, 0, 2], [1, 3, 1], [0, 2], 13, 0x70), ([4, 0, 2], [1, 9, 1], [3, 2], 13, 0x71),
    ([4, 0, 2], [1, 3, 1], [3, 2], 4, 0x72), ([4, 0, 2], [-4, 3, 1], [3, 6], 4, 0x73), ([4, 0, 2], [1, 3, 1], [6, 2], 13, 0x74),
    ([4, 0, 2], [1, 3, 1], [1, 2], 13, 0x75)])
def test_slot_map_each_refusal(lens, new, state, N, why):
    table, ring = _i32([[4, -1, -1], [-1, -1, -1], [5, -1, -1]]), _i32([2, -9, 6, 0, 1, 3])
    assert why in _check_slot_map(lens, new, table, ring, _i32(state), 4, N)


def test_slot_map_random_walk_in_place():
    """Sixty steps on the device's own state: no page is lost or held twice, whatever is refused."""
    d, rng = dev(), np.random.default_rng(14)
    B, page, P = 37, 4, 200
    lens, table = torch.zeros(B, dtype=torch.int32, device=d), torch.full((B, 16), -1, dtype=torch.int32, device=d)
    ring = torch.randperm(P).to(torch.int32).to(d)
    state = _i32([0, P]).to(d)
    refused = 0
    for _ in range(60):
        now = lens.cpu().numpy()
        new = np.where(rng.random(B) < 0.1, -now, rng.integers(-4, 9, B))
        ref = so.slot_map(now, new, table.cpu(), ring.cpu(), state.cpu(), page, 300)
        got = mla_slot_map(lens, _i32(new.tolist()).to(d), table, ring, state, page, 300, lens_out=lens, pool_state_out=state)
        for a, b in zip((*got, table, ring), ref):
            np.testing.assert_array_equal(to_np(a), b)
        if ref[7]:
            refused += 1
            with pytest.raises(MLAError):
                check_device_status()
        held = [int(p) for b in range(B) for p in table[b, :-(-int(lens[b]) // page)]]
        s = state.tolist()
        assert sorted(held + [int(ring[(s[0] + i) % P]) for i in range(s[1])]) == list(range(P))
    assert refused


# ---------------------------------------------------------------------------------------------
# RMS norm
# ---------------------------------------------------------------------------------------------
def _rows(T, D, pad, off, g, scale=1.0):
    """[T, D] rows inside a wider buffer, `off` elements from its (256-byte aligned) start."""
    buf = (torch.randn((T * (D + pad) + off,), generator=g) * scale).to(torch.bfloat16).to(dev())
    return buf[off:].view(T, D + pad)[:, :D]


def _check_norm(T, D, pad=0, off=0, residual=True, e4m3=False, group=0, eps=1e-6, seed=0, x=None, w=None, in_place=False):
    g = torch.Generator().manual_seed(1000 * T + D + seed)
    x = _rows(T, D, pad, off, g) if x is None else x
    r = _rows(T, D, pad, off, g, 3.0) if residual else None
    w = (1 + 0.3 * torch.randn(D, generator=g)).to(torch.bfloat16).to(dev()) if w is None else w
    ref = so.rms_norm(to_np(x), to_np(w), eps, None if r is None else to_np(r), group if e4m3 else None)
    buf = torch.full((T * (D + pad) + off + 64,), 7.0, device=dev()).to(torch.float8_e4m3fn if e4m3 else torch.bfloat16)
    out = buf[off:off + T * (D + pad)].view(T, D + pad)[:, :D]
    if in_place and not e4m3:
        out = x
    got, ro, scales = mla_rms_norm(x, w, eps, residual=r, residual_out=r if in_place else None, out=out, group=group)
    torch.cuda.synchronize()
    assert got is out
    if residual:
        _bf16(ro, ref[1], "residual_out")
    if not e4m3:
        _bf16(out, ref[0], "out")
    else:
        s = to_np(scales)
        _within(scales, ref[2], ref[2] * ARITH, "scales")
        s_col = np.repeat(s, group or D, axis=1)
        _within(torch.from_numpy(to_np(out) * s_col), ref[0], np.abs(ref[0]) * (E4M3 + 2 * ARITH) + s_col * 2.0 ** -10, "out")
        # where y / s is not next to a border between two values the code is the nearest one
        v = ref[0] / s_col
        sure = so.round_e4m3(v * (1 + 4 * ARITH)) == so.round_e4m3(v * (1 - 4 * ARITH))
        assert (to_np(out)[sure] == so.round_e4m3(v)[sure]).all() and sure.mean() > 0.99
    if not in_place:
        rest = buf.float()
        rest[off:off + T * (D + pad)].view(T, D + pad)[:, :D] = 7
        assert (rest == 7).all(), "columns between and behind the rows were written"


@pytest.mark.parametrize("T", [1, 3, 130])
@pytest.mark.parametrize("D", [1, 7, 8, 64, 255, 256, 257, 511, 512, 520, 1000, 1024, 1535, 1536, 2048, 2055, 4096, 5120, 8192, 8200,
                               16384, 16411, 32768])
def test_norm_widths(T, D):
    _check_norm(T, D, residual=T != 3)


@pytest.mark.parametrize("pad,off", [(0, 0), (8, 8), (64, 0), (65, 0), (3, 1), (0, 5), (8, 4)])
@pytest.mark.parametrize("D,e4m3,group", [(512, False, 0), (576, True, 64), (1536, True, 128), (1535, True, 0), (1536, True, 32), (96, True, 32),
                                          (8192, True, 128), (8200, True, 0), (16384, True, 64)])
def test_norm_strides_and_groups(pad, off, D, e4m3, group):
    _check_norm(5, D, pad, off, residual=pad != 64, e4m3=e4m3, group=group)


@pytest.mark.parametrize("D", [1, 9, 255, 333, 511, 1023, 2047, 8191, 8193])
@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_norm_odd_widths(D, e4m3):
    _check_norm(40, D, e4m3=e4m3, in_place=D % 3 == 0)
    _check_norm(3, D, pad=1, off=1, residual=e4m3, e4m3=e4m3)


@pytest.mark.parametrize("T,D,e4m3,group", [(4900, 2568, False, 0), (4900, 2560, True, 128), (310, 8200, False, 0)])
def test_norm_many_rows(T, D, e4m3, group):
    _check_norm(T, D, e4m3=e4m3, group=group)


def test_norm_in_place():
    for D, e4m3 in ((1536, False), (8192, False), (1535, False), (5120, True)):
        _check_norm(9, D, e4m3=e4m3, in_place=True)
    _check_norm(9, 512, residual=False, in_place=True)


def test_norm_no_rows():
    x = torch.empty((0, 512), dtype=torch.bfloat16, device=dev())
    w = torch.ones(512, dtype=torch.bfloat16, device=dev())
    assert mla_rms_norm(x, w)[0].shape == (0, 512)
    out, _, scales = mla_rms_norm(x, w, e4m3=True, group=128)
    assert out.shape == (0, 512) and scales.shape == (0, 4)


@pytest.mark.parametrize("D", [64, 1535, 8192, 20000])
@pytest.mark.parametrize("e4m3", [False, True])
def test_norm_extreme_rows(D, e4m3):
    """Rows of zeros (eps keeps them 0; the scale is its floor), of the type's largest and smallest values
    (their squares leave fp32's range), and a row shifted by a large mean."""
    big, tiny = torch.finfo(torch.bfloat16).max, 2.0 ** -126
    x = torch.zeros((6, D), dtype=torch.bfloat16)
    x[1], x[2, ::2], x[3] = big, big, tiny
    x[4] = torch.randn(D, generator=torch.Generator().manual_seed(5)) + 1000
    x[5, D // 2] = 2.0 ** 70
    w = torch.ones(D, dtype=torch.bfloat16, device=dev())
    for group in ((0, 32) if e4m3 and D % 32 == 0 else (0,)):
        _check_norm(6, D, residual=False, e4m3=e4m3, group=group, x=x.to(dev()), w=w)
    if not e4m3:   # eps = 0: a row far below 1 is still normed
        x = torch.full((2, D), 2.0 ** -60, dtype=torch.bfloat16, device=dev())
        _check_norm(2, D, residual=False, eps=0.0, x=x, w=w)


def test_norm_nan_and_infinity():
    x = torch.randn((4, 256), generator=torch.Generator().manual_seed(6)).to(torch.bfloat16)
    x[1, 17], x[2, 200] = float("nan"), float("inf")
    w = torch.ones(256, dtype=torch.bfloat16, device=dev())
    _check_norm(4, 256, residual=False, x=x.to(dev()), w=w)
    out, _, scales = mla_rms_norm(x.to(dev()), w, e4m3=True, group=64)
    y, s = to_np(out).reshape(4, 4, 64), to_np(scales)
    assert np.isnan(s[1]).all() and np.isnan(s[2]).tolist() == [False, False, False, True]
    assert np.isnan(y[1]).all() and np.isnan(y[2, 3]).all() and (y[2, :3] == 0).all() and np.isfinite(y[[0, 3]]).all()


def test_norm_infinite_weight_and_codes_at_borders():
    """An infinite weight makes its group's scale infinite and its finite values 0; with power-of-two rows the
    quotients are exact and every code is the nearest one, ties to even."""
    x = torch.ones((1, 128), dtype=torch.bfloat16, device=dev())
    w = torch.ones(128, dtype=torch.bfloat16)
    w[5] = float("inf")
    out, _, scales = mla_rms_norm(x, w.to(dev()), eps=0.0, e4m3=True, group=64)
    y, s = to_np(out)[0], to_np(scales)[0]
    assert np.isinf(s[0]) and np.isnan(y[5]) and (np.delete(y[:64], 5) == 0).all() and s[1] == np.float32(1 / 448) and (y[64:] == 448).all()
    # |x| = 1 everywhere: y = w; the first weight fixes the scale at 1, the others are e4m3 values and their midpoints
    steps = torch.arange(0, 448 * 2 + 1, dtype=torch.float32) / 2
    mids = steps[(steps == steps.to(torch.bfloat16).float())]
    w = torch.cat([torch.tensor([448.0]), mids]).to(torch.bfloat16).to(dev())
    x = torch.ones((1, w.numel()), dtype=torch.bfloat16, device=dev())
    x[:, ::2] = -1
    out, _, scales = mla_rms_norm(x, w, eps=0.0, e4m3=True)
    assert to_np(scales)[0, 0] == 1
    np.testing.assert_array_equal(to_np(out)[0], so.round_e4m3(to_np(x)[0] * to_np(w)))


def test_norm_rows_past_2_31_elements():
    T, D = 70000, 32768
    x = torch.zeros((T, D), dtype=torch.bfloat16, device=dev())
    g = torch.Generator().manual_seed(7)
    x[-3:] = _rows(3, D, 0, 0, g)
    w = torch.ones(D, dtype=torch.bfloat16, device=dev())
    out, _, _ = mla_rms_norm(x, w)
    _bf16(out[-3:], so.rms_norm(to_np(x[-3:]), to_np(w), 1e-6)[0], "last rows")
    assert not out[:-3].any()


# ---------------------------------------------------------------------------------------------
# cache append
# ---------------------------------------------------------------------------------------------
def _check_append(T, H, e4m3=False, neox=False, norm=True, rows_out=False, page=16, pages=None, strided=True, bad=False, seed=0):
    g = torch.Generator().manual_seed(77 * T + H + seed)
    d, max_pos = dev(), 300
    pages = -(-T // page) + 2 if pages is None else pages
    kv = gen.randn_bf16((T, 1536 + 576 if strided else 576), g).to(d)
    c_kv, k_pe = kv[:, -576:-64], kv[:, -64:]
    w = (1 + 0.3 * torch.randn(512, generator=g)).to(torch.bfloat16).to(d) if norm else None
    scale = 0.0173 if e4m3 else 1.0
    cache = gen.randn_bf16((pages, page, 576), g).to(torch.float8_e4m3fn if e4m3 else torch.bfloat16).to(d)
    slots = torch.randperm(pages * page, generator=g)[:T].to(torch.int32)
    pos = torch.randint(0, max_pos, (T,), generator=g).to(torch.int32)
    if T > 2:
        pos[1] = slots[1] = -1          # no token
        slots[2] = -1                   # a token that is not cached
    if bad:
        pos[0], slots[-1] = max_pos, pages * page
    cs = gen.rope_cos_sin(max_pos)
    q = gen.randn_bf16((T, max(H, 1), 192 if strided else 64), g).to(d)[:, :, -64:]
    q_out = gen.randn_bf16((T, max(H, 1), 584 if strided else 576), g).to(d)
    kv_out = gen.randn_bf16((T, 584 if strided else 576), g).to(d)
    before = [to_np(t) for t in (cache, q_out, kv_out)]
    mla_kv_append(c_kv, k_pe, slots.to(d), pos.to(d), cs.to(d), cache, scale, norm_weight=w, eps=1e-5, is_neox=neox,
                  q_pe=q if H else None, q_out=q_out[:, :, :576] if H else None, kv_out=kv_out[:, :576] if rows_out else None)
    torch.cuda.synchronize()
    if bad:
        with pytest.raises(MLAError) as e:
            check_device_status()
        assert e.value.status == 5
    check_device_status()
    live = np.flatnonzero((pos.numpy() >= 0) & (pos.numpy() < max_pos))
    ref, rq = so.kv_append(to_np(c_kv)[live], to_np(k_pe)[live], pos.numpy()[live], cs.numpy(),
                           None if w is None else to_np(w), 1e-5, to_np(q)[live] if H else None, neox)
    turned = 8 * 2.0 ** -22                                  # |a c| + |b s| <= 8 for N(0, 1) draws of a million
    more = np.zeros(576)
    more[512:] = turned
    cached = [(i, t) for i, t in enumerate(live) if 0 <= slots[t] < pages * page]
    rows = to_np(cache).reshape(-1, 576)
    at = [int(slots[t]) for _, t in cached]
    want = ref[[i for i, _ in cached]]
    if e4m3:
        clip = np.clip(want, -448 * scale, 448 * scale)
        _within(torch.from_numpy(rows[at] * scale), clip, np.abs(clip) * (E4M3 + ARITH) + scale * 2.0 ** -10 + more, "cache rows")
    else:
        _bf16(torch.from_numpy(rows[at]), want, "cache rows", more)
    other = np.ones(pages * page, bool)
    other[at] = False
    np.testing.assert_array_equal(rows[other], before[0].reshape(-1, 576)[other])
    if H:
        _bf16(q_out[torch.from_numpy(live).to(d), :, 512:576], rq, "turned q_pe", turned)
        rest = to_np(q_out)
        rest[live, :, 512:576] = before[1][live, :, 512:576]
        np.testing.assert_array_equal(rest, before[1])
    if rows_out:
        _bf16(kv_out[torch.from_numpy(live).to(d), :576], ref, "kv_out", more)
        rest = to_np(kv_out)
        rest[live, :576] = before[2][live, :576]
        np.testing.assert_array_equal(rest, before[2])
    else:
        np.testing.assert_array_equal(to_np(kv_out), before[2])


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("neox", [False, True], ids=["interleaved", "halves"])
@pytest.mark.parametrize("T,H", [(1, 0), (1, 128), (5, 1), (33, 40), (130, 16), (7, 33)])
def test_append_shapes(T, H, neox, e4m3):
    _check_append(T, H, e4m3, neox, norm=T != 5, rows_out=H % 2 == 0)


@pytest.mark.parametrize("page", [1, 64, 128])
def test_append_pages_and_dense_rows(page):
    _check_append(70, 8, e4m3=page == 64, page=page, strided=False, rows_out=True)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_append_reports_and_skips_bad_rows(e4m3):
    _check_append(40, 16, e4m3, rows_out=True, bad=True)


@pytest.mark.parametrize("neox", [False, True], ids=["interleaved", "halves"])
def test_append_in_place(neox):
    """kv_out over c_kv and k_pe themselves and q_out over q_pe: the same bits as into buffers of their own."""
    d, g, T, H = dev(), torch.Generator().manual_seed(9), 21, 5
    kv, q = gen.randn_bf16((T, 576), g).to(d), gen.randn_bf16((T, H, 576), g).to(d)
    w = (1 + 0.3 * torch.randn(512, generator=g)).bfloat16().to(d)
    slots, pos, cs = torch.randperm(32, generator=g)[:T].to(torch.int32).to(d), _i32(list(range(T))).to(d), gen.rope_cos_sin(64).to(d)
    one, two = torch.zeros((2, 16, 576), dtype=torch.bfloat16, device=d), torch.zeros((2, 16, 576), dtype=torch.bfloat16, device=d)
    rows, q2 = torch.empty_like(kv), q.clone()
    mla_kv_append(kv[:, :512], kv[:, 512:], slots, pos, cs, one, norm_weight=w, q_pe=q[:, :, 512:], q_out=q2, kv_out=rows, is_neox=neox)
    mla_kv_append(kv[:, :512], kv[:, 512:], slots, pos, cs, two, norm_weight=w, q_pe=q[:, :, 512:], q_out=q, kv_out=kv, is_neox=neox)
    _done()
    assert torch.equal(one, two) and torch.equal(rows, kv) and torch.equal(q2, q)
    assert torch.equal(one.view(-1, 576)[slots.long()], kv)


def test_append_norms_rows_whose_squares_overflow():
    g, d = torch.Generator().manual_seed(12), dev()
    c = torch.randn((4, 512), generator=g)
    c[0] *= 2.0 ** 80
    c[2, 7] = 2.0 ** 100
    c[3] *= 2.0 ** -30
    c = c.to(torch.bfloat16).to(d)
    pe = gen.randn_bf16((4, 64), g).to(d)
    w = (1 + 0.3 * torch.randn(512, generator=g)).to(torch.bfloat16).to(d)
    cs, pos = gen.rope_cos_sin(8), _i32([0, 3, 5, 7])
    cache = torch.zeros((1, 4, 576), dtype=torch.bfloat16, device=d)
    mla_kv_append(c, pe, _i32([0, 1, 2, 3]).to(d), pos.to(d), cs.to(d), cache, norm_weight=w, eps=0.0)
    ref, _ = so.kv_append(to_np(c), to_np(pe), pos.numpy(), cs.numpy(), to_np(w), 0.0, None, False)
    _bf16(cache[0, :, :512], ref[:, :512], "latents")


def test_append_saturates_and_keeps_nan():
    d = dev()
    c_kv, k_pe = torch.full((2, 512), 1000.0).bfloat16().to(d), torch.zeros((2, 64)).bfloat16().to(d)
    c_kv[1, 3], c_kv[1, 4], c_kv[1, 5] = float("nan"), -float("inf"), 449.0
    cache = torch.zeros((1, 16, 576), device=d).to(torch.float8_e4m3fn)
    mla_kv_append(c_kv, k_pe, _i32([3, 4]).to(d), _i32([0, 1]).to(d), gen.rope_cos_sin(4).to(d), cache, 1.0)
    _done()
    got = to_np(cache)[0]
    assert (got[3, :512] == 448).all() and np.isnan(got[4, 3]) and got[4, 4] == -448 and got[4, 5] == 448
    assert not got[:3].any() and not got[5:].any()


def test_append_into_a_cache_past_2_31_elements():
    d = dev()
    pages, page = 60000, 64                                  # 2.2e9 elements
    cache = torch.zeros((pages, page, 576), dtype=torch.bfloat16, device=d)
    g = torch.Generator().manual_seed(8)
    c_kv, k_pe = gen.randn_bf16((2, 512), g).to(d), gen.randn_bf16((2, 64), g).to(d)
    mla_kv_append(c_kv, k_pe, _i32([pages * page - 1, pages * page - 70]).to(d), _i32([0, 0]).to(d), gen.rope_cos_sin(4).to(d), cache)
    _done()
    rows = cache.view(-1, 576)
    for t, s in ((0, -1), (1, -70)):                         # position 0: no turn; no norm: copied exactly
        np.testing.assert_array_equal(to_np(rows[s]), np.concatenate([to_np(c_kv[t]), to_np(k_pe[t])]))
    assert int((rows[-80:] != 0).any(1).sum()) == 2


def test_append_equals_rope_append():
    """One token per request without a norm: the decode step's call and this one write the same bits."""
    D = gen.decode_inputs([n + 1 for n in (0, 10, 63, 64, 130)], H=16, seed=13, page_size=16)
    g, d, B = torch.Generator().manual_seed(14), dev(), 5
    q_pe, c_kv, k_pe = gen.randn_bf16((B, 16, 64), g).to(d), gen.randn_bf16((B, 512), g).to(d), gen.randn_bf16((B, 64), g).to(d)
    pos, cs, bt = _i32([0, 10, 63, 64, 130]).to(d), gen.rope_cos_sin(512).to(d), D.block_table.to(d)
    slots = bt[torch.arange(B, device=d), (pos // 16).long()] * 16 + pos % 16
    for neox in (False, True):
        one, two = D.cache.to(d).clone(), D.cache.to(d).clone()
        qa, qb = D.q.to(d).clone(), D.q.to(d).clone()
        mla_rope_append(q_pe, c_kv, k_pe, pos, cs, one, bt, qa, is_neox=neox)
        mla_kv_append(c_kv, k_pe, slots, pos, cs, two, q_pe=q_pe, q_out=qb, is_neox=neox)
        _done()
        assert torch.equal(one, two) and torch.equal(qa, qb)


# ---------------------------------------------------------------------------------------------
# products with 4-bit weights
# ---------------------------------------------------------------------------------------------
def _w4(H, N, K, group, f32, g):
    w4 = torch.randint(0, 256, (H, N, K // 2), generator=g).to(torch.uint8)
    scales = (0.3 + torch.rand((H, N, K // group), generator=g)) * (0.25 / K ** 0.5)
    return w4.to(dev()), (scales if f32 else scales.to(torch.bfloat16)).to(dev())


def _check_w4(T, H, N, K, group, f32=False, strided=False, seed=0):
    g = torch.Generator().manual_seed(31 * T + N + K + seed)
    w4, scales = _w4(H, N, K, group, f32, g)
    pad = 5 if strided else 0
    x = gen.randn_bf16((T, H, K + pad), g).to(dev())[:, :, pad:]
    buf = torch.full((T, H, N + 9 if strided else N), 3.0, dtype=torch.bfloat16, device=dev())
    out = mla_bmm_w4(x, w4, scales, out=buf[:, :, :N])
    torch.cuda.synchronize()
    ref, mass = so.bmm_w4(to_np(x), w4.cpu().numpy(), to_np(scales))
    _bf16(out, ref, "out", mass * K * 2.0 ** -24)
    assert (buf[:, :, N:] == 3).all()


@pytest.mark.parametrize("T", [0, 1, 2, 7, 8, 9, 16, 17, 24, 25, 31, 33, 48, 49, 64, 65, 130])
@pytest.mark.parametrize("H,N,K,group", [(3, 512, 128, 32), (2, 128, 512, 64), (1, 100, 1024, 128)])
def test_w4_tokens(T, H, N, K, group):
    _check_w4(T, H, N, K, group, f32=T % 2 == 0)


@pytest.mark.parametrize("H,N,K,group", [(1, 1, 32, 32), (1, 17, 96, 32), (2, 15, 64, 64), (5, 33, 160, 32), (1, 64, 128, 128), (1, 2, 4096, 64),
                                         (1, 1000, 2080, 32), (1, 7, 16384, 128), (4, 31, 1984, 64), (128, 16, 128, 128), (1, 4100, 640, 128)])
@pytest.mark.parametrize("T", [1, 5, 20])
def test_w4_widths(T, H, N, K, group):
    _check_w4(T, H, N, K, group, f32=N % 2 == 1, strided=T == 5)


@pytest.mark.parametrize("T,H,N,K,group", [(1, 128, 512, 128, 32), (3, 90, 700, 1024, 128), (5, 90, 700, 640, 64), (17, 60, 700, 512, 64),
                                           (64, 40, 700, 384, 32), (130, 24, 513, 256, 128)])
@pytest.mark.parametrize("strided", [False, True])
def test_w4_several_rounds_of_columns(T, H, N, K, group, strided):
    _check_w4(T, H, N, K, group, f32=strided, strided=strided)


def test_w4_most_columns():
    """34 GB of weights; the column numbers reach 2^31 - 2."""
    g, d, N = torch.Generator().manual_seed(8), dev(), 2 ** 31 - 1
    w4 = torch.empty((1, N, 16), dtype=torch.uint8, device=d).random_()
    scales = torch.empty((1, N, 1), dtype=torch.bfloat16, device=d).uniform_(0.5, 1.5)
    x = gen.randn_bf16((2, 1, 32), g).to(d)
    out = mla_bmm_w4(x, w4, scales)
    _done()
    at = torch.cat([torch.arange(300), torch.randint(0, N, (2000,), generator=g), torch.arange(N - 300, N)]).to(d)
    ref, mass = so.bmm_w4(to_np(x), w4[:, at].cpu().numpy(), to_np(scales[:, at]))
    _bf16(out[:, :, at], ref, "out", mass * 32 * 2.0 ** -24)
    del w4, scales, out
    torch.cuda.empty_cache()


def test_w4_infinity_in_several_rounds():
    g = torch.Generator().manual_seed(3)
    w4, scales = _w4(60, 700, 512, 64, False, g)
    x = gen.randn_bf16((20, 60, 512), g)
    x[3, 59, 500] = float("inf")
    out, clean = to_np(mla_bmm_w4(x.to(dev()), w4, scales)), x.clone()
    clean[3, 59, 500] = 0
    ref, mass = so.bmm_w4(to_np(clean), w4.cpu().numpy(), to_np(scales))
    code = so.unpack_w4(w4.cpu().numpy(), to_np(scales))[59, :, 500]
    assert (~np.isfinite(out[3, 59])).all() and (np.sign(out[3, 59])[code != 0] == np.sign(code)[code != 0]).all()
    rest = np.ones((20, 60), bool)
    rest[3, 59] = False
    _bf16(torch.from_numpy(out[rest]), ref[rest], "out", mass[rest] * 512 * 2.0 ** -24)


@pytest.mark.parametrize("f32", [False, True], ids=["bf16", "fp32"])
@pytest.mark.parametrize("off", [0, 1, 2, 4])
@pytest.mark.parametrize("H,N,K,group", [(3, 40, 256, 32), (1, 64, 1792, 64), (1, 64, 1792, 128), (2, 20, 1664, 128)])
def test_w4_scales_off_their_boundaries(H, N, K, group, off, f32):
    g = torch.Generator().manual_seed(N + K + off)
    w4, scales = _w4(H, N, K, group, f32, g)
    buf = torch.full((scales.numel() + off,), float("nan"), dtype=scales.dtype, device=dev())
    at = buf[off:].view(scales.shape)
    at.copy_(scales)
    x = gen.randn_bf16((3, H, K), g).to(dev())
    out = mla_bmm_w4(x, w4, at)
    ref, mass = so.bmm_w4(to_np(x), w4.cpu().numpy(), to_np(scales))
    _bf16(out, ref, "out", mass * K * 2.0 ** -24)


def test_w4_codes_are_exact():
    """One-hot rows read single weights back: every code of every k, times its own group's scale, in its own place."""
    H, N, K = 2, 24, 256
    g = torch.Generator().manual_seed(40)
    w4 = torch.randint(0, 256, (H, N, K // 2), generator=g).to(torch.uint8).to(dev())
    scales = torch.exp2(torch.randint(-3, 4, (H, N, K // 32), generator=g).float()).to(torch.bfloat16).to(dev())
    x = torch.eye(K, dtype=torch.bfloat16, device=dev())[:, None, :].expand(K, H, K)
    out = mla_bmm_w4(x, w4, scales)
    np.testing.assert_array_equal(to_np(out), so.unpack_w4(w4.cpu().numpy(), to_np(scales)).transpose(2, 0, 1))


def test_w4_infinity_stays_in_its_token():
    """A token's NaN or infinity reaches its own outputs only, the padded places of a tile none."""
    g = torch.Generator().manual_seed(41)
    w4, scales = _w4(2, 64, 256, 64, False, g)
    w4 |= 1                                                   # no code 8 at even k: every weight there is nonzero
    x = gen.randn_bf16((11, 2, 256), g)
    x[3, 0, 10], x[7, 1, 20] = float("nan"), float("inf")
    out = to_np(mla_bmm_w4(x.to(dev()), w4, scales))
    bad = ~np.isfinite(out)
    assert bad[3, 0].all() and bad[7, 1].all() and bad.sum() == 128


@pytest.mark.parametrize("T", [1, 9, 33])
def test_w4_large_and_small_values(T):
    """Rows of x far from one: sums beyond any scaling of the products are exact to the same bound, infinities keep
    their sign, NaN stays in its row."""
    g = torch.Generator().manual_seed(42 + T)
    H, N, K = 2, 40, 256
    w4, scales = _w4(H, N, K, 64, T == 9, g)
    w4 |= 0x11                                                # no code 8: every weight is nonzero
    x = gen.randn_bf16((T, H, K), g)
    x[0] *= 2.0 ** 100
    x[T // 2, 1] *= 2.0 ** -40
    x[T - 1, 0, 5] = 2.0 ** 120
    if T > 8:
        x[3, 0, 7], x[5, 1, 9], x[6, 1, 2] = float("inf"), -float("inf"), float("nan")
    out = mla_bmm_w4(x.to(dev()), w4, scales)
    with np.errstate(invalid="ignore"):
        ref, mass = so.bmm_w4(to_np(x), w4.cpu().numpy(), to_np(scales))
    finite = np.isfinite(ref)
    o = to_np(out)
    assert (np.isnan(o) == np.isnan(ref)).all() and (o[np.isinf(ref)] == ref[np.isinf(ref)]).all()
    err = np.abs(np.where(finite, o - np.where(finite, ref, 0), 0))
    assert (err <= np.where(finite, np.abs(np.where(finite, ref, 0)) * (BF16 + ARITH) + np.where(finite, mass, 0) * K * 2.0 ** -24, 0)).all()


# ---------------------------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------------------------
def _serve(e4m3, graph, stream=None):
    """A few steps of six requests (a prompt, decode steps, dropped draft tokens, a request that ends and
    one that starts) through every operator, with the attention in between; returns what must match."""
    d, g = dev(), torch.Generator().manual_seed(50)
    B, H, page, P, HID, N, max_pages = 6, 16, 16, 64, 1024, 64, 12
    kv_scale = 0.021 if e4m3 else 1.0
    table, ring = torch.full((B, max_pages), -1, dtype=torch.int32, device=d), torch.randperm(P, generator=g).to(torch.int32).to(d)
    state, lens, new = _i32([5, P]).to(d), torch.zeros(B, dtype=torch.int32, device=d), torch.zeros(B, dtype=torch.int32, device=d)
    cache = torch.zeros((P, page, 576), device=d).to(torch.float8_e4m3fn if e4m3 else torch.bfloat16)
    w_in = (1 + 0.2 * torch.randn(HID, generator=g)).bfloat16().to(d)
    w_lat = (1 + 0.2 * torch.randn(512, generator=g)).bfloat16().to(d)
    down = (torch.randn((HID, 576 + H * 192), generator=g) / HID ** 0.5).bfloat16().to(d)
    wk, sk = _w4(H, 512, 128, 64, False, g)
    wv, sv = _w4(H, 128, 512, 128, True, g)
    wo, s_o = _w4(1, HID, H * 128, 128, False, g)
    cs = gen.rope_cos_sin(256).to(d)
    i32 = dict(dtype=torch.int32, device=d)
    pos, slots, cu = torch.empty(N, **i32), torch.empty(N, **i32), torch.empty(B + 1, **i32)
    x, res = torch.zeros((N, HID), dtype=torch.bfloat16, device=d), torch.zeros((N, HID), dtype=torch.bfloat16, device=d)
    q = torch.zeros((N, H, 576), dtype=torch.bfloat16, device=d)
    kept = {}

    def step():
        mla_slot_map(lens, new, table, ring, state, page, N, positions=pos, slots=slots, cu_tokens=cu, lens_out=lens,
                     pool_state_out=state)
        h, _, _ = mla_rms_norm(x, w_in, residual=res, residual_out=res)
        y = h @ down
        qp = y[:, 576:].view(N, H, 192)
        mla_bmm_w4(qp[:, :, :128], wk, sk, out=q[:, :, :512])
        mla_kv_append(y[:, :512], y[:, 512:576], slots, pos, cs, cache, kv_scale, norm_weight=w_lat, q_pe=qp[:, :, 128:], q_out=q)
        last = q[(cu[1:] - 1).clamp(min=0).long()]
        if e4m3:
            o, lse = mla_decode_fp8(last, cache, kv_scale, table, lens, gen.SCALE_192)
        else:
            o, lse = mla_decode(last, cache, table, lens, gen.SCALE_192)
        v = mla_bmm_w4(o, wv, sv)
        z = mla_bmm_w4(v.view(B, 1, H * 128), wo, s_o)
        kept.update(h=h, y=y, last=last, o=o, lse=lse, v=v, z=z)

    steps = [[40, 0, 3, 1, 0, 9], [1, 20, 1, 1, 5, 1], [-2, 1, 1, 1, -3, 1], [1, 1, -99, 1, 1, 1], [1, 0, 7, 1, 1, 1]]
    xs = [gen.randn_bf16((N, HID), g).to(d) for _ in steps]
    torch.cuda.synchronize()
    got, run, G = [], step, None
    for k, n in enumerate(steps):
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            new.copy_(_i32(n))
            x.copy_(xs[k])
            if graph and k == 1:
                torch.cuda.synchronize()
                G = torch.cuda.CUDAGraph()
                with torch.cuda.graph(G):
                    step()
                run = G.replay
            before = dict(lens=lens.clone(), table=table.clone(), ring=ring.clone(), state=state.clone(), res=res.clone(), cache=cache.clone())
            run()
            got.append({**{a: b.clone() for a, b in kept.items()}, "pos": pos.clone(), "slots": slots.clone(), "lens": lens.clone(),
                        "table": table.clone(), "cache": cache.clone(), "res": res.clone(), "q": q.clone(), "before": before, "new": n, "x": xs[k]})
        torch.cuda.synchronize()
        check_device_status()
    return got, dict(w_in=w_in, w_lat=w_lat, wk=(wk, sk), wv=(wv, sv), wo=(wo, s_o), cs=cs, kv_scale=kv_scale, page=page, N=N)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_serving_steps(e4m3):
    """Each operator of each step against the oracle on its own inputs, and the attention over what they wrote."""
    got, c = _serve(e4m3, graph=False)
    for s in got:
        b = s["before"]
        ref = so.slot_map(b["lens"].cpu(), s["new"], b["table"].cpu(), b["ring"].cpu(), b["state"].cpu(), c["page"], c["N"])
        for name, r in zip(("pos", "slots"), ref):
            np.testing.assert_array_equal(to_np(s[name]), r)
        np.testing.assert_array_equal(to_np(s["table"]), ref[5])
        np.testing.assert_array_equal(to_np(s["lens"]), ref[3])
        y, h = so.rms_norm(to_np(s["x"]), to_np(c["w_in"]), 1e-6, to_np(b["res"]))
        _bf16(s["h"], y, "normed")
        _bf16(s["res"], h, "residual")
        live = np.flatnonzero(ref[0] >= 0)
        act = to_np(s["y"])[live]
        rows, rq = so.kv_append(act[:, :512], act[:, 512:576], ref[0][live], to_np(c["cs"]), to_np(c["w_lat"]), 1e-6,
                                act[:, 576:].reshape(-1, 16, 192)[:, :, 128:])
        cached = to_np(s["cache"]).reshape(-1, 576)[ref[1][live]] * c["kv_scale"]
        _within(torch.from_numpy(cached), rows, np.abs(rows) * ((E4M3 if e4m3 else BF16) + ARITH) + (c["kv_scale"] * 2.0 ** -10 if e4m3 else 0)
                + 2.0 ** -19, "rows in the cache")
        lift, mass = so.bmm_w4(act[:, 576:].reshape(-1, 16, 192)[:, :, :128], c["wk"][0].cpu().numpy(), to_np(c["wk"][1]))
        _bf16(s["q"][torch.from_numpy(live).to(dev())], np.concatenate([lift, rq], 2), "fused query",
              np.concatenate([mass * 2.0 ** -17, np.full(rq.shape, 2.0 ** -19)], 2))
        full = s["cache"].double().cpu().numpy() * c["kv_scale"]
        ro, rl = mo.mla_decode(s["last"].cpu(), torch.from_numpy(full), s["table"].cpu(), s["lens"].cpu(), gen.SCALE_192)
        assert_out_close(s["o"], ro)
        assert_lse_close(s["lse"], rl)
        v, mass = so.bmm_w4(to_np(s["o"]), c["wv"][0].cpu().numpy(), to_np(c["wv"][1]))
        _bf16(s["v"], v, "values", mass * 2.0 ** -15)
        z, mass = so.bmm_w4(to_np(s["v"]).reshape(6, 1, -1), c["wo"][0].cpu().numpy(), to_np(c["wo"][1]))
        _bf16(s["z"], z, "output", mass * 2.0 ** -13)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_serving_steps_captured_and_replayed(e4m3):
    """The step captured into a graph, its state advancing in place on every replay, gives the eager steps' bits."""
    eager, _ = _serve(e4m3, graph=False)
    graph, _ = _serve(e4m3, graph=True)
    for a, b in zip(eager, graph):
        for name in ("pos", "slots", "lens", "table", "res", "cache", "q", "o", "z"):
            assert torch.equal(a[name].view(torch.uint8), b[name].view(torch.uint8)), name


def test_serving_steps_on_another_stream():
    one, _ = _serve(False, graph=False)
    two, _ = _serve(False, graph=False, stream=torch.cuda.Stream())
    for a, b in zip(one, two):
        for name in ("pos", "slots", "cache", "q", "z"):
            assert torch.equal(a[name], b[name]), name


def test_a_refused_request_stops_no_other_call():
    """A pool that runs out is reported when the status is read, and until then nothing else gives up its waits."""
    d, g = dev(), torch.Generator().manual_seed(70)
    D = gen.decode_inputs([300, 17, 129], H=16, seed=71, page_size=16)
    w4, sc = _w4(16, 128, 512, 64, False, g)
    x = gen.randn_bf16((5, 16, 512), g).to(d)
    args = (D.q.to(d), D.cache.to(d), D.block_table.to(d), D.lens.to(d), D.scale)
    out, lse = mla_decode(*args)
    y = mla_bmm_w4(x, w4, sc)
    _done()
    z = torch.zeros(2, dtype=torch.int32, device=d)
    mla_slot_map(z, z + 50, torch.full((2, 9), -1, dtype=torch.int32, device=d), _i32([0, 1, 2, 3]).to(d), _i32([0, 4]).to(d), 16, 100)
    for _ in range(3):
        out2, lse2 = mla_decode(*args)
        assert torch.equal(out, out2) and torch.equal(lse, lse2) and torch.equal(y, mla_bmm_w4(x, w4, sc))
    with pytest.raises(MLAError) as e:
        check_device_status()
    assert e.value.status == 5 and "0x71" in str(e.value)
    check_device_status()


def test_a_graph_outlives_a_larger_workspace():
    """A captured step keeps the status word that it was captured with, whatever later calls need."""
    from mla_attention_gb300 import workspace
    d, g = dev(), torch.Generator().manual_seed(72)
    D = gen.decode_inputs([40, 17], H=16, seed=73, page_size=16)
    args = (D.q.to(d), D.cache.to(d), D.block_table.to(d), D.lens.to(d), D.scale)
    w4, sc = _w4(16, 128, 512, 64, False, g)
    mla_bmm_w4(mla_decode(*args)[0], w4, sc)
    torch.cuda.synchronize()
    G = torch.cuda.CUDAGraph()
    with torch.cuda.graph(G):
        o, lse = mla_decode(*args)
        y = mla_bmm_w4(o, w4, sc)
    G.replay()
    torch.cuda.synchronize()
    first = y.clone()
    ws = workspace(256, d)
    bigger = workspace(2 * ws.numel(), d)
    assert bigger.data_ptr() != ws.data_ptr()
    size = ws.numel()
    del ws
    junk = [torch.full((size,), 255, dtype=torch.uint8, device=d) for _ in range(4)]
    y.zero_()
    G.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, first) and all((j == 255).all() for j in junk)
    check_device_status()


def test_explicit_stream_argument():
    """The call runs on the stream it is given, after that stream's own work."""
    d, s = dev(), torch.cuda.Stream()
    w = torch.ones(4096, dtype=torch.bfloat16, device=d)
    x = torch.zeros((2048, 4096), dtype=torch.bfloat16, device=d)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(20):
            x.add_(1.0)
    out, _, _ = mla_rms_norm(x, w, stream=s)
    s.synchronize()
    assert (out == 1).all()


def test_outputs_lie_in_the_memory_of_the_stream_that_writes_them():
    """An output made for a call on another stream is not handed, when dropped, to the current stream's next
    tensor while the call may still write it."""
    d, s = dev(), torch.cuda.Stream()
    x = torch.ones((64, 8192), dtype=torch.bfloat16, device=d)
    w = torch.ones(8192, dtype=torch.bfloat16, device=d)
    torch.cuda.synchronize()
    for stream in (s, s.cuda_stream):
        out, _, _ = mla_rms_norm(x, w, stream=stream)
        at = out.data_ptr()
        del out
        assert torch.empty_like(x).data_ptr() != at
    torch.cuda.synchronize()
    assert (mla_rms_norm(x, w, stream=0)[0] == 1).all()


@pytest.mark.filterwarnings("ignore:The CUDA Graph is empty")
def test_a_first_call_inside_a_capture_is_refused():
    """It would put the status word into the graph's memory."""
    from mla_attention_gb300 import _lib
    d = dev()
    x, w4, scales = (torch.zeros(1, 1, 32, dtype=torch.bfloat16, device=d), torch.zeros(1, 1, 16, dtype=torch.uint8, device=d),
                     torch.zeros(1, 1, 1, dtype=torch.bfloat16, device=d))
    out = mla_bmm_w4(x, w4, scales)
    word = _lib._status_cache.pop(d.index or 0)
    try:
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            with pytest.raises(MLAError, match="capture"):
                mla_bmm_w4(x, w4, scales, out=out)
    finally:
        _lib._status_cache[d.index or 0] = word


def test_norm_refuses_an_output_of_another_type():
    x = torch.ones((2, 512), dtype=torch.bfloat16, device=dev())
    with pytest.raises(MLAError) as e:
        mla_rms_norm(x, x[0], out=torch.empty_like(x), e4m3=True)
    assert e.value.status == 1


def test_w4_stands_in_for_the_absorption_products():
    """The same step with 16-bit weights of the same values: mla_absorb_q / mla_project_out and mla_bmm_w4 agree."""
    g, d = torch.Generator().manual_seed(60), dev()
    wk, sk = _w4(16, 512, 128, 128, False, g)
    wv, sv = _w4(16, 128, 512, 128, False, g)
    sk, sv = torch.exp2(torch.round(torch.log2(sk.float()))).bfloat16(), torch.exp2(torch.round(torch.log2(sv.float()))).bfloat16()
    dense = [torch.from_numpy(so.unpack_w4(w.cpu().numpy(), to_np(s))).to(torch.bfloat16).to(d) for w, s in ((wk, sk), (wv, sv))]
    q, o = gen.randn_bf16((9, 16, 128), g).to(d), gen.randn_bf16((9, 16, 512), g).to(d)
    a, b = mla_absorb_q(q, dense[0])[:, :, :512], mla_bmm_w4(q, wk, sk)
    e, f = mla_project_out(o, dense[1]), mla_bmm_w4(o, wv, sv)
    for p, r, x, w in ((a, b, q, dense[0]), (e, f, o, dense[1])):
        mass = np.einsum("thk,hnk->thn", np.abs(to_np(x)), np.abs(to_np(w)))
        # two roundings to bf16 and two fp32 sums
        _within(p, to_np(r), np.abs(to_np(r)) * 2 * (BF16 + ARITH) + mass * 1024 * 2.0 ** -24, "products")
