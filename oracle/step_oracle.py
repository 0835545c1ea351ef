"""fp64 oracle of the serving step's operators (test infrastructure only): the slot map, the RMS
norm, the cache append by slots and the products with 4-bit weights, written from the definitions
in include/mla.h with plain loops and numpy; none of it is shared with the CUDA path."""
import numpy as np

__all__ = ["slot_map", "rms_norm", "kv_append", "bmm_w4", "round_e4m3", "unpack_w4"]

E4M3_MAX = 448.0


def round_e4m3(v):
    """Nearest e4m3 value (ties to even), saturating at +-448; NaN stays NaN."""
    v = np.asarray(v, dtype=np.float64)
    a = np.minimum(np.abs(v), E4M3_MAX)
    with np.errstate(invalid="ignore"):
        step = 2.0 ** (np.floor(np.log2(np.maximum(a, 2.0 ** -6))) - 3)
    return np.where(np.isnan(v), np.nan, np.copysign(np.rint(a / step) * step, v))


def slot_map(lens, new_tokens, block_table, pool, pool_state, page_size, N):
    """One step, request by request.  Returns positions, slots, cu_tokens, lens_out, pool_state_out,
    block_table, pool (new arrays) and the set of refusals seen (the details' low bytes)."""
    block_table, pool = np.asarray(block_table), np.asarray(pool)
    lens, new_tokens = [int(v) for v in lens], [int(v) for v in new_tokens]
    table, ring = np.array(block_table, dtype=np.int64), np.array(pool, dtype=np.int64)
    old_table, old_ring = table.copy(), ring.copy()
    B, P = len(lens), len(ring)
    cap = min(table.shape[1] * page_size, 2 ** 31 - 1)
    head, count = int(pool_state[0]), int(pool_state[1])
    why = set()
    pool_ok = 0 <= count <= P and (0 <= head < P or head == P == 0)
    if not pool_ok:
        why.add(0x74)
    room = count if pool_ok else 0
    positions, slots = np.full(N, -1, np.int64), np.full(N, -1, np.int64)
    cu, lens_out = [0], list(lens)
    tok = want_pop = want_put = popped = returned = 0
    for b in range(B):
        n, now = new_tokens[b], max(0, lens[b] + new_tokens[b])
        add = max(n, 0)
        tok += add
        cu.append(min(tok, N))
        if not 0 <= lens[b] <= cap or now > cap:
            why.add(0x70)
            continue
        have, need = -(-lens[b] // page_size), -(-now // page_size)
        grow, drop = max(need - have, 0), max(have - need, 0)
        want_pop += grow
        want_put += drop
        bad = None
        if add and tok > N:
            bad = 0x72
        if grow and want_pop > room:
            bad = 0x71
        if drop and (not pool_ok or count + want_put > P):
            bad = 0x73
        if bad:
            why.add(bad)
            continue
        lens_out[b] = now
        for i in range(grow):
            page = int(old_ring[(head + want_pop - grow + i) % P])
            if not 0 <= page < P:
                why.add(0x75)
                page = -1
            table[b, have + i] = page
        for i in range(drop):
            page = int(old_table[b, need + i])
            if not 0 <= page < P:
                why.add(0x75)
                page = -1
            ring[(head + count + want_put - drop + i) % P] = page
        popped = want_pop if grow else popped
        returned = want_put if drop else returned
        for i in range(add):
            pos, row = lens[b] + i, tok - add + i
            page = int(table[b, pos // page_size])
            positions[row] = pos
            if 0 <= page < P:
                slots[row] = page * page_size + pos % page_size
            else:
                why.add(0x75)
    state = [(head + popped) % P if P else 0, count - popped + returned] if pool_ok else [head, count]
    return positions, slots, np.array(cu), np.array(lens_out, dtype=np.int64), np.array(state), table, ring, why


def rms_norm(x, weight, eps, residual=None, group=None):
    """y (unrounded), h, and with `group` (0: the row) the scales and the e4m3 values of y / scale."""
    h = np.asarray(x, np.float64) + (0 if residual is None else np.asarray(residual, np.float64))
    with np.errstate(invalid="ignore", divide="ignore"):
        y = h / np.sqrt(np.mean(h * h, axis=1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    if group is None:
        return y, h
    T, D = y.shape
    parts = y.reshape(T, -1, group or D)
    scale = np.maximum(np.abs(parts).max(-1) / E4M3_MAX, 2.0 ** -126)   # np.maximum keeps a NaN
    return y, h, scale, round_e4m3(parts / scale[..., None]).reshape(T, D)


def _turn(x, cs, neox):
    x, out = np.asarray(x, np.float64), np.empty(np.shape(x))
    for i in range(32):
        j, k = (i, i + 32) if neox else (2 * i, 2 * i + 1)
        c, s = cs[..., i], cs[..., 32 + i]
        out[..., j] = x[..., j] * c - x[..., k] * s
        out[..., k] = x[..., j] * s + x[..., k] * c
    return out


def kv_append(c_kv, k_pe, positions, cos_sin, norm_weight=None, eps=1e-6, q_pe=None, neox=False):
    """The unrounded rows [T, 576] and turned queries [T, H, 64] (or None) of tokens at valid positions."""
    lat = np.asarray(c_kv, np.float64)
    if norm_weight is not None:
        lat = rms_norm(lat, norm_weight, eps)[0]
    cs = np.asarray(cos_sin, np.float64)[np.asarray(positions)]
    rows = np.concatenate([lat, _turn(k_pe, cs, neox)], 1)
    return rows, None if q_pe is None else _turn(q_pe, cs[:, None, :], neox)


def unpack_w4(w4, scales):
    """[H, N, K] weights from packed bytes [H, N, K/2] and scales [H, N, K/group]."""
    w4, scales = np.asarray(w4).astype(np.int64), np.asarray(scales, np.float64)
    H, N, half = w4.shape
    w = np.empty((H, N, 2 * half))
    w[..., 0::2], w[..., 1::2] = (w4 & 15) - 8, (w4 >> 4) - 8
    return w * np.repeat(scales, 2 * half // scales.shape[2], axis=2)


def bmm_w4(x, w4, scales):
    """out [T, H, N] and the sum of |terms| behind each value."""
    w, x = unpack_w4(w4, scales), np.asarray(x, np.float64)
    return np.einsum("thk,hnk->thn", x, w), np.einsum("thk,hnk->thn", np.abs(x), np.abs(w))
