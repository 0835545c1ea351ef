"""fp64 oracle of the smaller cache (test infrastructure only): 4-bit rows, decode over them, the keys' attention weights, the
choice of the rows that stay and their move, written from the definitions in include/mla.h with plain loops and numpy;
none of it is shared with the CUDA path."""
import numpy as np

from .step_oracle import kv_append, round_e4m3

__all__ = ["round_e2m1", "quantise_fp4", "fp4_rows", "fp4_values", "kv_append_fp4", "held_rows", "decode", "key_weights", "select_keys",
           "compact_rows"]

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def round_e2m1(v):
    """The code (0..15) of the nearest e2m1 value, of two equally near ones the even code, saturating."""
    v = np.asarray(v, np.float64)
    a = np.abs(v)
    code = np.zeros(v.shape, np.int64)
    for c in range(1, 8):
        border = (E2M1[c - 1] + E2M1[c]) / 2
        code = np.where((a > border) | ((a == border) & (c % 2 == 0)), c, code)
    return code + 8 * np.signbit(v)


def quantise_fp4(lat, kv_scale):
    """Codes [T, 512] and scales [T, 32] (their values) of unrounded latents."""
    v = np.asarray(lat, np.float64).reshape(len(lat), 32, 16) / kv_scale
    top = np.max(np.abs(v), axis=2)                             # np.max keeps a NaN
    scale = round_e4m3(np.minimum(np.maximum(top / 6, 2.0 ** -9), 448))
    with np.errstate(invalid="ignore"):
        code = round_e2m1(v / scale[:, :, None])
    return code.reshape(len(lat), 512), scale


def _e4m3_bytes(values):
    """The bytes of e4m3 values."""
    out = np.zeros(np.shape(values), np.uint8)
    for at, v in np.ndenumerate(values):
        if np.isnan(v):
            out[at] = 0x7F
            continue
        a = abs(v)
        e = max(int(np.floor(np.log2(a))), -6) if a > 0 else -6
        m = int(round(a / 2.0 ** (e - 3)))
        out[at] = (m if m < 8 else (e + 7) * 8 + (m - 8)) | (128 if np.signbit(v) else 0)
    return out


def fp4_rows(code, scale, pe_bits):
    """Rows of 416 bytes from codes [T, 512], scale values [T, 32] and the RoPE columns' bf16 bits [T, 64]."""
    code = np.asarray(code).astype(np.uint8)
    pe = np.ascontiguousarray(np.asarray(pe_bits).astype("<u2")).view(np.uint8).reshape(len(code), 128)
    return np.concatenate([code[:, 0::2] | (code[:, 1::2] << 4), _e4m3_bytes(scale), pe], 1)


def fp4_values(rows):
    """What rows of 416 bytes stand for, [.., 576], without kv_scale."""
    rows = np.asarray(rows, np.uint8)
    lead = rows.shape[:-1]
    rows = rows.reshape(-1, 416)
    code = np.empty((len(rows), 512), np.int64)
    code[:, 0::2], code[:, 1::2] = rows[:, :256] & 15, rows[:, :256] >> 4
    lat = np.where(code >= 8, -1.0, 1.0) * E2M1[code & 7]
    b = rows[:, 256:288].astype(np.int64)
    e, m = (b >> 3) & 15, b & 7
    s = np.where(e == 0, m * 2.0 ** -9, (1 + m / 8) * 2.0 ** (e - 7.0))
    s = np.where(b >= 128, -s, s)
    s = np.where((b & 127) == 127, np.nan, s)
    lat = lat * np.repeat(s, 16, axis=1)
    bits = np.ascontiguousarray(rows[:, 288:]).view("<u2").astype(np.uint32) << 16
    pe = bits.view(np.float32).astype(np.float64)
    return np.concatenate([lat, pe], 1).reshape(lead + (576,))


def kv_append_fp4(c_kv, k_pe, positions, cos_sin, kv_scale, norm_weight=None, eps=1e-6, q_pe=None, neox=False):
    """Codes, scales and unrounded RoPE columns / kv_scale of the tokens' rows, the unrounded rows, the turned queries."""
    rows, q = kv_append(c_kv, k_pe, positions, cos_sin, norm_weight, eps, q_pe, neox)
    code, scale = quantise_fp4(rows[:, :512], kv_scale)
    return code, scale, rows[:, 512:] / kv_scale, rows, q


def held_rows(cache, block_table, lens, b):
    """The cached rows of request b in order, through its pages."""
    page = cache.shape[1]
    return np.array([cache[block_table[b][j // page], j % page] for j in range(int(lens[b]))]).reshape(int(lens[b]), cache.shape[2])


def decode(q, keys, scale, sinks=None):
    """q [B, s, H, 576] over keys[b] [len, 576]: out [B, s, H, 512], lse [B, s, H]."""
    B, s, H, _ = q.shape
    out, lse = np.zeros((B, s, H, 512)), np.full((B, s, H), -np.inf)
    for b in range(B):
        for i in range(s):
            k = keys[b][:max(0, len(keys[b]) - s + 1 + i)]
            for h in range(H):
                score = scale * (k @ q[b, i, h])
                all_scores = score if sinks is None else np.append(score, sinks[h])
                if len(all_scores) == 0:
                    continue
                top = all_scores.max()
                if top == -np.inf:
                    continue
                total = np.exp(all_scores - top).sum()
                lse[b, i, h] = top + np.log(total)
                out[b, i, h] = np.exp(score - top) @ k[:, :512] / total
    return out, lse


def key_weights(q, lse, keys, scale, weights, decay):
    """weights [B, width] after the call (a new array)."""
    w = np.array(weights, np.float64)
    B, s, H, _ = q.shape
    for b in range(B):
        n = len(keys[b])
        w[b, :n] = decay * w[b, :n] if decay else 0.0
        for i in range(s):
            seen = max(0, n - s + 1 + i)
            for h in range(H):
                if lse[b, i, h] != -np.inf:
                    w[b, :seen] += np.exp(scale * (keys[b][:seen] @ q[b, i, h]) - lse[b, i, h])
    return w


def select_keys(weights, lens, keep, K, first, recent):
    B = len(lens)
    idx, count, dropped = np.full((B, K), -1, np.int64), np.zeros(B, np.int64), np.zeros(B, np.int64)
    bad = []
    for b in range(B):
        n = min(int(lens[b]), int(keep[b]))
        if lens[b] < 0 or lens[b] > weights.shape[1] or keep[b] < 0 or n > K:
            bad.append(b)
            continue
        last = min(recent, n)
        head = min(first, n - last)
        stay = set(range(head)) | set(range(int(lens[b]) - last, int(lens[b])))
        rest = [j for j in range(int(lens[b])) if j not in stay]
        rest.sort(key=lambda j: (-np.inf if np.isnan(weights[b, j]) else -float(weights[b, j]), not np.isnan(weights[b, j]), j))
        stay |= set(rest[:n - len(stay)])
        idx[b, :n] = sorted(stay)
        count[b], dropped[b] = n, n - int(lens[b])
    return idx, count, dropped, bad


def compact_rows(cache, block_table, idx, count, weights=None):
    """cache [pages, page, ..] and weights after the moves (new arrays)."""
    cache = np.array(cache)
    w = None if weights is None else np.array(weights)
    page = cache.shape[1]
    for b in range(len(count)):
        for i in range(int(count[b])):                 # ascending: a source is never behind what was written
            j = int(idx[b][i])
            cache[block_table[b][i // page], i % page] = cache[block_table[b][j // page], j % page]
            if w is not None:
                w[b, i] = w[b, j]
    return cache, w
