"""A smaller latent cache: ctypes binding of mla_kv_append_fp4 and mla_decode_fp4 (4-bit rows), mla_key_weights,
mla_select_keys and mla_compact_rows (rows kept by the attention they got).  Argument marshalling only, with the checks
and the stream rules of _step.
"""
from __future__ import annotations

import torch

from . import _lib
from ._lib import MLAError
from ._step import (_BF16, _E4M3, _F32, _I32, _INT_MAX, _U8, _call, _dense, _device, _empty, _on, _rows, _shape, _workspace)

FP4_ROW = 416     # bytes of a 4-bit cache row: 256 of codes, 32 scales, 64 RoPE columns in bf16


def _paged(kv_cache, block_table, dev, B):
    """num_pages, page_size and max_pages, with the addresses of the table."""
    pages, page, _ = _shape(kv_cache, "kv_cache", 3)
    max_pages = _shape(block_table, "block_table", 2)[1]
    if page > _INT_MAX or max_pages > _INT_MAX:
        raise MLAError(1, f"page size and max_pages must be below 2^31, got {page} and {max_pages}")
    return pages, page, max_pages, _dense(block_table, "block_table", _I32, dev, (B, max_pages))


def _scratch(nbytes, dev, stream):
    """The device's scratch buffer of mla_decode_fp4 and mla_key_weights.  It is not the attention's, whose kernels give up their
    waits while their word is set: a length that was cut is recorded in this one.  A new one is filled on the call's stream: in a
    capture the zeros are a node of the graph, which comes before the call's."""
    device = torch.device("cuda", dev)
    ws = _lib._scratch_cache.get(("cuda", dev))
    if ws is not None and ws.numel() >= nbytes:
        return ws
    if stream is None:
        return _lib.grown(_lib._scratch_cache, nbytes, device)
    with _on(stream, device):
        return _lib.grown(_lib._scratch_cache, nbytes, device)


def _query(q):
    """q as [B, s, H, 576], its device and whether it came as [B, H, 576]."""
    try:
        single = len(q.shape) == 3
    except AttributeError:
        raise MLAError(1, f"q must be a CUDA tensor, got {type(q).__name__}") from None
    q4 = q.unsqueeze(1) if single else q
    dev, (B, s, H, _) = _device(q4, "q", 4)
    if s < 1 or H < 1 or s * H > 1 << 20:
        raise MLAError(1, f"q must be [B, H, 576] or [B, q_per_req, H, 576] with 1 <= q_per_req * H <= 2^20, got {tuple(q.shape)}")
    return q4, dev, B, s, H, single


def _per_row(t, name, dtype, dev, B, s, H, tail, single):
    """The address of an [B, s, H, ..] tensor, or [B, H, ..] of a single token."""
    if single and isinstance(t, torch.Tensor) and t.dim() == 2 + len(tail):
        return _dense(t, name, dtype, dev, (B, H) + tail)
    return _dense(t, name, dtype, dev, (B, s, H) + tail)


def mla_kv_append_fp4(c_kv, k_pe, slots, positions, cos_sin, kv_cache, kv_scale: float = 1.0, norm_weight=None,
                      eps: float = 1e-6, q_pe=None, q_out=None, kv_out=None, is_neox: bool = False, ws=None, stream=None):
    """mla_kv_append into a 4-bit cache, uint8 [pages,page,416]: e2m1 codes of the latent with an e4m3 scale for
    16 columns, the turned k_pe in bf16, both of row / kv_scale.  Arguments otherwise as mla_kv_append (kv_out: the
    rows in bf16, before the 4 bits).  Returns q_out, kv_out."""
    dev, (T, _) = _device(c_kv, "c_kv", 2)
    pages, page, _ = _shape(kv_cache, "kv_cache", 3)
    pc = _rows(c_kv, "c_kv", _BF16, dev, (T, 512))
    pk = _rows(k_pe, "k_pe", _BF16, dev, (T, 64))
    pcache = _dense(kv_cache, "kv_cache", _U8, dev, (pages, page, FP4_ROW))
    max_pos = _shape(cos_sin, "cos_sin", 2)[0]
    if page > _INT_MAX or max_pos > _INT_MAX:
        raise MLAError(1, f"page size and max_pos must be below 2^31, got {page} and {max_pos}")
    pcs = _dense(cos_sin, "cos_sin", _F32, dev, (max_pos, 64))
    pw = None if norm_weight is None else _dense(norm_weight, "norm_weight", _BF16, dev, (512,))
    pq = pqo = pkv = None
    H = qt = qh = ot = oh = st = 0
    if q_pe is not None:
        H = _shape(q_pe, "q_pe", 3)[1]
        if not 1 <= H <= _INT_MAX:
            raise MLAError(1, f"q_pe must have between 1 and 2^31 - 1 heads (H), got {H}")
        if q_out is None:
            q_out = _empty((T, H, 576), _BF16, dev, stream)
        pq, pqo = _rows(q_pe, "q_pe", _BF16, dev, (T, H, 64)), _rows(q_out, "q_out", _BF16, dev, (T, H, 576))
        (qt, qh, _), (ot, oh, _) = q_pe.stride(), q_out.stride()
    elif q_out is not None:
        raise MLAError(1, "q_out goes with q_pe")
    if kv_out is not None:
        pkv, st = _rows(kv_out, "kv_out", _BF16, dev, (T, 576)), kv_out.stride(0)
    _call("mla_kv_append_fp4", dev, stream, pc, c_kv.stride(0), pk, k_pe.stride(0), pw, float(eps), pq, qt, qh,
          _dense(positions, "positions", _I32, dev, (T,)), _dense(slots, "slots", _I32, dev, (T,)), pcs, max_pos,
          int(bool(is_neox)), T, H, pcache, float(kv_scale), pages, page, pqo, ot, oh, pkv, st, *_workspace(ws, dev))
    return q_out, kv_out


def mla_decode_fp4(q, kv_cache_fp4, kv_scale: float, block_table, lens, scale: float, sinks=None, num_splits: int = 0,
                   out=None, lse=None, ws=None, stream=None):
    """Decode over a 4-bit latent cache (uint8 [pages,page,416], see mla_kv_append_fp4).  q bf16 [B,H,576] or
    [B,s,H,576]; sinks fp32 [H].  Returns out, lse shaped like mla_decode / mla_decode_ex."""
    q4, dev, B, s, H, single = _query(q)
    pq = _dense(q4, "q", _BF16, dev, (B, s, H, 576))
    pages, page, max_pages, pt = _paged(kv_cache_fp4, block_table, dev, B)
    pc = _dense(kv_cache_fp4, "kv_cache_fp4", _U8, dev, (pages, page, FP4_ROW))
    pl = _dense(lens, "lens", _I32, dev, (B,))
    ps = None if sinks is None else _dense(sinks, "sinks", _F32, dev, (H,))
    if out is None:
        out = _empty((B, H, 512) if single else (B, s, H, 512), _BF16, dev, stream)
    if lse is None:
        lse = _empty((B, H) if single else (B, s, H), _F32, dev, stream)
    po = _per_row(out, "out", _BF16, dev, B, s, H, (512,), single)
    pe = _per_row(lse, "lse", _F32, dev, B, s, H, (), single)
    num_splits = int(num_splits)
    if not 0 <= num_splits <= 65535:
        raise MLAError(1, f"num_splits must be between 0 and 65535, got {num_splits}")
    if ws is None:
        ws = _scratch(_lib.lib().mla_decode_fp4_workspace_size(B, s, H, num_splits), dev, stream)
    _call("mla_decode_fp4", dev, stream, pq, s, pc, float(kv_scale), pages, page, pt, max_pages, pl, B, H, float(scale), ps,
          num_splits, po, pe, *_workspace(ws, dev))
    if single:
        return out if out.dim() == 3 else out[:, 0], lse if lse.dim() == 2 else lse[:, 0]
    return out, lse


def mla_key_weights(q, lse, kv_cache, block_table, lens, scale: float, weights, kv_scale: float = 1.0, decay: float = 1.0,
                    ws=None, stream=None):
    """weights[b, j] = decay * weights[b, j] + the attention that key j of request b got from the tokens of q, added up over
    tokens and heads; in place, for j < lens[b].  q bf16 [B,H,576] or [B,s,H,576] and lse as the decode over the same
    keys took and gave them; kv_cache [pages,page,576] in bf16 or e4m3, or uint8 [pages,page,416] (4-bit rows);
    weights fp32 [B,W] (rows may be strided).  Returns weights."""
    q4, dev, B, s, H, single = _query(q)
    pq = _dense(q4, "q", _BF16, dev, (B, s, H, 576))
    pe = _per_row(lse, "lse", _F32, dev, B, s, H, (), single)
    pages, page, max_pages, pt = _paged(kv_cache, block_table, dev, B)
    dtype = kv_cache.dtype
    fmt = {_BF16: 0, _E4M3: 1, _U8: 2}.get(dtype)
    if fmt is None:
        raise MLAError(1, f"kv_cache must be bf16, e4m3 or uint8 (4-bit rows), got {dtype}")
    pc = _dense(kv_cache, "kv_cache", dtype, dev, (pages, page, FP4_ROW if fmt == 2 else 576))
    width = _shape(weights, "weights", 2)[1]
    if width > _INT_MAX:
        raise MLAError(1, f"weights has too many columns ({width})")
    pw = _rows(weights, "weights", _F32, dev, (B, width))
    if ws is None and s * H > 128:
        ws = _scratch(_lib.lib().mla_key_weights_workspace_size(B, s, H, width), dev, stream)
    _call("mla_key_weights", dev, stream, pq, s, pe, pc, fmt, float(kv_scale), pages, page, pt, max_pages,
          _dense(lens, "lens", _I32, dev, (B,)), B, H, float(scale), float(decay), pw, weights.stride(0), width,
          *_workspace(ws, dev))
    return weights


def mla_select_keys(weights, lens, keep, K: int, first: int = 0, recent: int = 0, idx=None, count=None, dropped=None, ws=None,
                    stream=None):
    """The rows that stay of requests with lens[b] rows and a budget of keep[b] (int32 [B]) of at most K: the first `first`, the
    last `recent` and those with the largest weights [B,W] (fp32, rows may be strided).  Returns idx int32 [B,K]
    (ascending, -1 behind the last), count [B] and dropped [B] = count - lens (what mla_slot_map takes as new_tokens)."""
    dev, (B, width) = _device(weights, "weights", 2)
    K, first, recent = int(K), int(first), int(recent)
    if not 0 <= K <= _INT_MAX - 65536 or width > _INT_MAX - 65536:
        raise MLAError(1, f"K must be between 0 and 2^31 - 2^16 and weights at most that wide, got {K} and {width}")
    if not 0 <= first <= _INT_MAX or not 0 <= recent <= _INT_MAX:
        raise MLAError(1, f"first and recent must be between 0 and 2^31 - 1, got {first} and {recent}")
    pw = _rows(weights, "weights", _F32, dev, (B, width))
    if idx is None:
        idx = _empty((B, K), _I32, dev, stream)
    if count is None:
        count = _empty(B, _I32, dev, stream)
    if dropped is None:
        dropped = _empty(B, _I32, dev, stream)
    _call("mla_select_keys", dev, stream, pw, weights.stride(0), width, _dense(lens, "lens", _I32, dev, (B,)),
          _dense(keep, "keep", _I32, dev, (B,)), first, recent, B, K, _dense(idx, "idx", _I32, dev, (B, K)),
          _dense(count, "count", _I32, dev, (B,)), _dense(dropped, "dropped", _I32, dev, (B,)), *_workspace(ws, dev))
    return idx, count, dropped


def mla_compact_rows(kv_cache, block_table, idx, count, weights=None, ws=None, stream=None):
    """Row i of request b becomes its row idx[b, i] (i < count[b]), in place in kv_cache [pages,page,row] (any type, rows of a
    multiple of 16 bytes) and, if given, in weights fp32 [B,W].  idx as mla_select_keys gives it.  Weights behind count are the old
    rows' still: set them to 0 before new tokens come there."""
    dev, (B, K) = _device(idx, "idx", 2)
    pages, page, max_pages, pt = _paged(kv_cache, block_table, dev, B)
    row = kv_cache.shape[2] * kv_cache.element_size()
    if row > 65536 or row < 16 or row % 16:
        raise MLAError(1, f"rows of kv_cache must have a multiple of 16 bytes up to 65536, got {row}")
    if K > _INT_MAX:
        raise MLAError(1, f"idx has too many columns ({K})")
    pc = _dense(kv_cache, "kv_cache", kv_cache.dtype, dev, tuple(kv_cache.shape))
    pw, st, width = None, 0, 0
    if weights is not None:
        width = _shape(weights, "weights", 2)[1]
        if width > _INT_MAX:
            raise MLAError(1, f"weights has too many columns ({width})")
        pw, st = _rows(weights, "weights", _F32, dev, (B, width)), weights.stride(0)
    _call("mla_compact_rows", dev, stream, pc, row, pages, page, pt, max_pages, _dense(idx, "idx", _I32, dev, (B, K)), K,
          _dense(count, "count", _I32, dev, (B,)), B, pw, st, width, *_workspace(ws, dev))
