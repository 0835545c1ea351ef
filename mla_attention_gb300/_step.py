"""The serving step around the latent attention: ctypes binding of mla_slot_map, mla_rms_norm,
mla_kv_append and mla_bmm_w4 (argument marshalling only, as in _lib).

A decode step makes hundreds of these calls, most of them a few microseconds long on the GPU, so the
host's part is kept short: one expression checks a tensor, and only a tensor that fails it is looked at
for what is wrong.  A call is issued on `stream` or on the current stream of the tensors' device,
whichever device is current.  The first call on a device that takes a workspace allocates the status word's
buffer: make it before any stream capture.
"""
from __future__ import annotations

import torch

from . import _lib
from ._lib import MLAError, _check

_BF16, _I32, _F32, _E4M3, _U8 = torch.bfloat16, torch.int32, torch.float32, torch.float8_e4m3fn, torch.uint8
_INT_MAX = 2 ** 31 - 1
# the handle alone: torch.cuda.current_stream() builds a Stream, 2 us (a torch without CUDA has none, and no tensor that asks for it)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _dense(t, name, dtype, dev, shape):
    """The address of a contiguous tensor of this type, device and shape."""
    try:
        if t.dtype is dtype and t.is_contiguous() and t.get_device() == dev and t.shape == shape:
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, dtype, dev, shape)
    raise MLAError(1, f"{name} must be contiguous")


def _rows(t, name, dtype, dev, shape):
    """The same with free strides but for a contiguous last dimension."""
    try:
        if t.dtype is dtype and t.get_device() == dev and t.shape == shape and (t.is_contiguous() or t.stride(-1) == 1):
            return t.data_ptr()
    except AttributeError:
        pass
    _refuse(t, name, dtype, dev, shape)
    if shape[-1] > 1:
        raise MLAError(1, f"{name} needs a contiguous last dimension")
    return t.data_ptr()


def _refuse(t, name, dtype, dev, shape):
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype:
        raise MLAError(1, f"{name} must be a torch.Tensor of {dtype}, got {getattr(t, 'dtype', type(t).__name__)}")
    if t.get_device() != dev:
        raise MLAError(1, f"{name} is on {t.device}, expected cuda:{dev}")
    if t.shape != shape:
        raise MLAError(1, f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _device(t, name, dims):
    """The index of the GPU that holds t, and t's shape."""
    try:
        dev, shape = t.get_device(), t.shape
    except AttributeError:
        raise MLAError(1, f"{name} must be a CUDA tensor, got {type(t).__name__}") from None
    if dev < 0:
        raise MLAError(1, f"{name} must be a CUDA tensor")
    if len(shape) != dims:
        raise MLAError(1, f"{name} must have {dims} dimensions, got {len(shape)}")
    if shape[0] > _INT_MAX:
        raise MLAError(1, f"{name} has too many rows ({shape[0]})")
    return dev, shape


def _shape(t, name, dims):
    try:
        shape = t.shape
    except AttributeError:
        raise MLAError(1, f"{name} must be a torch.Tensor, got {type(t).__name__}") from None
    if len(shape) != dims:
        raise MLAError(1, f"{name} must have {dims} dimensions, got {len(shape)}")
    return shape


def _empty(shape, dtype, dev, stream):
    """An output in the memory of the stream that writes it, as under torch.cuda.stream(stream)."""
    device = torch.device("cuda", dev)
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        handle = int(getattr(stream, "cuda_stream", stream))
        stream = torch.cuda.ExternalStream(handle, device) if handle else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _workspace(ws, dev):
    """Address and size of the status word's buffer: the caller's, or the device's own for these calls.  It is not
    the attention's, whose kernels give up their waits while their word is set: a refused request of
    mla_slot_map is an everyday answer."""
    if ws is None:
        ws = _lib._status_cache.get(dev)
        if ws is None:
            if torch.cuda.is_current_stream_capturing():
                raise MLAError(1, "the first call on a device without a ws allocates the status word: make it before a capture")
            ws = torch.zeros(256, dtype=_U8, device=torch.device("cuda", dev))
            torch.cuda.current_stream(dev).synchronize()   # the call may be issued on another stream
            ws = _lib._status_cache.setdefault(dev, ws)    # of two threads' first calls one buffer stays, and both use it
    elif not isinstance(ws, torch.Tensor) or ws.get_device() != dev or not ws.is_contiguous():
        raise MLAError(1, f"ws must be a contiguous tensor on cuda:{dev}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


_functions = {}
_several_devices = None


def _call(name, dev, stream, *args):
    global _several_devices
    fn = _functions.get(name)
    if fn is None:
        _several_devices = torch.cuda.device_count() > 1    # before the function: a thread that finds that goes by it
        fn = _functions[name] = getattr(_lib.lib(), name)
    if stream is None:
        stream = _current_stream(dev)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    if _several_devices and dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    else:
        status = fn(*args, stream)
    if status:
        _check(status)


def mla_slot_map(lens, new_tokens, block_table, pool, pool_state, page_size: int, N: int, positions=None, slots=None,
                 cu_tokens=None, lens_out=None, pool_state_out=None, ws=None, stream=None):
    """Page tables, positions and slots of a step's tokens: lens, new_tokens int32 [B] (negative: tokens
    dropped), block_table int32 [B,max_pages] and pool int32 [num_pages] in place, pool_state int32 [2]
    (ring head, free pages).  Rows behind the last token get -1.  lens_out / pool_state_out may be
    lens / pool_state.  Returns positions [N], slots [N], cu_tokens [B+1], lens_out, pool_state_out."""
    dev, (B,) = _device(lens, "lens", 1)
    max_pages, num_pages, N, page_size = _shape(block_table, "block_table", 2)[1], _shape(pool, "pool", 1)[0], int(N), int(page_size)
    if not 0 <= N <= _INT_MAX:
        raise MLAError(1, f"N must be between 0 and 2^31 - 1, got {N}")
    if not 1 <= page_size <= _INT_MAX or max_pages > _INT_MAX:
        raise MLAError(1, f"page_size must be between 1 and 2^31 - 1 and max_pages at most that, got {page_size} and {max_pages}")
    if positions is None:
        positions = _empty(N, _I32, dev, stream)
    if slots is None:
        slots = _empty(N, _I32, dev, stream)
    if cu_tokens is None:
        cu_tokens = _empty(B + 1, _I32, dev, stream)
    if lens_out is None:
        lens_out = _empty(B, _I32, dev, stream)
    if pool_state_out is None:
        pool_state_out = _empty(2, _I32, dev, stream)
    _call("mla_slot_map", dev, stream, _dense(lens, "lens", _I32, dev, (B,)),
          _dense(new_tokens, "new_tokens", _I32, dev, (B,)), B,
          _dense(block_table, "block_table", _I32, dev, (B, max_pages)), max_pages, page_size, num_pages,
          _dense(pool, "pool", _I32, dev, (num_pages,)), _dense(pool_state, "pool_state", _I32, dev, (2,)), N,
          _dense(cu_tokens, "cu_tokens", _I32, dev, (B + 1,)), _dense(positions, "positions", _I32, dev, (N,)),
          _dense(slots, "slots", _I32, dev, (N,)), _dense(lens_out, "lens_out", _I32, dev, (B,)),
          _dense(pool_state_out, "pool_state_out", _I32, dev, (2,)), *_workspace(ws, dev))
    return positions, slots, cu_tokens, lens_out, pool_state_out


def mla_rms_norm(x, weight, eps: float = 1e-6, residual=None, residual_out=None, out=None, e4m3: bool = False,
                 group: int = 0, scales=None, stream=None):
    """y = h / sqrt(mean(h^2) + eps) * weight with h = x (+ residual); x, residual bf16 [T,D] rows.
    Returns out, residual_out, scales: out bf16, or e4m3 (e4m3=True or an e4m3 `out`) with fp32 scales
    [T, D / group] ([T, 1] with group 0); residual_out = h in bf16 (None without a residual; may be
    the residual itself); scales None with a bf16 out."""
    dev, (T, D) = _device(x, "x", 2)
    if D > _INT_MAX:
        raise MLAError(2, f"D is far above the 32768 that a row may have (got {D})")
    if out is None:
        e4m3 = bool(e4m3)
    elif e4m3 and getattr(out, "dtype", None) is not _E4M3:
        raise MLAError(1, f"out must be a torch.Tensor of {_E4M3} with e4m3")
    else:
        e4m3 = getattr(out, "dtype", None) is _E4M3
    group = int(group)
    if group and (not e4m3 or group not in (32, 64, 128) or D % group):
        raise MLAError(1, f"group must be 0, or with e4m3 32, 64 or 128 dividing D (got {group}, D = {D})")
    if out is None:
        out = _empty((T, D), _E4M3 if e4m3 else _BF16, dev, stream)
    px = _rows(x, "x", _BF16, dev, (T, D))
    pw = _dense(weight, "weight", _BF16, dev, (D,))
    po = _rows(out, "out", _E4M3 if e4m3 else _BF16, dev, (T, D))
    pr = pro = ps = None
    sr = sro = 0
    if residual is not None:
        if residual_out is None:
            residual_out = _empty((T, D), _BF16, dev, stream)
        pr, pro = _rows(residual, "residual", _BF16, dev, (T, D)), _rows(residual_out, "residual_out", _BF16, dev, (T, D))
        sr, sro = residual.stride(0), residual_out.stride(0)
    elif residual_out is not None:
        raise MLAError(1, "residual_out goes with a residual")
    if e4m3:
        shape = (T, D // group if group else 1)
        if scales is None:
            scales = _empty(shape, _F32, dev, stream)
        ps = _dense(scales, "scales", _F32, dev, shape)
    elif scales is not None:
        raise MLAError(1, "scales go with an e4m3 output")
    _call("mla_rms_norm", dev, stream, px, x.stride(0), pr, sr, pw, float(eps), T, D, pro, sro, int(e4m3), group, po,
          out.stride(0), ps)
    return out, residual_out, scales


def mla_kv_append(c_kv, k_pe, slots, positions, cos_sin, kv_cache, kv_scale: float = 1.0, norm_weight=None,
                  eps: float = 1e-6, q_pe=None, q_out=None, kv_out=None, is_neox: bool = False, ws=None, stream=None):
    """Cache rows by slot: [norm(c_kv) * norm_weight | turned k_pe] of tokens [T] into kv_cache [pages,page,576]
    (bf16, or e4m3 of row / kv_scale) in place at rows slots[t]; the turned q_pe [T,H,64] into
    q_out[:, :, 512:576]; kv_out [T,576] (if given) the rows in bf16.  positions[t] = -1: no token;
    slots[t] = -1: no cache row.  Returns q_out, kv_out."""
    dev, (T, _) = _device(c_kv, "c_kv", 2)
    pages, page, _ = _shape(kv_cache, "kv_cache", 3)
    e4m3 = kv_cache.dtype is _E4M3
    pc = _rows(c_kv, "c_kv", _BF16, dev, (T, 512))
    pk = _rows(k_pe, "k_pe", _BF16, dev, (T, 64))
    pcache = _dense(kv_cache, "kv_cache", _E4M3 if e4m3 else _BF16, dev, (pages, page, 576))
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
    _call("mla_kv_append", dev, stream, pc, c_kv.stride(0), pk, k_pe.stride(0), pw, float(eps), pq, qt, qh,
          _dense(positions, "positions", _I32, dev, (T,)), _dense(slots, "slots", _I32, dev, (T,)), pcs, max_pos,
          int(bool(is_neox)), T, H, pcache, int(e4m3), float(kv_scale), pages, page, pqo, ot, oh, pkv, st,
          *_workspace(ws, dev))
    return q_out, kv_out


def mla_bmm_w4(x, w4, scales, out=None, ws=None, stream=None):
    """out[t, h, n] = sum_k x[t, h, k] (code[h, n, k] - 8) scales[h, n, k // group]: x bf16 [T,H,K], w4 uint8
    [H,N,K/2] (byte j of a row: code 2j low, 2j+1 high), scales bf16 or fp32 [H,N,K/group], group 32, 64 or
    128 -> bf16 [T,H,N] (a strided `out` is fine)."""
    dev, (T, H, K) = _device(x, "x", 3)
    N, groups = _shape(w4, "w4", 3)[1], _shape(scales, "scales", 3)[2]
    if H > _INT_MAX or N > _INT_MAX or K > _INT_MAX:
        raise MLAError(1, f"H, N and K must be below 2^31, got {H}, {N}, {K}")
    if groups < 1 or K % groups or K // groups not in (32, 64, 128):
        raise MLAError(1, f"scales must have K / group columns, group 32, 64 or 128 (got {groups}, K = {K})")
    f32 = scales.dtype is _F32
    px = _rows(x, "x", _BF16, dev, (T, H, K))
    pw = _dense(w4, "w4", _U8, dev, (H, N, K // 2))
    ps = _dense(scales, "scales", _F32 if f32 else _BF16, dev, (H, N, groups))
    if out is None:
        out = _empty((T, H, N), _BF16, dev, stream)
    po = _rows(out, "out", _BF16, dev, (T, H, N))
    (xt, xh, _), (ot, oh, _) = x.stride(), out.stride()
    _call("mla_bmm_w4", dev, stream, px, xt, xh, pw, ps, int(f32), K // groups, T, H, N, K, po,
          ot, oh, *_workspace(ws, dev))
    return out
