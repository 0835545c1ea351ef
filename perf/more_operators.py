"""A latent cache made smaller, in bits and in rows, as measured cases.

Five operators (include/mla.h has their definitions):

* append:  mla_kv_append_fp4  latent norm, RoPE and the write of 4-bit cache rows by slot
* decode:  mla_decode_fp4     attention of a request's last tokens over a 4-bit latent cache
* weights: mla_key_weights    how much attention each cached key got, added up over heads and query tokens
* select:  mla_select_keys    which rows of each request stay: the first ones, the last ones and the heaviest
* compact: mla_compact_rows   the kept rows moved to the front of their request, in place, in a paged cache

A row of the 4-bit cache has 416 bytes: 256 of e2m1 codes (column 2j in the low half of byte j), 32 e4m3 scales, one for
16 columns, and 64 RoPE columns in bf16.  `run` computes each operator in plain torch or, where `own` is true, by the
library's call.  `exact` follows the definitions in 64 bits.
"""
import torch

own = False

DEV = "cuda"
LATENT, ROPE, DK = 512, 64, 576
FP4_ROW, CODES, SCALES = 416, 256, 32
ROW_BYTES = dict(bf16=2 * DK, e4m3=DK, fp4=FP4_ROW)


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # a decode step's rows into the cache, a batch padded to its captured size
        dict(name="append-decode-64", op="append", T=64, H=128, page=64, neox=False, norm=True, rows_out=False, padded=9),
        # a prompt's rows into the cache and, as dense rows, for the prefill attention
        dict(name="append-prompt-8192", op="append", T=8192, H=128, page=64, neox=True, norm=True, rows_out=True, padded=0),
        # one request of a lone user: the latency of a step
        dict(name="decode-1", op="decode", B=1, s=1, H=128, page=64, lo=4097, hi=4097, sinks=False),
        # a small odd batch with two tokens a request, few heads on this GPU, small pages, sinks
        dict(name="decode-17x2-heads-16", op="decode", B=17, s=2, H=16, page=16, lo=1, hi=8191, sinks=True),
        # a decode batch of 64 requests at 4K..32K tokens
        dict(name="decode-64", op="decode", B=64, s=1, H=128, page=64, lo=4096, hi=32768, sinks=False),
        # the weights of a short request's keys after a step
        dict(name="weights-1-e4m3", op="weights", fmt="e4m3", B=1, s=1, H=40, page=32, lo=1533, hi=1533),
        # a decode batch's weights, added up step by step over a 16-bit cache
        dict(name="weights-64-bf16", op="weights", fmt="bf16", B=64, s=1, H=128, page=64, lo=4096, hi=32768),
        # the weights that a long prompt's last 32 tokens give, over a 4-bit cache
        dict(name="weights-prompt-32-fp4", op="weights", fmt="fp4", B=1, s=32, H=128, page=64, lo=32768, hi=32768),
        # one long request cut to a budget
        dict(name="select-1", op="select", B=1, lo=32767, hi=32767, keep=4096, first=4, recent=512),
        # a batch of 64 requests cut to half of its longest
        dict(name="select-64", op="select", B=64, lo=4096, hi=32768, keep=16384, first=4, recent=256),
        # one long request's rows in a 16-bit cache, two thirds stay, with their weights
        dict(name="compact-1-bf16", op="compact", fmt="bf16", B=1, page=64, lo=32767, hi=32767, keep=21845),
        # the rows of a batch of 64 requests in a 4-bit cache
        dict(name="compact-64-fp4", op="compact", fmt="fp4", B=64, page=64, lo=4096, hi=32768, keep=16384),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["append", "decode", "weights", "select", "compact"])
    page = rng.choice([16, 32, 64, 128])
    if op == "append":
        H = rng.choice([0, 1, 8, 16, 40, 64, 128])
        T = _log(rng, 1, 8192)
        return dict(op=op, T=T, H=H, page=page, neox=rng.random() < 0.5, norm=rng.random() < 0.8,
                    rows_out=rng.random() < 0.4, padded=rng.randrange(T) if rng.random() < 0.3 else 0)
    B = _log(rng, 1, 64)
    hi = _log(rng, 16, min(131072, 1200000 // B))
    lo = rng.choice([1, max(1, hi // 8), hi])
    if op in ("decode", "weights"):
        H = rng.choice([1, 5, 16, 40, 64, 128])
        s = rng.choice([1, 1, 2, 3, 4] if op == "decode" else [1, 1, 2, 4, 32])
        while B * s * H * hi > 1.5e8 and s > 1:
            s //= 2
        if op == "decode":
            return dict(op=op, B=B, s=s, H=H, page=page, lo=lo, hi=hi, sinks=rng.random() < 0.3)
        return dict(op=op, fmt=rng.choice(["bf16", "e4m3", "fp4"]), B=B, s=s, H=H, page=page, lo=lo, hi=hi)
    keep = _log(rng, 1, hi)
    if op == "select":
        return dict(op=op, B=B, lo=lo, hi=hi, keep=keep, first=rng.choice([0, 1, 4, 64]), recent=rng.choice([0, 1, 32, 512]))
    return dict(op=op, fmt=rng.choice(["bf16", "e4m3", "fp4"]), B=B, page=page, lo=lo, hi=hi, keep=keep)


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(shape, g, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


def _lengths(c):
    """Lengths spread evenly over lo .. hi, so that their sum is the case's; the seed gives their order."""
    n = c["B"]
    return [c["lo"] + (c["hi"] - c["lo"]) * (2 * i + 1) // (2 * n) for i in range(n)]


def _pages(c, g):
    """lens, block table and row count of a paged cache: page ids at random, two pages that nobody holds."""
    B, page = c["B"], c["page"]
    lens = torch.tensor(_lengths(c), dtype=torch.int32, device=DEV)[torch.randperm(B, generator=g, device=DEV)]
    max_pages = -(-c["hi"] // page)
    held = (lens + page - 1) // page
    used = int(held.sum())
    ids = torch.randperm(used + 2, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(max_pages, device=DEV)[None, :] < held[:, None]] = ids[:used]
    return lens, table, used + 2


def _fp4_rows(x, pe):
    """4-bit rows of latents x and RoPE columns pe as bytes."""
    v = x.float().view(-1, SCALES, 16)
    s = torch.clamp(v.abs().amax(2, keepdim=True) / 6, 2.0 ** -9, 448).to(torch.float8_e4m3fn)
    t = v / s.float()
    a = t.abs().clamp(max=6.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=1.0))) - 1)
    a = torch.round(a / step) * step                       # 0 .5 1 1.5 2 3 4 6
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8) | (torch.signbit(t).to(torch.uint8) << 3)
    code = code.view(-1, LATENT)
    return torch.cat([code[:, 0::2] | (code[:, 1::2] << 4), s.view(-1, SCALES).view(torch.uint8),
                      pe.contiguous().view(torch.uint8).view(-1, 2 * ROPE)], 1)


def _cache(fmt, rows, g):
    """`rows` rows of a cache and the scale of its values."""
    if fmt == "fp4":
        buf = torch.empty((rows, FP4_ROW), dtype=torch.uint8, device=DEV)
        for at in range(0, rows, 1 << 18):
            n = min(1 << 18, rows - at)
            buf[at:at + n] = _fp4_rows(torch.randn((n, LATENT), generator=g, device=DEV), _normal((n, ROPE), g))
        return buf, 1.0
    if fmt == "bf16":
        buf = torch.empty((rows, DK), dtype=torch.bfloat16, device=DEV)
        return buf.normal_(generator=g), 1.0
    buf = torch.randn((rows, DK), generator=g, device=DEV, dtype=torch.float32)
    return (buf / 0.05).to(torch.float8_e4m3fn), 0.05


def _prepare_append(c, g):
    T, H, page = c["T"], c["H"], c["page"]
    kv_a = _normal((T, DK), g)                       # the down-projection's output: latent and RoPE columns
    pages = -(-T // page) + 3
    rows = pages * page
    buf, _ = _cache("fp4", rows + 1, g)              # and one spare row
    slots = torch.randperm(rows, generator=g, device=DEV)[:T].to(torch.int32)
    max_pos = 32768
    pos = torch.randint(0, max_pos, (T,), generator=g, device=DEV, dtype=torch.int32)
    if c["padded"]:
        slots[T - c["padded"]:] = -1
        pos[T - c["padded"]:] = -1
    ang = (torch.arange(max_pos, device=DEV, dtype=torch.float64)[:, None]
           * 10000.0 ** (-2.0 * torch.arange(32, device=DEV, dtype=torch.float64)[None, :] / 64))
    s = dict(c_kv=kv_a[:, :LATENT], k_pe=kv_a[:, LATENT:], slots=slots, positions=pos, neox=c["neox"], eps=1e-6,
             cos_sin=torch.cat([ang.cos(), ang.sin()], 1).float(), buf=buf, kv_scale=1.0 if T % 2 == 0 else 0.75,
             cache=buf[:rows].view(pages, page, FP4_ROW), weight=None, q_pe=None, q_out=None, kv_out=None)
    if c["norm"]:
        s["weight"] = (1 + 0.2 * torch.randn(LATENT, generator=g, device=DEV)).bfloat16()
    if H:
        s["q_pe"] = _normal((T, H, 128 + ROPE), g)[:, :, 128:]
        s["q_out"] = _normal((T, H, DK), g)
    if c["rows_out"]:
        s["kv_out"] = _normal((T, DK), g)
    return s


def _prepare_paged(c, g, fmt):
    lens, table, pages = _pages(c, g)
    buf, kv_scale = _cache(fmt, pages * c["page"] + 1, g)      # one spare row behind the pages
    return dict(lens=lens, table=table, buf=buf, kv_scale=kv_scale, page=c["page"], fmt=fmt,
                cache=buf[:pages * c["page"]].view(pages, c["page"], -1))


def _prepare_decode(c, g):
    s = _prepare_paged(c, g, "fp4")
    B, n, H = c["B"], c["s"], c["H"]
    s.update(q=_normal((B, n, H, DK), g), scale=192.0 ** -0.5, sinks=None)
    if c["sinks"]:
        s["sinks"] = 2 * torch.randn(H, generator=g, device=DEV)
    return s


def _prepare_weights(c, g):
    s = _prepare_paged(c, g, c["fmt"])
    B, n, H = c["B"], c["s"], c["H"]
    s.update(q=_normal((B, n, H, DK), g), scale=192.0 ** -0.5, decay=0.875)
    score = _scores(s, torch.float32, s["scale"] * s["kv_scale"])[0]
    s["lse"] = torch.logsumexp(score, 3)                      # what the decode before it gives
    s["weights"] = torch.rand((B, s["table"].shape[1] * c["page"]), generator=g, device=DEV)
    return s


def _prepare_select(c, g):
    B, W = c["B"], c["hi"]
    lens = torch.tensor(_lengths(c), dtype=torch.int32, device=DEV)[torch.randperm(B, generator=g, device=DEV)]
    w = torch.exp(2.5 * torch.randn((B, W), generator=g, device=DEV)) / W   # few keys get most of the attention
    w[torch.rand((B, W), generator=g, device=DEV) < 0.1] = 0                # some none that fp32 holds
    keep = torch.clamp(torch.randint(c["keep"] * 3 // 4, c["keep"] + 1, (B,), generator=g, device=DEV, dtype=torch.int32), min=1)
    keep[0] = c["keep"]
    i32 = dict(dtype=torch.int32, device=DEV)
    return dict(weights=w, lens=lens, keep=keep, K=c["keep"], first=c["first"], recent=c["recent"],
                idx=torch.empty((B, c["keep"]), **i32), count=torch.empty(B, **i32), dropped=torch.empty(B, **i32))


def _prepare_compact(c, g):
    s = _prepare_paged(c, g, c["fmt"])
    B, K, W = c["B"], c["keep"], s["table"].shape[1] * c["page"]
    s["weights"] = torch.rand((B, W), generator=g, device=DEV)
    order = s["weights"].masked_fill(torch.arange(W, device=DEV)[None, :] >= s["lens"][:, None], -1.0)
    count = torch.clamp(s["lens"], max=K)
    idx = torch.sort(order, dim=1, descending=True).indices[:, :K]
    idx = torch.where(torch.arange(K, device=DEV)[None, :] < count[:, None], idx, W).sort(1).values
    s.update(count=count, idx=torch.where(idx < W, idx, -1).to(torch.int32))
    return s


def prepare(case, seed):
    make = dict(append=_prepare_append, decode=_prepare_decode, weights=_prepare_weights, select=_prepare_select,
                compact=_prepare_compact)[case["op"]]
    return dict(make(case, _gen(seed)), op=case["op"])


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def _rotate(x, cs, neox):
    c, t = cs[..., :32], cs[..., 32:]
    if neox:
        a, b = x[..., :32], x[..., 32:]
        return torch.cat([a * c - b * t, a * t + b * c], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * t, a * t + b * c], -1).flatten(-2)


def _nearest(a, low, bits, most):
    """The nearest value with `bits` bits behind the leading one and no step below that of `low`, ties to even."""
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=low))) - bits)
    return torch.clamp(torch.round(a / step) * step, max=most)


def _plain_append(s):
    pos, slots, buf = s["positions"], s["slots"], s["buf"]
    cs = s["cos_sin"][pos.clamp(min=0).long()]
    live = pos >= 0
    lat = s["c_kv"].double()                          # 64 bits: a value next to a border falls on its own side
    if s["weight"] is not None:
        lat = lat * torch.rsqrt((lat * lat).mean(1, keepdim=True) + s["eps"]) * s["weight"].double()
    pe = _rotate(s["k_pe"].float(), cs, s["neox"])
    spare = buf.shape[0] - 1
    at = torch.where(live & (slots >= 0), slots.long(), spare)
    v = (lat / s["kv_scale"]).view(-1, SCALES, 16)
    scale = _nearest(torch.clamp(v.abs().amax(2, keepdim=True) / 6, 2.0 ** -9, 448), 2.0 ** -6, 3, 448)
    a = _nearest(v.abs() / scale, 1.0, 1, 6.0)
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8) | (torch.signbit(v).to(torch.uint8) << 3)
    code = code.view(-1, LATENT)
    buf[at, :CODES] = code[:, 0::2] | (code[:, 1::2] << 4)
    buf[at, CODES:CODES + SCALES] = scale[:, :, 0].float().to(torch.float8_e4m3fn).view(torch.uint8)
    buf[at, CODES + SCALES:] = (pe / s["kv_scale"]).bfloat16().view(torch.uint8)
    got = _cache_values(s)
    if s["q_pe"] is not None:
        q = _rotate(s["q_pe"].float(), cs[:, None, :], s["neox"]).bfloat16()
        part = s["q_out"][:, :, LATENT:]
        part.copy_(torch.where(live[:, None, None], q, part))
        got["q"] = s["q_out"]
    if s["kv_out"] is not None:
        row = torch.cat([lat.float(), pe], 1)
        s["kv_out"].copy_(torch.where(live[:, None], row.bfloat16(), s["kv_out"]))
        got["rows"] = s["kv_out"]
    return got


def _cache_values(s):
    """The whole cache: the pairs of codes (of all columns, so equal or not), the scales and the RoPE columns."""
    c = s["cache"]
    return dict(codes=c[..., :CODES], scales=c[..., CODES:CODES + SCALES].view(torch.float8_e4m3fn),
                pe=c[..., CODES + SCALES:].view(torch.bfloat16))


E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


def _row_values(rows, fmt, d):
    if fmt != "fp4":
        return rows.to(d)
    table = torch.tensor(E2M1, dtype=d, device=rows.device)
    code = torch.stack([rows[..., :CODES] & 15, rows[..., :CODES] >> 4], -1).flatten(-2)
    scale = rows[..., CODES:CODES + SCALES].view(torch.float8_e4m3fn).to(d)
    lat = table[code.int()].unflatten(-1, (SCALES, 16)) * scale[..., None]
    return torch.cat([lat.flatten(-2), rows[..., CODES + SCALES:].contiguous().view(torch.bfloat16).to(d)], -1)


def _gathered(s):
    """Where each request's keys are [B, W] (the spare row for those that are none), W up to the longest."""
    table, page = s["table"], s["page"]
    W = table.shape[1] * page
    at = table[:, :, None].long() * page + torch.arange(page, device=table.device)
    return torch.where(torch.arange(W, device=table.device)[None, :] < s["lens"][:, None], at.view(-1, W), s["buf"].shape[0] - 1)


def _scores(s, d, factor):
    """Scores [B, s, H, W] with the hidden ones at -inf, and the keys' values [B, W, 576]."""
    k = _row_values(s["buf"].view(torch.uint8)[_gathered(s)].view(s["buf"].dtype), s["fmt"], d)
    B, n, H, _ = s["q"].shape
    W = k.shape[1]
    score = torch.matmul(s["q"].to(d).view(B, n * H, DK), k.transpose(1, 2)).view(B, n, H, W) * factor
    last = s["lens"][:, None] - n + torch.arange(n, device=k.device)[None, :]
    hidden = torch.arange(W, device=k.device)[None, None, :] > last[:, :, None]
    return score.masked_fill_(hidden[:, :, None, :], float("-inf")), k


def _plain_decode(s):
    score, k = _scores(s, torch.float32, s["scale"] * s["kv_scale"])
    B, n, H, W = score.shape
    top = score.amax(3, keepdim=True)
    if s["sinks"] is not None:
        top = torch.maximum(top, s["sinks"].view(1, 1, H, 1))
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    p = torch.exp_(score - top)
    total = p.sum(3, keepdim=True)
    if s["sinks"] is not None:
        total = total + torch.exp(s["sinks"].view(1, 1, H, 1) - top)
    out = torch.matmul(p.view(B, n * H, W), k[:, :, :LATENT]).view(B, n, H, LATENT) * s["kv_scale"]
    out = torch.where(total > 0, out / total, torch.zeros_like(out))
    return dict(out=out.bfloat16(), lse=(top + torch.log(total))[..., 0])


def _plain_weights(s):
    score, _ = _scores(s, torch.float32, s["scale"] * s["kv_scale"])
    lse = s["lse"][..., None]
    p = torch.exp_(score - torch.where(torch.isinf(lse), torch.zeros_like(lse), lse))
    w = s["weights"]
    live = torch.arange(w.shape[1], device=w.device)[None, :] < s["lens"][:, None]
    w.copy_(torch.where(live, s["decay"] * w + p.sum((1, 2)), w))
    return dict(weights=w)


def _plain_select(s):
    w, lens, K = s["weights"], s["lens"].long()[:, None], s["K"]
    B, W = w.shape
    j = torch.arange(W, device=w.device)[None, :]
    n = torch.minimum(lens, s["keep"].long()[:, None])
    recent = torch.clamp(n, max=s["recent"])
    first = torch.clamp(n - recent, max=s["first"])
    w = torch.where((j < first) | (j >= lens - recent), float("inf"), w)
    w = torch.where(j < lens, w, float("-inf"))
    order = torch.sort(w, dim=1, descending=True, stable=True).indices[:, :K]
    kept = torch.arange(order.shape[1], device=w.device)[None, :] < n
    idx = torch.where(kept, order, W).sort(1).values
    s["idx"].copy_(torch.where(idx < W, idx, -1))
    return dict(idx=s["idx"], count=n[:, 0].to(torch.int32), dropped=(n - lens)[:, 0].to(torch.int32))


def _plain_compact(s):
    idx, buf, w = s["idx"], s["buf"], s["weights"]
    at = _gathered(s)
    spare = buf.shape[0] - 1
    kept = torch.arange(idx.shape[1], device=idx.device)[None, :] < s["count"][:, None]
    src = torch.gather(at, 1, idx.long().clamp(min=0))
    raw = buf.view(torch.uint8)
    raw[torch.where(kept, at[:, :idx.shape[1]], spare)] = raw[torch.where(kept, src, spare)]
    w[:, :idx.shape[1]] = torch.where(kept, torch.gather(w, 1, idx.long().clamp(min=0)), w[:, :idx.shape[1]])
    return dict(cache=s["cache"].view(torch.uint8), weights=w)


def _own_append(s):
    from mla_attention_gb300 import mla_kv_append_fp4
    mla_kv_append_fp4(s["c_kv"], s["k_pe"], s["slots"], s["positions"], s["cos_sin"], s["cache"], s["kv_scale"],
                      norm_weight=s["weight"], eps=s["eps"], q_pe=s["q_pe"], q_out=s["q_out"], kv_out=s["kv_out"],
                      is_neox=s["neox"])
    got = _cache_values(s)
    if s["q_out"] is not None:
        got["q"] = s["q_out"]
    if s["kv_out"] is not None:
        got["rows"] = s["kv_out"]
    return got


def _own_decode(s):
    from mla_attention_gb300 import mla_decode_fp4
    out, lse = mla_decode_fp4(s["q"], s["cache"], s["kv_scale"], s["table"], s["lens"], s["scale"], sinks=s["sinks"])
    return dict(out=out, lse=lse)


def _own_weights(s):
    from mla_attention_gb300 import mla_key_weights
    return dict(weights=mla_key_weights(s["q"], s["lse"], s["cache"], s["table"], s["lens"], s["scale"], s["weights"],
                                        kv_scale=s["kv_scale"], decay=s["decay"]))


def _own_select(s):
    from mla_attention_gb300 import mla_select_keys
    idx, count, dropped = mla_select_keys(s["weights"], s["lens"], s["keep"], s["K"], first=s["first"], recent=s["recent"],
                                          idx=s["idx"], count=s["count"], dropped=s["dropped"])
    return dict(idx=idx, count=count, dropped=dropped)


def _own_compact(s):
    from mla_attention_gb300 import mla_compact_rows
    mla_compact_rows(s["cache"], s["table"], s["idx"], s["count"], weights=s["weights"])
    return dict(cache=s["cache"].view(torch.uint8), weights=s["weights"])


def run(state):
    if own:
        return dict(append=_own_append, decode=_own_decode, weights=_own_weights, select=_own_select,
                    compact=_own_compact)[state["op"]](state)
    return dict(append=_plain_append, decode=_plain_decode, weights=_plain_weights, select=_plain_select,
                compact=_plain_compact)[state["op"]](state)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "append":
        live = c["T"] - c["padded"]
        row = 2 * DK + FP4_ROW + (2 * DK if c["rows_out"] else 0)
        return dict(bytes=live * (row + c["H"] * ROPE * 4 + 8 + ROPE * 4), flops=live * (LATENT * 6 + (c["H"] + 1) * ROPE * 3))
    keys = sum(_lengths(c))
    if c["op"] == "decode":
        rows = c["s"] * c["H"]
        table = 4 * (keys // c["page"] + c["B"])
        return dict(bytes=keys * FP4_ROW + table + c["B"] * rows * (2 * DK + 2 * LATENT + 4), flops=2 * keys * rows * (DK + LATENT))
    if c["op"] == "weights":
        rows = c["s"] * c["H"]
        table = 4 * (keys // c["page"] + c["B"])
        return dict(bytes=keys * (ROW_BYTES[c["fmt"]] + 8) + table + c["B"] * rows * (2 * DK + 4), flops=2 * keys * rows * DK)
    if c["op"] == "select":
        return dict(bytes=4 * keys + 4 * c["B"] * c["keep"] + 16 * c["B"], flops=0)
    kept = sum(min(n, c["keep"]) if n > c["keep"] else 0 for n in _lengths(c))    # shorter requests stay as they are
    listed_rows = sum(min(n, c["keep"]) for n in _lengths(c))
    return dict(bytes=2 * kept * (ROW_BYTES[c["fmt"]] + 4) + 4 * listed_rows + 4 * c["B"], flops=0)


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def _turned(x, angles_cos, angles_sin, neox):
    """Each pair as a complex number, times its angle's."""
    pairs = torch.complex(x[..., :32], x[..., 32:]) if neox else torch.view_as_complex(x.unflatten(-1, (32, 2)).contiguous())
    turned = pairs * torch.complex(angles_cos, angles_sin)
    return torch.cat([turned.real, turned.imag], -1) if neox else torch.view_as_real(turned).flatten(-2)


def _held(s, b, d):
    """The values that request b's cached rows stand for, [len, 576]."""
    n, page = int(s["lens"][b]), s["page"]
    j = torch.arange(n, device=DEV)
    rows = s["cache"].view(torch.uint8).flatten(0, 1)[s["table"][b][j // page].long() * page + j % page].view(s["cache"].dtype)
    if s["fmt"] != "fp4":
        return rows.to(d) * s["kv_scale"]
    sign_and_size = torch.stack([rows[:, :CODES] % 16, torch.div(rows[:, :CODES], 16, rounding_mode="floor")], 2).flatten(1).to(d)
    size = sign_and_size % 8
    exponent = torch.div(size, 2, rounding_mode="floor")
    value = torch.where(exponent == 0, size / 2, (1 + (size % 2) / 2) * 2.0 ** (exponent - 1))
    value = torch.where(sign_and_size >= 8, -value, value)
    scales = rows[:, CODES:CODES + SCALES].view(torch.float8_e4m3fn).to(d).repeat_interleave(16, 1)
    return torch.cat([value * scales, rows[:, CODES + SCALES:].contiguous().view(torch.bfloat16).to(d)], 1) * s["kv_scale"]


def exact(case, seed):
    if case["op"] in ("select", "compact"):
        return None               # whole numbers, moved rows
    s = prepare(case, seed)
    d = torch.float64
    if case["op"] == "append":
        live = torch.nonzero(s["positions"] >= 0)[:, 0]
        lat, pe = s["c_kv"][live].to(d), s["k_pe"][live].to(d)
        if case["norm"]:
            lat = lat / torch.sqrt((lat ** 2).sum(1, keepdim=True) / LATENT + s["eps"]) * s["weight"].to(d)
        table = s["cos_sin"][s["positions"][live].long()].to(d)
        cos, sin = table[:, :32], table[:, 32:]
        pe = _turned(pe, cos, sin, case["neox"])
        at = s["slots"][live].long()
        parts = _cache_values(s)
        held = parts["pe"].to(d).flatten(0, 1)
        held[at] = pe / s["kv_scale"]
        top = torch.clamp((lat / s["kv_scale"]).unflatten(1, (SCALES, 16)).abs().max(-1).values / 6.0, 2.0 ** -9, 448.0)
        unit = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -6))) - 3)
        scales = parts["scales"].to(d).flatten(0, 1)
        scales[at] = torch.clamp(torch.round(top / unit) * unit, max=448.0)
        got = dict(codes=None, scales=scales.view(parts["scales"].shape), pe=held.view(parts["pe"].shape))
        if case["H"]:
            q = s["q_out"].to(d)
            q[live, :, LATENT:] = _turned(s["q_pe"][live].to(d), cos[:, None], sin[:, None], case["neox"])
            got["q"] = q
        if case["rows_out"]:
            rows = s["kv_out"].to(d)
            rows[live] = torch.cat([lat, pe], 1)
            got["rows"] = rows
        return got
    B, n, H, _ = s["q"].shape
    if case["op"] == "decode":
        out = torch.zeros((B, n, H, LATENT), dtype=d, device=DEV)
        lse = torch.full((B, n, H), float("-inf"), dtype=d, device=DEV)
        for b in range(B):
            k = _held(s, b, d)
            for i in range(n):
                m = max(0, k.shape[0] - n + 1 + i)
                score = s["scale"] * torch.einsum("hd,kd->hk", s["q"][b, i].to(d), k[:m])
                if s["sinks"] is not None:                   # one more key, with no value
                    score = torch.cat([score, s["sinks"].to(d)[:, None]], 1)
                if score.shape[1]:
                    lse[b, i] = torch.logsumexp(score, 1)
                    out[b, i] = torch.softmax(score, 1)[:, :m] @ k[:m, :LATENT]
        return dict(out=out, lse=lse)
    w = s["weights"].to(d)
    for b in range(B):
        k = _held(s, b, d)
        m = k.shape[0]
        w[b, :m] *= s["decay"]
        for i in range(n):
            seen = max(0, m - n + 1 + i)
            score = s["scale"] * torch.einsum("hd,kd->hk", s["q"][b, i].to(d), k[:seen])
            w[b, :seen] += torch.exp(score - s["lse"][b, i].to(d)[:, None]).sum(0)
    return dict(weights=w)
