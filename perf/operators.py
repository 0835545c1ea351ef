"""The operators of the serving step around the latent attention, as measured cases.

Four operators (include/mla.h has their definitions):

* slots:  mla_slot_map   block tables, positions and slots of a step's tokens, built on the GPU from request lengths
* norm:   mla_rms_norm   root-mean-square norm with the residual's addition, out in bf16 or in e4m3 with scales
* append: mla_kv_append  latent norm, RoPE and the write of cache rows by slot, into a bf16 or an e4m3 cache
* w4:     mla_bmm_w4     per-head products of a few tokens with 4-bit weights and group scales

`run` computes each in plain torch (32-bit arithmetic, rounded once at the end) or, where `own` is true, by the
library's call.  `exact` follows the definitions in 64 bits.
"""
import torch

own = False

DEV = "cuda"
LATENT, ROPE, DK = 512, 64, 576


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # one request generates one token: the latency of a lone user's step
        dict(name="slots-one-request", op="slots", mode="decode", B=1, page=64, max_len=32768, N=1),
        # a decode batch of 64 requests at 4K..32K tokens in 64-token pages, two draft tokens kept or dropped
        dict(name="slots-verify-64", op="slots", mode="verify", B=64, page=64, max_len=32768, N=256),
        # a scheduler's step that mixes prompts and running requests, 64K tokens in 16-token pages
        dict(name="slots-mixed-512", op="slots", mode="mixed", B=512, page=16, max_len=16384, N=65536),
        # the norm before a layer, for one token
        dict(name="norm-1x8192", op="norm", T=1, D=8192, pad=0, residual=True, e4m3=False, group=0),
        # an odd width inside a wider row (a norm of a slice of a fused projection), 8-bit rows for the next product
        dict(name="norm-257x1535-e4m3", op="norm", T=257, D=1535, pad=66, residual=False, e4m3=True, group=0),
        # the norm before a layer over a long prompt, 8 bits out with a scale for each 128 columns
        dict(name="norm-16384x5120-e4m3", op="norm", T=16384, D=5120, pad=0, residual=True, e4m3=True, group=128),
        # a decode step's rows into an 8-bit cache, a batch padded to its captured size
        dict(name="append-decode-64-e4m3", op="append", T=64, H=128, page=64, e4m3=True, neox=False, norm=True,
             rows_out=False, padded=9),
        # a prompt's rows into the cache and, as dense rows, for the prefill attention
        dict(name="append-prefill-8192", op="append", T=8192, H=128, page=64, e4m3=False, neox=True, norm=True,
             rows_out=True, padded=0),
        # cache rows alone for a packed batch of prompts
        dict(name="append-rows-32768-e4m3", op="append", T=32768, H=0, page=16, e4m3=True, neox=False, norm=True,
             rows_out=False, padded=0),
        # the absorption of one token's query, weights in 4 bits
        dict(name="w4-absorb-1", op="w4", T=1, H=128, N=512, K=128, group=32, wide=False),
        # the value projection of a small odd batch, fp32 scales
        dict(name="w4-project-17", op="w4", T=17, H=128, N=128, K=512, group=64, wide=True),
        # the projection of 128 heads x 128 values back to the hidden width, four draft tokens
        dict(name="w4-linear-4", op="w4", T=4, H=1, N=8192, K=16384, group=128, wide=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["slots", "norm", "append", "w4"])
    if op == "slots":
        mode = rng.choice(["decode", "verify", "mixed"])
        B, page = _log(rng, 1, 512), rng.choice([16, 32, 64, 128])
        max_len = _log(rng, 64, 32768 if B <= 128 else 8192)
        N = {"decode": B + rng.randrange(8), "verify": 4 * B, "mixed": B + _log(rng, 64, 65000)}[mode]
        return dict(op=op, mode=mode, B=B, page=page, max_len=max_len, N=N)
    if op == "norm":
        e4m3 = rng.random() < 0.5
        group = rng.choice([0, 32, 64, 128]) if e4m3 else 0
        D = _log(rng, 64, 16384)
        D = max(group, D // group * group) if group else (D // 8 * 8 if rng.random() < 0.6 else D)
        T = _log(rng, 1, max(1, min(32768, 52428800 // D)))
        return dict(op=op, T=T, D=D, pad=rng.choice([0, 0, 8, 64, 65]), residual=rng.random() < 0.6, e4m3=e4m3,
                    group=group)
    if op == "append":
        H = rng.choice([0, 1, 8, 16, 40, 64, 128])
        T = _log(rng, 1, 32768 if H == 0 else 8192)
        return dict(op=op, T=T, H=H, page=rng.choice([16, 32, 64, 128]), e4m3=rng.random() < 0.5,
                    neox=rng.random() < 0.5, norm=rng.random() < 0.8, rows_out=rng.random() < 0.4,
                    padded=rng.randrange(T) if rng.random() < 0.3 else 0)
    group = rng.choice([32, 64, 128])
    if rng.random() < 0.5:
        H, (N, K) = rng.choice([8, 16, 64, 128]), rng.choice([(512, 128), (128, 512), (576, 256), (100, 384)])
    else:
        H, N, K = 1, _log(rng, 64, 8192), group * max(1, _log(rng, 512, 16384) // group)
    return dict(op=op, T=_log(rng, 1, 64), H=H, N=N, K=K, group=group, wide=rng.random() < 0.4)


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(shape, g, scale=1.0):
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


def _ints(lo, hi, shape, g):
    return torch.randint(lo, hi, shape, generator=g, device=DEV, dtype=torch.int32)


def _prepare_slots(c, g):
    B, page, N, L = c["B"], c["page"], c["N"], c["max_len"]
    lens = _ints(max(1, L // 8), L + 1, (B,), g)
    u = torch.rand((B,), generator=g, device=DEV)
    if c["mode"] == "decode":      # one token each; one request in thirty ends and gives its pages back
        new = torch.where(u < 1 / 30, -lens, torch.ones_like(lens))
    elif c["mode"] == "verify":    # draft tokens are appended, or rejected ones dropped
        new = _ints(-3, 5, (B,), g)
    else:                          # one request in eight is a prompt that starts or goes on, the others decode
        prompt = u < 1 / 8
        lens = torch.where(u < 1 / 16, torch.zeros_like(lens), lens)
        w = torch.rand((B,), generator=g, device=DEV) * prompt
        new = torch.where(prompt, (w / w.sum().clamp(min=1e-9) * (N - B)).floor().to(torch.int32), 1)
    new = new.to(torch.int32)
    have = (lens + page - 1) // page
    max_pages = -(-(L + N) // page) + 1
    num_pages = B * (-(-L // page)) + N // page + B + 1
    used = int(have.sum())
    free = num_pages - used
    ids = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device=DEV)
    table[torch.arange(max_pages, device=DEV)[None, :] < have[:, None]] = ids[:used]
    pool = torch.full((num_pages,), -1, dtype=torch.int32, device=DEV)
    head = int(_ints(0, num_pages, (1,), g))
    pool[(head + torch.arange(free, device=DEV)) % num_pages] = ids[used:]
    i32 = dict(dtype=torch.int32, device=DEV)
    return dict(lens=lens, new=new, table=table, pool=pool, pool_state=torch.tensor([head, free], **i32), page=page,
                N=N, positions=torch.empty(N, **i32), slots=torch.empty(N, **i32), cu=torch.empty(B + 1, **i32),
                lens_out=torch.empty(B, **i32), pool_state_out=torch.empty(2, **i32))


def _prepare_norm(c, g):
    T, D, pad = c["T"], c["D"], c["pad"]
    s = dict(x=_normal((T, D + pad), g)[:, :D], weight=(1 + 0.2 * torch.randn(D, generator=g, device=DEV)).bfloat16(),
             eps=1e-6, group=c["group"], residual=None, residual_out=None, scales=None)
    if c["residual"]:
        s["residual"] = _normal((T, D), g, 4.0)
        s["residual_out"] = torch.empty((T, D), dtype=torch.bfloat16, device=DEV)
    if c["e4m3"]:
        s["out"] = torch.empty((T, D), dtype=torch.float8_e4m3fn, device=DEV)
        s["scales"] = torch.empty((T, D // c["group"] if c["group"] else 1), dtype=torch.float32, device=DEV)
    else:
        s["out"] = torch.empty((T, D), dtype=torch.bfloat16, device=DEV)
    return s


def _prepare_append(c, g):
    T, H, page = c["T"], c["H"], c["page"]
    kv_a = _normal((T, DK), g)                       # the down-projection's output: latent and RoPE columns
    pages = -(-T // page) + 3
    rows = pages * page
    buf = _normal((rows + 1, DK), g)                 # the cache, and one spare row behind it
    kv_scale = 0.02 if c["e4m3"] else 1.0
    if c["e4m3"]:
        buf = (buf.float() / 0.05).to(torch.float8_e4m3fn)
    slots = torch.randperm(rows, generator=g, device=DEV)[:T].to(torch.int32)
    max_pos = 32768
    pos = _ints(0, max_pos, (T,), g)
    if c["padded"]:
        slots[T - c["padded"]:] = -1
        pos[T - c["padded"]:] = -1
    ang = (torch.arange(max_pos, device=DEV, dtype=torch.float64)[:, None]
           * 10000.0 ** (-2.0 * torch.arange(32, device=DEV, dtype=torch.float64)[None, :] / 64))
    s = dict(c_kv=kv_a[:, :LATENT], k_pe=kv_a[:, LATENT:], slots=slots, positions=pos, neox=c["neox"], eps=1e-6,
             cos_sin=torch.cat([ang.cos(), ang.sin()], 1).float(), buf=buf, kv_scale=kv_scale,
             cache=buf[:rows].view(pages, page, DK), weight=None, q_pe=None, q_out=None, kv_out=None)
    if c["norm"]:
        s["weight"] = (1 + 0.2 * torch.randn(LATENT, generator=g, device=DEV)).bfloat16()
    if H:
        s["q_pe"] = _normal((T, H, 128 + ROPE), g)[:, :, 128:]
        s["q_out"] = _normal((T, H, DK), g)
    if c["rows_out"]:
        s["kv_out"] = _normal((T, DK), g)
    return s


def _prepare_w4(c, g):
    T, H, N, K = c["T"], c["H"], c["N"], c["K"]
    scales = (0.5 + torch.rand((H, N, K // c["group"]), generator=g, device=DEV)) * (0.2 / K ** 0.5)
    return dict(x=_normal((T, H, K), g), w4=torch.randint(0, 256, (H, N, K // 2), generator=g, device=DEV, dtype=torch.uint8),
                scales=scales if c["wide"] else scales.bfloat16(),
                out=torch.empty((T, H, N), dtype=torch.bfloat16, device=DEV))


def prepare(case, seed):
    make = dict(slots=_prepare_slots, norm=_prepare_norm, append=_prepare_append, w4=_prepare_w4)[case["op"]]
    return dict(make(case, _gen(seed)), op=case["op"])


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------
def _plain_slots(s):
    lens, new, table, pool, page, N = s["lens"], s["new"], s["table"], s["pool"], s["page"], s["N"]
    B, P = lens.numel(), pool.numel()
    head, count = s["pool_state"][0], s["pool_state"][1]
    now = torch.clamp(lens + new, min=0)
    have, need = (lens + page - 1) // page, (now + page - 1) // page
    add = torch.clamp(new, min=0)
    zero = torch.zeros(1, dtype=torch.int64, device=lens.device)
    cu = torch.cat([zero, add.cumsum(0)])
    pops = torch.cat([zero, torch.clamp(need - have, min=0).cumsum(0)])
    puts = torch.cat([zero, torch.clamp(have - need, min=0).cumsum(0)])
    # pages: entry i of request b, taken from the ring's head or given back behind its tail
    col = torch.arange(table.shape[1], device=lens.device)[None, :]
    grow = (col >= have[:, None]) & (col < need[:, None])
    drop = (col >= need[:, None]) & (col < have[:, None])
    take = (head + pops[:B, None] + col - have[:, None]) % P
    table.copy_(torch.where(grow, pool[take], table))
    put = torch.where(drop, (head + count + puts[:B, None] + col - need[:, None]) % P, P)
    ring = torch.cat([pool, pool[:1]])
    ring.scatter_(0, put.reshape(-1), table.reshape(-1))
    pool.copy_(ring[:P])
    # tokens
    tok = torch.arange(N, device=lens.device)
    b = torch.searchsorted(cu[1:], tok, right=True).clamp(max=B - 1)
    real = tok < cu[B]
    pos = torch.where(real, lens[b] + tok - cu[b], 0)
    slot = table[b, pos // page].long() * page + pos % page
    i32 = torch.int32
    return dict(positions=torch.where(real, pos, -1).to(i32), slots=torch.where(real, slot, -1).to(i32), cu=cu.to(i32),
                lens=now.to(i32), pool_state=torch.stack([(head + pops[B]) % P, count - pops[B] + puts[B]]).to(i32),
                table=table, pool=pool)


def _plain_norm(s):
    h = s["x"].float()
    got = {}
    if s["residual"] is not None:
        h = h + s["residual"].float()
        got["residual"] = h.bfloat16()
    y = h * torch.rsqrt((h * h).mean(1, keepdim=True) + s["eps"]) * s["weight"].float()
    if s["scales"] is None:
        return dict(got, out=y.bfloat16())
    T, D = y.shape
    y = y.view(T, -1, s["group"] or D)
    scale = torch.clamp(y.abs().amax(2, keepdim=True) / 448, min=2.0 ** -126)
    q = torch.clamp(y / scale, -448, 448).to(torch.float8_e4m3fn)
    return dict(got, out=q.view(T, D), scales=scale.view(T, -1))


def _rotate(x, cs, neox):
    c, t = cs[..., :32], cs[..., 32:]
    if neox:
        a, b = x[..., :32], x[..., 32:]
        return torch.cat([a * c - b * t, a * t + b * c], -1)
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * c - b * t, a * t + b * c], -1).flatten(-2)


def _plain_append(s):
    pos, slots, buf = s["positions"], s["slots"], s["buf"]
    cs = s["cos_sin"][pos.clamp(min=0).long()]
    live = pos >= 0
    lat = s["c_kv"].float()
    if s["weight"] is not None:
        lat = lat * torch.rsqrt((lat * lat).mean(1, keepdim=True) + s["eps"]) * s["weight"].float()
    row = torch.cat([lat, _rotate(s["k_pe"].float(), cs, s["neox"])], 1)
    spare = buf.shape[0] - 1
    at = torch.where(live & (slots >= 0), slots.long(), spare)
    if buf.dtype == torch.bfloat16:
        buf[at] = row.bfloat16()
    else:
        q = torch.clamp(row / s["kv_scale"], -448, 448).to(torch.float8_e4m3fn)
        buf.view(torch.uint8)[at] = q.view(torch.uint8)
    got = dict(cache=s["cache"])
    if s["q_pe"] is not None:
        q = _rotate(s["q_pe"].float(), cs[:, None, :], s["neox"]).bfloat16()
        part = s["q_out"][:, :, LATENT:]
        part.copy_(torch.where(live[:, None, None], q, part))
        got["q"] = s["q_out"]
    if s["kv_out"] is not None:
        s["kv_out"].copy_(torch.where(live[:, None], row.bfloat16(), s["kv_out"]))
        got["rows"] = s["kv_out"]
    return got


def _plain_w4(s):
    H, N, half = s["w4"].shape
    w = torch.stack([s["w4"] & 15, s["w4"] >> 4], -1).view(H, N, s["scales"].shape[2], -1).float() - 8
    w = (w * s["scales"].float()[..., None]).view(H, N, 2 * half)
    y = torch.matmul(s["x"].float().transpose(0, 1), w.transpose(1, 2))
    return dict(out=y.transpose(0, 1).bfloat16())


def _own_slots(s):
    from mla_attention_gb300 import mla_slot_map
    mla_slot_map(s["lens"], s["new"], s["table"], s["pool"], s["pool_state"], s["page"], s["N"],
                 positions=s["positions"], slots=s["slots"], cu_tokens=s["cu"], lens_out=s["lens_out"],
                 pool_state_out=s["pool_state_out"])
    return dict(positions=s["positions"], slots=s["slots"], cu=s["cu"], lens=s["lens_out"],
                pool_state=s["pool_state_out"], table=s["table"], pool=s["pool"])


def _own_norm(s):
    from mla_attention_gb300 import mla_rms_norm
    out, residual, scales = mla_rms_norm(s["x"], s["weight"], s["eps"], residual=s["residual"],
                                         residual_out=s["residual_out"], out=s["out"], group=s["group"],
                                         scales=s["scales"])
    got = dict(out=out)
    if residual is not None:
        got["residual"] = residual
    if scales is not None:
        got["scales"] = scales
    return got


def _own_append(s):
    from mla_attention_gb300 import mla_kv_append
    mla_kv_append(s["c_kv"], s["k_pe"], s["slots"], s["positions"], s["cos_sin"], s["cache"], s["kv_scale"],
                  norm_weight=s["weight"], eps=s["eps"], q_pe=s["q_pe"], q_out=s["q_out"], kv_out=s["kv_out"],
                  is_neox=s["neox"])
    got = dict(cache=s["cache"])
    if s["q_out"] is not None:
        got["q"] = s["q_out"]
    if s["kv_out"] is not None:
        got["rows"] = s["kv_out"]
    return got


def _own_w4(s):
    from mla_attention_gb300 import mla_bmm_w4
    return dict(out=mla_bmm_w4(s["x"], s["w4"], s["scales"], out=s["out"]))


def run(state):
    if own:
        return dict(slots=_own_slots, norm=_own_norm, append=_own_append, w4=_own_w4)[state["op"]](state)
    return dict(slots=_plain_slots, norm=_plain_norm, append=_plain_append, w4=_plain_w4)[state["op"]](state)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------------------------
def work(case):
    c = case
    if c["op"] == "slots":
        # lens, new_tokens in; lens, cu_tokens out; position and slot of every token; the table entry of every
        # touched page (each read from the pool or the table, and written where it is new)
        touched = c["N"] // c["page"] + c["B"]
        return dict(bytes=4 * (4 * c["B"] + 2 * c["N"] + 2 * touched + 4), flops=0)
    if c["op"] == "norm":
        T, D = c["T"], c["D"]
        cols = 2 + (4 if c["residual"] else 0) + (1 if c["e4m3"] else 2)
        scales = 4 * T * (D // c["group"] if c["group"] else 1) if c["e4m3"] else 0
        return dict(bytes=T * D * cols + 2 * D + scales, flops=T * D * 5)
    if c["op"] == "append":
        live = c["T"] - c["padded"]
        row = 2 * DK + DK * (1 if c["e4m3"] else 2) + (2 * DK if c["rows_out"] else 0)
        return dict(bytes=live * (row + c["H"] * ROPE * 4 + 8 + ROPE * 4), flops=live * (LATENT * 4 + (c["H"] + 1) * ROPE * 3))
    T, H, N, K = c["T"], c["H"], c["N"], c["K"]
    scales = H * N * (K // c["group"]) * (4 if c["wide"] else 2)
    return dict(bytes=H * N * K // 2 + scales + 2 * T * H * (K + N), flops=2 * T * H * N * K)


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------
def _e4m3(v):
    """Nearest e4m3 value (ties to even), saturating at 448."""
    a = v.abs().clamp(max=448.0)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.copysign(torch.round(a / step) * step, v)


def _turned(x, angles_cos, angles_sin, neox):
    """Each pair as a complex number, times its angle's."""
    pairs = torch.complex(x[..., :32], x[..., 32:]) if neox else torch.view_as_complex(x.unflatten(-1, (32, 2)).contiguous())
    turned = pairs * torch.complex(angles_cos, angles_sin)
    return torch.cat([turned.real, turned.imag], -1) if neox else torch.view_as_real(turned).flatten(-2)


def exact(case, seed):
    if case["op"] == "slots":
        return None               # whole numbers
    s = prepare(case, seed)
    d = torch.float64
    if case["op"] == "norm":
        h = s["x"].to(d) if s["residual"] is None else s["x"].to(d) + s["residual"].to(d)
        rms = torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / h.shape[1] + s["eps"])
        y = h / rms * s["weight"].to(d)
        got = {} if s["residual"] is None else dict(residual=h)
        if not case["e4m3"]:
            return dict(got, out=y)
        parts = y.unflatten(1, (-1, case["group"])) if case["group"] else y[:, None, :]
        scale = (parts.abs().max(-1).values / 448.0).clamp(min=2.0 ** -126)
        return dict(got, out=_e4m3(parts / scale[..., None]).flatten(1), scales=scale)
    if case["op"] == "append":
        live = torch.nonzero(s["positions"] >= 0)[:, 0]
        lat, pe = s["c_kv"][live].to(d), s["k_pe"][live].to(d)
        if case["norm"]:
            lat = lat / torch.sqrt((lat ** 2).sum(1, keepdim=True) / LATENT + s["eps"]) * s["weight"].to(d)
        table = s["cos_sin"][s["positions"][live].long()].to(d)
        cos, sin = table[:, :32], table[:, 32:]
        row = torch.cat([lat, _turned(pe, cos, sin, case["neox"])], 1)
        cache = s["cache"].to(d).flatten(0, 1)
        cache[s["slots"][live].long()] = _e4m3(row / s["kv_scale"]) if case["e4m3"] else row
        got = dict(cache=cache.view(s["cache"].shape))
        if case["H"]:
            q = s["q_out"].to(d)
            q[live, :, LATENT:] = _turned(s["q_pe"][live].to(d), cos[:, None], sin[:, None], case["neox"])
            got["q"] = q
        if case["rows_out"]:
            rows = s["kv_out"].to(d)
            rows[live] = row
            got["rows"] = rows
        return got
    low, high = (s["w4"] % 16).to(d) - 8, torch.div(s["w4"], 16, rounding_mode="floor").to(d) - 8
    half = case["group"] // 2
    scale = s["scales"].to(d).repeat_interleave(half, 2)
    x = s["x"].to(d)
    return dict(out=torch.einsum("thk,hnk->thn", x[..., 0::2], low * scale) + torch.einsum("thk,hnk->thn", x[..., 1::2], high * scale))
