"""The serving step's operators on values far from one, against the fp64 oracle.

Tolerances as in test_gpu_step.py: half a step of the output's type, the fp32 arithmetic, and for sums their
error bound over the sum of the terms' magnitudes."""
import numpy as np
import pytest
import torch

import oracle.step_oracle as so
from mla_attention_gb300 import inputs as gen, mla_bmm_w4, mla_kv_append
from tests.helpers import dev, to_np
from tests.test_gpu_step import ARITH, E4M3, _bf16, _check_norm, _done, _w4, _within

pytestmark = pytest.mark.gpu

TOKENS = [1, 9, 17, 25, 33, 49]          # one for each width of the token tiles


# ---------------------------------------------------------------------------------------------
# products with 4-bit weights
# ---------------------------------------------------------------------------------------------
def _set_code(w4, k, code):
    """Every column's code of this k."""
    keep, put = (0xF0, code) if k % 2 == 0 else (0x0F, code << 4)
    w4[:, :, k // 2] = (w4[:, :, k // 2] & keep) | put


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T", TOKENS)
def test_w4_a_large_value_under_a_weight_of_zero_adds_nothing(T, group):
    """Code 8 is the weight 0: what x holds there is not part of any sum, however large."""
    g = torch.Generator().manual_seed(T + group)
    H, N, K = 2, 70, 384
    w4, scales = _w4(H, N, K, group, T % 2 == 1, g)
    x = gen.randn_bf16((T, H, K), g)
    for k, size in ((5, 2.0 ** 16), (100, -2.0 ** 20), (170, 2.0 ** 24), (255, 2.0 ** 30), (383, -2.0 ** 40)):
        _set_code(w4, k, 8)
        x[:, :, k] = size
    out = mla_bmm_w4(x.to(dev()), w4, scales)
    _done()
    ref, mass = so.bmm_w4(to_np(x), w4.cpu().numpy(), to_np(scales))
    _bf16(out, ref, "out", mass * K * 2.0 ** -24)


@pytest.mark.parametrize("T", [1, 17, 64])
def test_w4_weights_of_zero_give_zero(T):
    w4 = torch.full((1, 33, 256), 0x88, dtype=torch.uint8, device=dev())
    scales = torch.ones((1, 33, 4), dtype=torch.bfloat16, device=dev())
    x = gen.randn_bf16((T, 1, 512), torch.Generator().manual_seed(2)).to(dev())
    assert not mla_bmm_w4(x, w4, scales).any()


@pytest.mark.parametrize("T", TOKENS)
def test_w4_rows_of_any_size(T):
    """Tokens of 2^-110 to 2^100: each to the bound of its own terms."""
    g = torch.Generator().manual_seed(T)
    H, N, K = 2, 40, 256
    w4, scales = _w4(H, N, K, 64, True, g)
    x = gen.randn_bf16((T, H, K), g)
    size = torch.tensor([2.0 ** -110, 2.0 ** -90, 2.0 ** -74, 1.0, 2.0 ** 50, 2.0 ** 100])
    x = (x.float() * size[torch.arange(T * H).view(T, H, 1) % 6]).to(torch.bfloat16)
    scales[:, :, 0] *= 2.0 ** 10         # out of the smallest rows stays a normal number
    out = mla_bmm_w4(x.to(dev()), w4, scales)
    _done()
    ref, mass = so.bmm_w4(to_np(x), w4.cpu().numpy(), to_np(scales))
    _bf16(out, ref, "out", mass * K * 2.0 ** -24)


@pytest.mark.parametrize("N", [200, 4500, 4700])       # k cut eight, four and two ways
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("T", TOKENS)
def test_w4_whole_numbers_are_exact(T, group, N):
    """Whole numbers in x and powers of two as scales: every sum is a multiple of 1/4 below 2^22, exact in fp32 in any order,
    so out is the exact value rounded once."""
    g = torch.Generator(device=dev()).manual_seed(N + T + group)
    K = 16384
    w4 = torch.randint(0, 256, (1, N, K // 2), generator=g, device=dev(), dtype=torch.uint8)
    scales = torch.exp2(torch.randint(-2, 2, (1, N, K // group), generator=g, device=dev()).float()).to(torch.bfloat16)
    x = torch.randint(-8, 9, (T, 1, K), generator=g, device=dev()).to(torch.bfloat16)
    out = mla_bmm_w4(x, w4, scales)
    w = torch.stack([w4[0] & 15, w4[0] >> 4], -1).view(N, K).double() - 8
    w *= scales[0].double().repeat_interleave(group, 1)
    ref = x[:, 0].double() @ w.T
    assert torch.equal(out[:, 0].double(), ref.to(torch.float32).to(torch.bfloat16).double())


def test_w4_most_columns_of_several_tokens_in_wider_rows():
    """2^31 - 1 columns, eight a store, in rows of 2^31: the last group is cut at its seventh column."""
    g, d, T, N = torch.Generator().manual_seed(8), dev(), 9, 2 ** 31 - 1
    w4 = torch.empty((1, N, 16), dtype=torch.uint8, device=d).random_()
    scales = torch.empty((1, N, 1), dtype=torch.bfloat16, device=d).uniform_(0.5, 1.5)
    x = gen.randn_bf16((T, 1, 32), g).to(d)
    rows = torch.full((T, 1, N + 1), 3.0, dtype=torch.bfloat16, device=d)
    out = mla_bmm_w4(x, w4, scales, out=rows[:, :, :N])
    _done()
    assert (rows[:, :, N] == 3).all()
    at = torch.cat([torch.arange(300), torch.randint(0, N, (1000,), generator=g), torch.arange(N - 300, N)]).to(d)
    ref, mass = so.bmm_w4(to_np(x), w4[:, at].cpu().numpy(), to_np(scales[:, at]))
    _bf16(out[:, :, at], ref, "out", mass * 32 * 2.0 ** -24)
    del w4, scales, rows, out
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------------------------------
# RMS norm
# ---------------------------------------------------------------------------------------------
@pytest.mark.parametrize("D", [64, 1535, 8192, 20000])
def test_norm_keeps_the_small_values_of_huge_rows(D):
    """2^-50 next to 2^70 is a normal number of the output, to the output's precision."""
    g = torch.Generator().manual_seed(D)
    x = torch.randn((3, D), generator=g)
    x[0] *= 2.0 ** 70
    x[1] *= 2.0 ** 100
    x[2] *= 2.0 ** 120
    x[:, ::2] = torch.randn((3, (D + 1) // 2), generator=g) * 2.0 ** -50
    w = torch.full((D,), 2.0 ** 60, dtype=torch.bfloat16, device=dev())
    _check_norm(3, D, residual=False, x=x.to(torch.bfloat16).to(dev()), w=w)


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
@pytest.mark.parametrize("D", [64, 500, 1535, 8192, 20000])
def test_norm_rows_far_below_one(D, e4m3):
    """Without an eps, or with one as small as the rows' squares, a row of any size is normed."""
    g = torch.Generator().manual_seed(D)
    sizes = [2.0 ** -62, 2.0 ** -72, 2.0 ** -76, 2.0 ** -100, 2.0 ** -122, 2.0 ** -126]
    x = torch.randn((len(sizes), D), generator=g) * torch.tensor(sizes)[:, None]
    x[4, : D // 2] = 0
    x[5] = 2.0 ** -130                   # below the smallest normal number
    x = x.to(torch.bfloat16).to(dev())
    w = (1 + 0.3 * torch.randn(D, generator=g)).to(torch.bfloat16).to(dev())
    for eps in (0.0, float(np.float32(2.0 ** -140)), float(np.float32(2.0 ** -125))):
        _check_norm(len(sizes), D, residual=False, e4m3=e4m3, eps=eps, x=x, w=w)


# ---------------------------------------------------------------------------------------------
# cache append
# ---------------------------------------------------------------------------------------------
def _append(c, w, eps, e4m3, scale=1.0):
    d, T = dev(), c.shape[0]
    pe = torch.zeros((T, 64), dtype=torch.bfloat16, device=d)
    cache = torch.zeros((1, T, 576), device=d).to(torch.float8_e4m3fn if e4m3 else torch.bfloat16)
    at = torch.arange(T, dtype=torch.int32, device=d)
    mla_kv_append(c.to(d), pe, at, at, gen.rope_cos_sin(T).to(d), cache, scale, norm_weight=None if w is None else w.to(d), eps=eps)
    _done()
    return cache[0, :, :512]


def test_append_keeps_the_small_values_of_huge_latents():
    g = torch.Generator().manual_seed(32)
    c = torch.randn((3, 512), generator=g) * torch.tensor([2.0 ** 62, 2.0 ** 70, 2.0 ** 120])[:, None]
    c[:, ::2] = torch.randn((3, 256), generator=g) * 2.0 ** -64
    c = c.to(torch.bfloat16)
    w = torch.full((512,), 2.0 ** 70, dtype=torch.bfloat16)
    _bf16(_append(c, w, 1e-6, False), so.rms_norm(to_np(c), to_np(w), 1e-6)[0], "latents")


@pytest.mark.parametrize("e4m3", [False, True], ids=["bf16", "e4m3"])
def test_append_norms_latents_far_below_one(e4m3):
    g = torch.Generator().manual_seed(31)
    sizes = [2.0 ** -62, 2.0 ** -72, 2.0 ** -76, 2.0 ** -100, 1.0, 2.0 ** -126, 2.0 ** 80]
    c = torch.randn((len(sizes), 512), generator=g) * torch.tensor(sizes)[:, None]
    c[5] = 2.0 ** -130
    c = c.to(torch.bfloat16)
    w = (1 + 0.3 * torch.randn(512, generator=g)).to(torch.bfloat16)
    scale = 0.021 if e4m3 else 1.0
    s = float(np.float32(scale))
    for eps in (0.0, float(np.float32(2.0 ** -140))):
        ref = so.rms_norm(to_np(c), to_np(w), eps)[0]
        got = _append(c, w, eps, e4m3, scale)
        if e4m3:
            _within(torch.from_numpy(to_np(got) * s), ref, np.abs(ref) * (E4M3 + ARITH) + s * 2.0 ** -10, "latents")
        else:
            _bf16(got, ref, "latents")


def test_append_next_to_a_nan_or_an_infinity_rounds_to_nearest():
    """1.3671875 / 0.109375 is 12.5, between the codes of 12 and 13: to even, whatever else the row holds."""
    c = torch.full((4, 512), 1.3671875)
    c[1, 3::8], c[2, 6::8], c[3, 1::8] = float("nan"), float("inf"), -3e38
    got = to_np(_append(c.to(torch.bfloat16), None, 0.0, True, 0.109375))
    want = np.full((4, 512), 12.0)
    want[1, 3::8], want[2, 6::8], want[3, 1::8] = np.nan, 448, -448
    np.testing.assert_array_equal(got, want)


def test_append_norms_far_latents_in_place():
    """Rows that are read twice, written over themselves: the same bits as into a buffer of their own."""
    g, d, T = torch.Generator().manual_seed(33), dev(), 5
    kv = torch.randn((T, 576), generator=g)
    kv[0] *= 2.0 ** 80
    kv[3] *= 2.0 ** -90
    kv, w = kv.to(torch.bfloat16).to(d), (1 + 0.3 * torch.randn(512, generator=g)).to(torch.bfloat16).to(d)
    at, cs, rows = torch.arange(T, dtype=torch.int32, device=d), gen.rope_cos_sin(T).to(d), torch.empty_like(kv)
    one, two = torch.zeros((1, T, 576), dtype=torch.bfloat16, device=d), torch.zeros((1, T, 576), dtype=torch.bfloat16, device=d)
    mla_kv_append(kv[:, :512], kv[:, 512:], at, at, cs, one, norm_weight=w, eps=0.0, kv_out=rows)
    mla_kv_append(kv[:, :512], kv[:, 512:], at, at, cs, two, norm_weight=w, eps=0.0, kv_out=kv)
    _done()
    assert torch.equal(one, two) and torch.equal(rows, kv) and torch.equal(one[0], kv)


@pytest.mark.parametrize("T", [1, 9, 64])
def test_w4_smallest_numbers_in_x(T):
    """x below the smallest normal number, scales that bring out back up."""
    g = torch.Generator().manual_seed(50 + T)
    w4, scales = _w4(1, 64, 512, 64, True, g)
    x = (torch.randn((T, 1, 512), generator=g) * 2.0 ** -128).to(torch.bfloat16)
    out = mla_bmm_w4(x.to(dev()), w4, scales * 2.0 ** 60)
    _done()
    ref, mass = so.bmm_w4(to_np(x), w4.cpu().numpy(), to_np(scales * 2.0 ** 60))
    _bf16(out, ref, "out", mass * 512 * 2.0 ** -24)
