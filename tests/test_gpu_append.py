"""mla_cache_append (norm, rotation, quantisation, scatter) against the same
formulas in fp64, for the four cache row formats.

Tolerances.  The kernel forms y (normalised, rotated) in fp32: three rounded
factors at most for the norm (each 2^-24) and, for the rotation, an angle
reduced in fp64 whose sine and cosine carry about 2^-23, so
|y - y64| <= SLACK * (|a| + |b|) with (a, b) the rotated pair (twice |y| for
other dims) and SLACK = 2^-21.  One rounding follows: half a step, 2^-8 of the
value for bf16, 2^-4 (at least 2^-10) for an E4M3 code, and half the gap
between neighbours for E2M1.
"""
import numpy as np
import pytest
import torch

import oracle
from mla_paged_kv_03_b200 import binding as B
from parity_util import assert_lse_close, assert_out_close

pytestmark = pytest.mark.gpu

SLACK = 2.0 ** -21
FORMATS = ["bf16", "656", "528", "288"]
E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def width(fmt):
    return 576 if fmt in ("bf16", "656") else 512


def row_bytes(fmt):
    return 1152 if fmt == "bf16" else int(fmt)


def make_cache(fmt, blocks, dev, gen):
    raw = torch.randint(0, 256, (blocks, 64, row_bytes(fmt)), generator=gen, dtype=torch.uint8)
    if fmt == "bf16":
        return raw.view(torch.bfloat16).view(blocks, 64, 1, 576).to(dev)
    return raw.to(dev)


def raw_rows(cache):
    return cache.cpu().contiguous().view(torch.uint8).view(-1, cache.shape[-1] *
                                                           cache.element_size())


def expected(kv, positions, gain, eps, base):
    """(y in fp64, the size its fp32 error is relative to)."""
    y = kv.cpu().double()
    n, d = y.shape
    if gain is not None:
        rms = torch.sqrt(y[:, :512].pow(2).mean(1, keepdim=True) + eps)
        y[:, :512] = y[:, :512] / rms * gain.cpu().double()
    size = 2 * y.abs()
    if positions is not None:
        k = torch.arange(32, dtype=torch.float64)
        angle = positions.cpu().double()[:, None] * base ** (-2 * k / 64)
        a, b = y[:, d - 64::2].clone(), y[:, d - 63::2].clone()
        y[:, d - 64::2] = a * torch.cos(angle) - b * torch.sin(angle)
        y[:, d - 63::2] = a * torch.sin(angle) + b * torch.cos(angle)
        both = a.abs() + b.abs()
        size[:, d - 64::2] = both
        size[:, d - 63::2] = both
    return y, size


def e4m3(b):
    return b.contiguous().view(torch.float8_e4m3fn).double()


def bf16_once(x):
    """fp64 -> the nearest bf16 (ties to even), as fp64.  torch rounds to fp32 on the way: the
    product -224 * 0x1.2edb6ep-7 = -0x1.0900004p+1 of a code and an fp32 scale lies above the tie
    0x1.09p+1 and goes to 0x1.0ap+1, but its fp32 rounding is the tie, which goes to 0x1.08p+1."""
    step = torch.exp2((torch.frexp(x)[1].clamp(min=-125) - 8).double())
    return torch.round(x / step) * step


def check_bf16(got, y, size, what):
    err = (got.double() - y).abs()
    bound = y.abs() * 2.0 ** -8 * (1 + 2.0 ** -14) + SLACK * size
    assert (err <= bound).all(), f"{what}: {(err > bound).sum()} off, worst {err.max():.3e}"


def check_codes(value, y, size, scale, half, what):
    """value (of the codes) within half a step of y / scale; `half` of |y / scale|."""
    v = y / scale
    bound = half(v.abs()) + SLACK * size / scale
    err = (value - v.clamp(-448, 448)).abs()
    assert (err <= bound).all(), f"{what}: {(err > bound).sum()} codes off"


def check_rows(fmt, raw, y, size, stands=None):
    """The written cache rows (bytes [m, row_bytes]) against y [m, d]."""
    m = y.shape[0]
    if fmt == "bf16":
        check_bf16(raw.view(torch.bfloat16), y, size, "row")
        if stands is not None:
            assert torch.equal(stands, raw.view(torch.bfloat16))
        return
    if fmt in ("656", "528"):
        per = 128 if fmt == "656" else 32
        amax = y[:, :512].reshape(m, 512 // per, per).abs().amax(2)
        if fmt == "656":
            scale = raw[:, 512:528].contiguous().view(torch.float32).double()
            want = torch.where(amax > 0, amax / 448, 1.0)
            assert ((scale - want).abs() <= 2 * SLACK * want).all()
        else:
            scale = torch.exp2(raw[:, 512:].double() - 127)
            lo, hi = amax * (1 - 2 * SLACK) / 448, amax * (1 + 2 * SLACK) / 448
            least = 2.0 ** -127
            ok = ((scale >= lo) & (scale < 2 * hi)) | ((scale == least) & (hi <= least))
            ok |= (amax == 0) & (scale == 1)
            assert ok.all()
        scale = scale.repeat_interleave(per, 1)
        value = e4m3(raw[:, :512])
        check_codes(value, y[:, :512], size[:, :512], scale,
                    lambda v: (v * 2.0 ** -4).clamp(min=2.0 ** -10), fmt)
        if fmt == "656":
            check_bf16(raw[:, 528:].contiguous().view(torch.bfloat16), y[:, 512:], size[:, 512:],
                       "rope")
    else:
        amax = y.reshape(m, 32, 16).abs().amax(2)
        scale = e4m3(raw[:, 256:])
        want = (amax / 6).clamp(max=448)
        ok = (scale - want).abs() <= (want * 2.0 ** -4).clamp(min=2.0 ** -10) + 2 * SLACK * want
        tiny = amax / 6 <= 2.0 ** -10 * (1 + 2 * SLACK)  # rounds to 0, or is 0
        assert (ok | (tiny & (scale == 1))).all()
        scale = scale.repeat_interleave(16, 1)
        code = torch.stack([raw[:, :256] & 15, raw[:, :256] >> 4], 2).reshape(m, 512).long()
        value = E2M1[code & 7] * torch.where(code >= 8, -1.0, 1.0)
        v = (y / scale).clamp(-6, 6)
        bound = torch.where(v.abs() < 2, 0.25, torch.where(v.abs() < 4, 0.5, 1.0))
        assert ((value - v).abs() <= bound + SLACK * size / scale).all()
    if stands is not None:
        # code * scale is exact in fp64: the row is its bf16 rounding
        assert torch.equal(stands[:, :512].double(), bf16_once(value * scale))
        if fmt == "656":
            assert torch.equal(stands[:, 512:], raw[:, 528:].contiguous().view(torch.bfloat16))


def run(fmt, n, *, norm=True, rope=True, stride=None, rows=True, pad=(), seed=0, blocks=None,
        values=None, gain=None, positions=None, base=1e4, eps=1e-6):
    dev = torch.device("cuda")
    g = torch.Generator().manual_seed(seed)
    d = width(fmt)
    wide = torch.randn((n, stride or d), generator=g)
    wide = (wide * torch.exp(0.5 * torch.randn(wide.shape[1], generator=g))).to(torch.bfloat16)
    kv = wide[:, wide.shape[1] - d:]
    if values is not None:
        kv[...] = values
    if norm and gain is None:
        gain = 1 + 0.1 * torch.randn(512, generator=g)
    if rope and positions is None:
        positions = torch.randint(0, 1 << 17, (n,), generator=g, dtype=torch.int32)
    blocks = blocks or n // 64 + 3
    cache = make_cache(fmt, blocks, dev, g)
    before = raw_rows(cache).clone()
    slots = torch.randperm(blocks * 64, generator=g)[:n].to(torch.int32)
    for i in pad:
        slots[i] = -1
    out = torch.full((n, d), 7.0, dtype=torch.bfloat16, device=dev) if rows else None
    kv_dev = wide.to(dev)[:, wide.shape[1] - d:]
    B.mla_cache_append(kv_dev, slots.to(dev), cache,
                       positions=positions.to(dev) if rope else None,
                       norm_gain=gain.to(dev) if norm else None, eps=eps, rope_base=base, rows=out)
    torch.cuda.synchronize()
    assert B.device_status() == 0
    after = raw_rows(cache)
    y, size = expected(kv, positions if rope else None, gain if norm else None, eps, base)
    live = slots >= 0
    at = slots[live].long()
    check_rows(fmt, after[at], y[live], size[live], out.cpu()[live] if rows else None)
    untouched = torch.ones(blocks * 64, dtype=torch.bool)
    untouched[at] = False
    assert torch.equal(after[untouched], before[untouched])
    if rows and not live.all():
        assert (out.cpu()[~live] == 7.0).all()
    return after[at], out


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", [1, 7, 64, 1001, 9000])
def test_append_sizes(fmt, n):
    run(fmt, n, seed=n)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("norm,rope", [(False, False), (True, False), (False, True)])
def test_append_without_norm_or_rotation(fmt, norm, rope):
    run(fmt, 130, norm=norm, rope=rope, seed=3)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("size,eps", [(1e25, 1e-6), (3e37, 0.0), (1e-13, 0.0), (1e-28, 0.0),
                                      (1e-37, 0.0)])
def test_norm_of_rows_whose_squares_leave_fp32(fmt, size, eps):
    g = torch.Generator().manual_seed(9)
    x = (torch.rand((40, width(fmt)), generator=g) + 0.5) * size
    # (the dims behind the norm's 512 keep an ordinary size)
    x[:, 512:] = torch.randn((40, width(fmt) - 512), generator=g)
    run(fmt, 40, values=x.to(torch.bfloat16), eps=eps, seed=10)


@pytest.mark.parametrize("fmt", ["656", "528", "288"])
@pytest.mark.parametrize("rope", [False, True])
def test_codes_are_those_of_fp64(fmt, rope):
    """The codes equal the definition's in fp64 (656-byte rows: with the unrounded absmax/448),
    except for rotated dims that nearly cancel and values within 2^-45 of a border."""
    n, d, gen = 6000, width(fmt), torch.Generator().manual_seed(31)
    kv = torch.randn((n, d), generator=gen).to(torch.bfloat16)
    gain = 1 + 0.1 * torch.randn(512, generator=gen)
    positions = torch.randint(0, 1 << 17, (n,), generator=gen, dtype=torch.int32)
    cache = make_cache(fmt, n // 64 + 1, "cuda", gen)
    B.mla_cache_append(kv.cuda(), torch.arange(n, dtype=torch.int32, device="cuda"), cache,
                       positions=positions.cuda() if rope else None, norm_gain=gain.cuda())
    raw = raw_rows(cache)[:n]
    y, size = expected(kv, positions if rope else None, gain, 1e-6, 1e4)
    y, size = y[:, :512], size[:, :512]
    per = {"656": 128, "528": 32, "288": 16}[fmt]
    g = y.reshape(n, 512 // per, per)
    amax = g.abs().amax(2, keepdim=True)

    def e4m3_step(v):
        return torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)

    def e2m1_step(v):
        return torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0)).double()

    if fmt == "288":
        scale = amax / 6
        scale = torch.round(scale / e4m3_step(scale)) * e4m3_step(scale)
        assert torch.equal(e4m3(raw[:, 256:]), scale[..., 0])
        code = torch.stack([raw[:, :256] & 15, raw[:, :256] >> 4], 2).reshape(n, 512).long()
        got = E2M1[code & 7] * torch.where(code >= 8, -1.0, 1.0)
        step, most = e2m1_step, 6.0
    else:
        scale = amax / 448
        if fmt == "528":
            scale = torch.exp2(torch.ceil(torch.log2(scale)))
            assert torch.equal(torch.exp2(raw[:, 512:].double() - 127), scale[..., 0])
        got = e4m3(raw[:, :512])
        step, most = e4m3_step, 448.0
    v = (g / scale).reshape(n, 512)
    steps = v / step(v)
    want = (torch.round(steps) * step(v)).clamp(-most, most)
    border = (steps - torch.floor(steps) - 0.5).abs() < 2.0 ** -45 * steps.abs()
    cancels = y.abs() < size / 16  # size: 2 |y|, or |a| + |b| of a rotated pair
    wrong = (got != want) & ~border & ~cancels
    assert not wrong.any(), f"{int(wrong.sum())} codes differ"


@pytest.mark.parametrize("rope", [False, True])
def test_528_scales_next_to_a_power_of_two(rope):
    """Group maxima a few 2^-25 off 448 2^e, which fp32 rounds onto it: the scale is 2^e up to
    there and 2^(e+1) above."""
    wrong, sides = 0, set()
    for seed in range(40):
        gen = torch.Generator().manual_seed(seed)
        x = (0.25 * torch.randn((1, 512), generator=gen).clamp(-3, 3)).to(torch.bfloat16)
        x[:, ::32], x[:, 1::32] = 1.0, 0.0  # the maximum of each group; the dim it rotates with
        pos = torch.randint(0, 1 << 17, (1,), generator=gen, dtype=torch.int32) if rope else None
        # the gains that bring those next to 3.5, up to two steps of fp32 away
        y, _ = expected(x, pos, torch.ones(512), 0.0, 1e4)
        top = torch.maximum(y[0, ::32].abs(), y[0, 1::32].abs())
        gain = torch.ones(512)
        near = (3.5 / top).float()
        gain[::32] = (near.view(torch.int32) + torch.arange(16, dtype=torch.int32) % 5 - 2).view(
            torch.float32)
        y, _ = expected(x, pos, gain, 0.0, 1e4)
        amax = y.reshape(16, 32).abs().amax(1)
        assert ((amax / 3.5 - 1).abs() < 2.0 ** -21).all()
        sides |= {bool(v) for v in amax > 3.5}
        cache = make_cache("528", 1, "cuda", gen)
        B.mla_cache_append(x.cuda(), torch.zeros(1, dtype=torch.int32, device="cuda"), cache,
                           positions=pos.cuda() if rope else None, norm_gain=gain.cuda(), eps=0.0)
        got = raw_rows(cache)[0, 512:].int() - 127
        wrong += int((got != torch.where(amax > 3.5, -6, -7)).sum())
    assert len(sides) == 2 and wrong == 0, f"{wrong} scales differ"


@pytest.mark.parametrize("fmt", ["656", "528", "288"])
def test_codes_of_bf16_values_are_the_definitions(fmt):
    """Without norm and rotation the values are bf16, products with 448 are exact in fp64 and a
    quotient on a rounding border is formed exactly: every code has one value, ties to even."""
    n, d, gen = 6000, width(fmt), torch.Generator().manual_seed(37)
    kv = torch.randn((n, d), generator=gen).to(torch.bfloat16)
    kv[:1000] = (kv[:1000].float() * 8).round().to(torch.bfloat16)  # maxima that 7 divides
    kv[5000:] = (kv[5000:].float() * 2.0 ** -100).to(torch.bfloat16)
    if fmt == "656":
        kv[5500:, :512] = (kv[5500:, :512].float() * 2.0 ** -12).to(torch.bfloat16)
        kv[5800:, :512] = (kv[5800:, :512].float() * 2.0 ** -9).to(torch.bfloat16)
    cache = make_cache(fmt, n // 64 + 1, "cuda", gen)
    B.mla_cache_append(kv.cuda(), torch.arange(n, dtype=torch.int32, device="cuda"), cache)
    raw = raw_rows(cache)[:n]
    y = kv[:, :512].double()
    per = {"656": 128, "528": 32, "288": 16}[fmt]
    g = y.reshape(n, 512 // per, per)
    amax = g.abs().amax(2, keepdim=True)
    if fmt == "288":
        step = torch.exp2(torch.floor(torch.log2((amax / 6).clamp(min=2.0 ** -6))) - 3)
        scale = torch.round(amax / 6 / step) * step
        scale = torch.where(scale > 0, scale, 1.0)
        assert torch.equal(e4m3(raw[:, 256:]), scale[..., 0])
        v = (g / scale).reshape(n, 512)
        step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0)).double()
        code = torch.stack([raw[:, :256] & 15, raw[:, :256] >> 4], 2).reshape(n, 512).long()
        got = E2M1[code & 7] * torch.where(code >= 8, -1.0, 1.0)
    else:
        if fmt == "528":
            scale = torch.exp2(raw[:, 512:].double() - 127)[..., None]
            assert ((scale >= amax / 448) & (scale < amax / 224)).all()
            v = g / scale
        else:  # the stored scale counts below fp32's normal range
            scale = raw[:, 512:528].contiguous().view(torch.float32).double()[..., None]
            least = amax < 448 * 2.0 ** -126
            assert least.any() and not least.all()
            v = torch.where(least, g / scale, g * 448 / amax).clamp(-448, 448)
        v = v.reshape(n, 512)
        step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
        got = e4m3(raw[:, :512])
    assert (v / step == torch.floor(v / step) + 0.5).any()  # ties are among them
    want = torch.round(v / step) * step
    assert torch.equal(got, want), f"{int((got != want).sum())} codes differ"


@pytest.mark.parametrize("fmt", ["528", "288"])
def test_codes_of_rotated_values_without_norm(fmt):
    """Only the last 64 of the 512 dims are rotated (exceptions as with a norm)."""
    n, gen = 6000, torch.Generator().manual_seed(43)
    kv = torch.randn((n, 512), generator=gen).to(torch.bfloat16)
    positions = torch.randint(0, 1 << 17, (n,), generator=gen, dtype=torch.int32)
    cache = make_cache(fmt, n // 64 + 1, "cuda", gen)
    B.mla_cache_append(kv.cuda(), torch.arange(n, dtype=torch.int32, device="cuda"), cache,
                       positions=positions.cuda())
    raw = raw_rows(cache)[:n]
    y, size = expected(kv, positions, None, 0.0, 1e4)
    per, most = (32, 448.0) if fmt == "528" else (16, 6.0)
    g = y.reshape(n, 512 // per, per)
    amax = g.abs().amax(2, keepdim=True)
    if fmt == "528":
        scale = torch.exp2(torch.ceil(torch.log2(amax / 448)))
        assert torch.equal(torch.exp2(raw[:, 512:].double() - 127), scale[..., 0])
        got = e4m3(raw[:, :512])
    else:
        step = torch.exp2(torch.floor(torch.log2((amax / 6).clamp(min=2.0 ** -6))) - 3)
        scale = torch.round(amax / 6 / step) * step
        assert torch.equal(e4m3(raw[:, 256:]), scale[..., 0])
        code = torch.stack([raw[:, :256] & 15, raw[:, :256] >> 4], 2).reshape(n, 512).long()
        got = E2M1[code & 7] * torch.where(code >= 8, -1.0, 1.0)
    v = (g / scale).reshape(n, 512)
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    if fmt == "288":
        step = torch.where(v.abs() < 2, 0.5, torch.where(v.abs() < 4, 1.0, 2.0)).double()
    want = (torch.round(v / step) * step).clamp(-most, most)
    steps = v / step
    unsure = (steps - torch.floor(steps) - 0.5).abs() < 2.0 ** -45 * steps.abs()
    unsure |= y.abs() < size / 16
    unsure[:, :448] = False  # exact values
    assert ((got == want) | unsure).all(), f"{int(((got != want) & ~unsure).sum())} codes differ"


@pytest.mark.parametrize("fmt", FORMATS)
def test_append_strided_rows_padding_and_no_rows_output(fmt):
    run(fmt, 77, stride=width(fmt) + 520, pad=(0, 5, 76), seed=4)
    run(fmt, 3, pad=(0, 1, 2), seed=5)
    run(fmt, 65, rows=False, seed=6)


@pytest.mark.parametrize("n", [1, 2])
def test_append_rows_far_apart(n):
    # the last token of sequences whose hidden states lie 2^32 values apart
    dev = torch.device("cuda")
    stride = (1 << 32) + 8
    wide = torch.empty((n - 1) * stride + 576, dtype=torch.bfloat16, device=dev)
    kv = wide.as_strided((n, 576), (stride, 1))
    kv[:] = torch.randn((n, 576), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    cache = torch.zeros((1, 64, 1, 576), dtype=torch.bfloat16, device=dev)
    B.mla_cache_append(kv, torch.arange(n, dtype=torch.int32, device=dev), cache)
    assert torch.equal(cache[0, :n, 0], kv) and (cache[0, n:] == 0).all()
    # (one row's stride does not count, whatever it is)
    one = wide.as_strided((1, 576), (7, 1))
    B.mla_cache_append(one, torch.full((1,), 9, dtype=torch.int32, device=dev), cache)
    assert torch.equal(cache[0, 9, 0], one[0])


@pytest.mark.parametrize("fmt", FORMATS)
def test_append_a_cache_past_2_gib(fmt):
    # slots whose byte offsets pass 32 bits
    dev = torch.device("cuda")
    rb, d = row_bytes(fmt), width(fmt)
    blocks = (5 << 30) // (rb * 64)
    cache = torch.zeros((blocks, 64, rb), dtype=torch.uint8, device=dev)
    view = cache.view(torch.bfloat16).view(blocks, 64, 1, 576) if fmt == "bf16" else cache
    slots = torch.tensor([blocks * 64 - 1, 0, (1 << 31) // rb + 1, (1 << 32) // rb + 1],
                         dtype=torch.int32)
    kv = torch.randn((4, d), generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    B.mla_cache_append(kv.to(dev), slots.to(dev), view)
    torch.cuda.synchronize()
    y, size = expected(kv, None, None, 0.0, 1e4)
    check_rows(fmt, cache.view(-1, rb)[slots.long().to(dev)].cpu(), y, size)
    assert B.device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_append_extreme_values(fmt):
    # zero groups, tiny groups (scales at their lower end), large groups, one outlier
    n = 8
    values = torch.zeros((n, width(fmt)))
    g = torch.Generator().manual_seed(9)
    values[1] = torch.randn(width(fmt), generator=g) * 1e-30
    values[2] = torch.randn(width(fmt), generator=g) * 1e30
    values[3, 100] = 5.0
    values[4] = torch.randn(width(fmt), generator=g) * 1e-6
    values[5] = 448.0
    values[6] = -3.0
    values[7, ::2] = torch.randn(width(fmt) // 2, generator=g)
    if fmt == "288":
        values[2] = 0  # past 6 * 448 the FP4 row saturates
        values[5] = 2688.0
    run(fmt, n, norm=False, rope=False, values=values.to(torch.bfloat16), seed=9)
    values[1] = 1e-3
    values[2] = 1e3
    run(fmt, n, norm=True, rope=True, values=values.to(torch.bfloat16), seed=10)


@pytest.mark.parametrize("base", [1e4, 5e5, 1.0])
def test_append_far_and_negative_positions(base):
    pos = torch.tensor([0, 1, -1, 1 << 20, (1 << 24) + 1, (1 << 31) - 1, -(1 << 31)],
                       dtype=torch.int32)
    # the angle itself is formed in fp64: 2^31 * 2^-53 turns of error at most
    run("bf16", 7, positions=pos, base=base, seed=11)
    run("528", 7, positions=pos, base=base, seed=12)


def test_append_bad_slots_are_skipped_and_recorded():
    dev = torch.device("cuda")
    cache = torch.zeros((2, 64, 1, 576), dtype=torch.bfloat16, device=dev)
    kv = torch.full((4, 576), float("nan"), dtype=torch.bfloat16, device=dev)
    kv[3] = 2.0
    slots = torch.tensor([128, -5, 2 ** 31 - 1, 127], dtype=torch.int32, device=dev)
    B.mla_cache_append(kv, slots, cache)
    assert B.device_status() >> 16 == B.MLA_DEVERR_BAD_INDEX
    want = torch.zeros((128, 576), dtype=torch.bfloat16, device=dev)
    want[127] = 2.0
    assert torch.equal(cache.view(128, 576), want)


def test_int64_slots_past_int32_are_out_of_range():
    # 2^32 + 5 is not slot 5
    dev = torch.device("cuda")
    kv = torch.ones((6, 576), dtype=torch.bfloat16, device=dev)
    kv[5] = 2.0
    cache = torch.zeros((2, 64, 1, 576), dtype=torch.bfloat16, device=dev)
    B.mla_cache_append(kv, torch.tensor([-1, -2 ** 32 + 5, -2 ** 63, -7, -2 ** 31 - 2 ** 32, 127],
                                        device=dev), cache)
    assert B.device_status() == 0  # padding
    B.mla_cache_append(kv, torch.tensor([2 ** 32 + 5, 2 ** 31, 2 ** 63 - 1, 2 ** 32, -1, 127],
                                        device=dev), cache)
    assert B.device_status() >> 16 == B.MLA_DEVERR_BAD_INDEX
    want = torch.zeros((128, 576), dtype=torch.bfloat16, device=dev)
    want[127] = 2.0
    assert torch.equal(cache.view(128, 576), want)


@pytest.mark.parametrize("fmt", FORMATS)
def test_append_keeps_non_finite_rows_apart(fmt):
    dev = torch.device("cuda")
    g = torch.Generator().manual_seed(2)
    kv = torch.randn((3, width(fmt)), generator=g).to(torch.bfloat16)
    slots = torch.tensor([3, 70, 9], dtype=torch.int32, device=dev)
    caches = []
    for bad in (0.5, float("nan"), float("inf")):
        kv[1, 40] = bad
        cache = torch.zeros((2, 64, row_bytes(fmt)), dtype=torch.uint8, device=dev)
        view = cache.view(torch.bfloat16).view(2, 64, 1, 576) if fmt == "bf16" else cache
        B.mla_cache_append(kv.to(dev), slots, view, norm_gain=torch.ones(512, device=dev))
        caches.append(cache.view(128, -1))
    others = [i for i in range(128) if i != 70]
    assert torch.equal(caches[0][others], caches[1][others])
    assert torch.equal(caches[0][others], caches[2][others])
    assert B.device_status() == 0


def test_append_side_stream_and_graph_replay():
    dev = torch.device("cuda")
    g = torch.Generator().manual_seed(3)
    kv = torch.randn((40, 576), generator=g).to(torch.bfloat16).to(dev)
    slots = torch.randperm(256, generator=g)[:40].to(torch.int32).to(dev)
    pos = torch.arange(40, dtype=torch.int32, device=dev)
    gain = torch.ones(512, device=dev)
    want = torch.zeros((4, 64, 656), dtype=torch.uint8, device=dev)
    got = want.clone()
    B.mla_cache_append(kv, slots, want, positions=pos, norm_gain=gain)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        B.mla_cache_append(kv, slots, got, positions=pos, norm_gain=gain)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.mla_cache_append(kv, slots, got, positions=pos, norm_gain=gain)
    kv.copy_(kv.flip(0))
    graph.replay()
    B.mla_cache_append(kv, slots, want, positions=pos, norm_gain=gain)
    torch.cuda.synchronize()
    assert torch.equal(got, want)


def test_appended_rows_feed_the_dense_and_sparse_decodes():
    # prompts appended token by token positions, then decoded; the oracle reads
    # the very cache that the append wrote
    dev = torch.device("cuda")
    g = torch.Generator().manual_seed(5)
    lengths = [70, 129]
    n = sum(lengths)
    kv = torch.randn((n, 576), generator=g).to(torch.bfloat16)
    table = torch.tensor([[4, 1, -1], [0, 5, 2]], dtype=torch.int32)
    slots, pos = [], []
    for b, length in enumerate(lengths):
        for t in range(length):
            slots.append(int(table[b, t // 64]) * 64 + t % 64)
            pos.append(t)
    slots = torch.tensor(slots, dtype=torch.int32)
    pos = torch.tensor(pos, dtype=torch.int32)
    gain = 1 + 0.1 * torch.randn(512, generator=g)
    q = torch.randn((2, 1, 16, 576), generator=g).to(torch.bfloat16)
    sl = torch.tensor(lengths, dtype=torch.int32)
    scale = 1.0 / 24
    dense = torch.zeros((6, 64, 1, 576), dtype=torch.bfloat16, device=dev)
    B.mla_cache_append(kv.to(dev), slots.to(dev), dense, pos.to(dev), gain.to(dev))
    meta, ns, parts = B.mla_get_metadata(sl.to(dev), 16, 1)
    out, lse = B.mla_decode_fwd(q.to(dev), dense, table.to(dev), sl.to(dev), 512, meta, ns, parts)
    ro, rl = oracle.dense_decode(q, dense.cpu(), table, sl, 512, scale, causal=True)
    assert_out_close(out, ro)
    assert_lse_close(lse, rl)
    fp8 = torch.zeros((6, 64, 656), dtype=torch.uint8, device=dev)
    B.mla_cache_append(kv.to(dev), slots.to(dev), fp8, pos.to(dev), gain.to(dev))
    idx = torch.full((2, 1, 130), -1, dtype=torch.int32)
    idx[0, 0, :70] = slots[:70]
    idx[1, 0, :129] = slots[70:]
    out, lse = B.mla_sparse_decode(q.to(dev), fp8, idx.to(dev), 512, scale)
    ro, rl = oracle.sparse_decode(q, fp8.cpu(), idx, 512, scale)
    assert_out_close(out, ro)
    assert_lse_close(lse, rl)
    assert B.device_status() == 0


def test_append_rejects_wrong_shapes():
    dev = torch.device("cuda")
    cache = torch.zeros((2, 64, 528), dtype=torch.uint8, device=dev)
    kv = torch.zeros((3, 512), dtype=torch.bfloat16, device=dev)
    slots = torch.zeros(3, dtype=torch.int32, device=dev)
    bad = [dict(kv=torch.zeros((3, 576), dtype=torch.bfloat16, device=dev)),
           dict(kv=kv.float()), dict(slots=slots[:2]), dict(slots=slots.float()),
           dict(slots=slots.cpu()), dict(kcache=cache[..., :500]), dict(kcache=cache.int()),
           dict(kcache=cache.transpose(0, 1)), dict(positions=slots[:1]),
           dict(norm_gain=torch.ones(576, device=dev)), dict(rows=kv[:2]), dict(rows=kv.float())]
    for change in bad:
        args = dict(kv=kv, slots=slots, kcache=cache) | change
        with pytest.raises((ValueError, B.MLAError)):
            B.mla_cache_append(**args)
