"""Softmax weights far below a row's largest: sinks whose value is zero, blocks whose value
scale dwarfs the others', and scores so large that fp32 has no fractions left. Outputs then
come from weights that are 2^-17 to 2^-30 of the largest, and must be as exact as any."""
import math

import numpy as np
import pytest
import torch

import gqa_reference as ref
from test_gpu_gqa import DEV, E4, I8, Dev

pytestmark = pytest.mark.gpu

# Bits of f16's range that lie above a row's largest weight at least (gqa_attend.cu, gqa_tiles.cu).
LIFT = 11


def exact(c, sm, rows):
    """Rows of the attention in 64 bits with a bound of each output, from the kernels'
    roundings: a score's D-term fp32 sum is off by D * 2^-24 of sum |q k|, so a weight by twice
    that relatively; it is rounded to f16, half a step of 2^-11 relatively or, below f16's normal
    range, half of its smallest step: 2^-25 where the largest weight (times value scale) is 2^LIFT;
    the exponential adds 2^-21, the scale's logarithm and the maximum's rounding 2^-18 (scales
    within 2^40 of one); fp32 sums of n terms n * 2^-24; the output is rounded to bf16, 2^-8."""
    k, v = c.k.double(), c.v.double()
    for t, b, pos in c.tokens():
        if t not in rows or pos < 0:
            continue
        page, slot = c.block_table[b, torch.arange(pos + 1) // 64].long(), torch.arange(pos + 1) % 64
        for h in range(c.Hkv):
            code = v[page, h, slot].numpy()
            vs = c.v_scale[page, h].double().numpy()[:, None]
            kk = k[page, h, slot].numpy() * c.k_scale[page, h].double().numpy()[:, None]
            for hh in range(h * c.G, (h + 1) * c.G):
                q = c.q[t, hh].double().numpy()
                z = sm * (kk @ q)
                w = np.exp(z - z.max())[:, None]
                l = w.sum()
                out = (w * vs * code).sum(0) / l
                mag = (w * vs * np.abs(code)).sum(0) / l
                dots = sm * (np.abs(kk) @ np.abs(q)).max()
                rel = 2 * c.D * 2.0 ** -24 * dots + 2.0 ** -11 + 2.0 ** -21 + 2.0 ** -18 + (pos + 1) * 2.0 ** -24
                low = 2.0 ** -(25 + LIFT) * (w * vs).max() * np.abs(code).sum(0) / l
                yield t, hh, out, np.abs(out) * 2.0 ** -8 + (1 + 2.0 ** -8) * (2 * rel * mag + low), z.max() + math.log(l), rel


def check(c, sm, rows=None):
    d = Dev(c)
    out, lse = d.attend(sm)
    rows = set(range(c.T)) if rows is None else set(rows)
    got, le, n = out.double().cpu().numpy(), lse.double().cpu().numpy(), 0
    for t, hh, want, bound, want_lse, rel in exact(c, sm, rows):
        off = np.abs(got[t, hh] - want)
        assert (off <= bound).all(), (t, hh, float((off / bound).max()), float((off / np.abs(want)).max()))
        assert abs(le[t, hh] - want_lse) <= rel + 2.0 ** -20 + abs(want_lse) * 2.0 ** -22, (t, hh)
        n += 1
    assert n > 0
    return out, lse


# lens, new, H, Hkv, D: few rows (a warp's or a team's), and tiles of many rows; the last of each with several units a run
FEW = [([64], [1], 1, 1, 128), ([100, 128], [1, 2], 8, 2, 64), ([64, 40], [3, 4], 16, 1, 128), ([900] * 160, [1] * 160, 16, 8, 64)]
MANY = [([64, 60], [64, 60], 16, 1, 128), ([64], [64], 5, 1, 64), ([300] * 40, [40] * 40, 32, 8, 64)]


def sample(c, n=24):
    return range(0, c.T, max(1, c.T // n))


@pytest.mark.parametrize("dtype", [E4, I8], ids=["e4m3", "i8"])
@pytest.mark.parametrize("gap", [10.0, 17.0, 20.0])
@pytest.mark.parametrize("lens,new,H,Hkv,D", FEW + MANY)
def test_sink_with_a_zero_value(lens, new, H, Hkv, D, gap, dtype):
    """The first key outscores all others by `gap` nats and its value is 0: what a row gives
    are the others' weights, e^-10 to e^-20 of the sink's."""
    c = ref.Case(lens, new, H, Hkv, D, dtype, seed=int(gap) + D)
    c.q = (1 + 0.1 * torch.randn(c.T, H, D, generator=c.gen)).bfloat16()
    qmax = float(ref.QMAX[dtype])
    sm = D ** -0.5
    c.k = (8 * torch.randn(c.P, Hkv, 64, D, generator=c.gen)).clamp(-60, 60).round().to(dtype)
    c.k_scale[:] = gap / (sm * D * 64)
    c.v = (qmax / 8 + (qmax / 4 * torch.randn(c.P, Hkv, 64, D, generator=c.gen)).abs()).clamp(max=qmax).round().to(dtype)
    first = c.block_table[:, 0].long()
    c.k.view(torch.uint8)[first, :, 0] = torch.full((1,), 64.0).to(dtype).view(torch.uint8).item()
    c.v.view(torch.uint8)[first, :, 0] = 0
    check(c, sm, sample(c))


@pytest.mark.parametrize("dtype", [E4, I8], ids=["e4m3", "i8"])
@pytest.mark.parametrize("up", [10, 20])
@pytest.mark.parametrize("lens,new,H,Hkv,D", [
    ([128], [1], 2, 2, 64), ([128, 110], [2, 1], 8, 1, 128), ([128] * 40, [20] * 40, 32, 8, 64)])
def test_value_scale_above_the_others(lens, new, H, Hkv, D, up, dtype):
    """One outlier value raises its block's scale by 2^up, so that the block's other values
    are coded as 0: the other blocks' values still reach the output in every other column."""
    c = ref.Case(lens, new, H, Hkv, D, dtype, seed=up)
    qmax = float(ref.QMAX[dtype])
    c.v = (qmax / 8 + (qmax / 4 * torch.randn(c.P, Hkv, 64, D, generator=c.gen)).abs()).clamp(max=qmax).round().to(dtype)
    first = c.block_table[:, 0].long()
    c.v_scale[first] *= 2.0 ** up
    c.v.view(torch.uint8)[first] = 0
    c.v.view(torch.uint8)[first, :, 7, 5] = torch.full((1,), qmax).to(dtype).view(torch.uint8).item()
    check(c, D ** -0.5, sample(c))


@pytest.mark.parametrize("dtype", [E4, I8], ids=["e4m3", "i8"])
@pytest.mark.parametrize("size", [2.0 ** 10, 2.0 ** 20, 2.0 ** 24])
@pytest.mark.parametrize("lens,new,H,Hkv,D", [([200], [1], 8, 2, 64), ([200], [9], 8, 2, 128), ([200], [70], 8, 2, 128)])
def test_scores_without_fractions(lens, new, H, Hkv, D, size, dtype):
    """Two equal keys of one block far above all others (scores of `size` and twice that, sums
    of whole numbers): a row gives the mean of their values. Each weight is rounded to f16 and may
    be cut at f16's largest value, 2^-11 of 2^16; the output is rounded to bf16. The LSE is the score
    after six fp32 roundings (two constants, three products, a sum)."""
    c = ref.Case(lens, new, H, Hkv, D, dtype, seed=5)
    c.q = torch.ones(c.T, H, D).bfloat16()
    c.k = torch.ones(c.P, Hkv, 64, D).to(dtype)
    c.k_scale[:] = size / D
    two = torch.full((1,), 2.0).to(dtype).view(torch.uint8).item()
    page = int(c.block_table[0, 1])
    c.k.view(torch.uint8)[page, :, [3, 40]] = two
    out, lse = Dev(c).attend(1.0)
    v = c.v[page].double() * c.v_scale[page].double()[:, None, None]
    want = (0.5 * (v[:, 3] + v[:, 40])).repeat_interleave(c.G, 0)
    mag = (0.5 * (v[:, 3].abs() + v[:, 40].abs())).repeat_interleave(c.G, 0)
    off = (out.double().cpu() - want[None]).abs()
    assert (off <= 2.0 ** -8 * want.abs() + (1 + 2.0 ** -8) * 2.0 ** -10 * mag).all()
    assert (lse.double().cpu() - (2 * size + math.log(2))).abs().max() <= 2 * size * 2.0 ** -21 + 2.0 ** -20


@pytest.mark.parametrize("dtype", [E4, I8], ids=["e4m3", "i8"])
@pytest.mark.parametrize("other", [2.0 ** -100, 2.0 ** -60, 2.0 ** 8])
@pytest.mark.parametrize("lens,new,H,Hkv,D", [([128], [1], 2, 2, 64), ([700, 333], [2, 1], 8, 1, 128), ([600, 130], [300, 64], 8, 2, 128)])
def test_blocks_of_zeros(lens, new, H, Hkv, D, other, dtype):
    """Every second block holds zeros, at the least scale that the append writes, and the others'
    scales are up to 2^108 above it: the zeros' weights count in the denominator all the same. (The
    sum of a score in powers of two and a scale's logarithm is rounded to 2^-18 up to 128: 2^-15 for
    a weight's relative error of several such.)"""
    c = ref.Case(lens, new, H, Hkv, D, dtype, seed=8)
    c.v_scale[:] = other * (1 + torch.rand(c.v_scale.shape, generator=c.gen)) / 2
    for b, n in enumerate(lens):
        zeros = c.block_table[b, :-(-n // 64):2].long()
        c.v_scale[zeros] = 2.0 ** -100
        c.v.view(torch.uint8)[zeros] = 0
    out, lse = Dev(c).attend(D ** -0.5)
    r = ref.attend(c, D ** -0.5)
    rel = 2 * D * 2.0 ** -24 * r["dots"] + 2.0 ** -11 + 2.0 ** -15
    got, le = out.double().cpu().numpy(), lse.double().cpu().numpy()
    bound = np.abs(r["out"]) * 2.0 ** -8 + (1 + 2.0 ** -8) * r["mag"] * 2 * rel[..., None]
    assert (np.abs(got - r["out"]) <= bound).all()
    assert (np.abs(le - r["lse"]) <= rel - 2.0 ** -11 + 2.0 ** -20 + np.abs(r["lse"]) * 2.0 ** -22).all()
