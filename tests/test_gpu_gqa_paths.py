"""Forms of the grouped-query kernels that only sizes choose: twelve warps over many lists,
items cut into runs of more than 32 blocks, rows of scores of every length in the selection's
tiles, notes of NaN values that come round again, and prompts of more than 4096 rows. Rows are
sampled for the comparison with 64 bits. Caches stay small: block tables repeat pages."""
import math

import numpy as np
import pytest
import torch

import gqa_reference as ref
from dsa_sparse_attention_02_gb300 import _lib
from test_gpu_gqa import DEV, E4, I8, Dev

pytestmark = pytest.mark.gpu


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def wide_case(lens, new, H, Hkv, D, dtype, seed, pages, pad=0):
    """A batch whose block tables take their pages at random from a small cache."""
    c = ref.Case([64 * pages], [1], H, Hkv, D, dtype, seed=seed, spare=0)
    c.lens, c.new, c.T, c.max_len = list(lens), list(new), sum(new) + pad, max(lens)
    c.seq_lens = torch.tensor(c.lens, dtype=torch.int32)
    c.cu_q = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
    c.block_table = torch.randint(0, pages, (len(lens), -(-c.max_len // 64)), generator=c.gen, dtype=torch.int32)
    c.q = (1.5 * torch.randn(c.T, H, D, generator=c.gen)).bfloat16()
    return c


def sampled(c, n, always=()):
    """The case restricted to n of its tokens for the references; their numbers."""
    ts = sorted(set(torch.randperm(sum(c.new), generator=c.gen)[:n].tolist()) | set(always))
    c.tokens = lambda: [x for x in ref.Case.tokens(c) if x[0] in ts]
    return ts


def same_rows(c, ts, got, sm, blocks=None):
    out, lse = got
    with np.errstate(invalid="ignore"):
        r = ref.attend(c, sm, blocks)
        bo, bl = ref.attend_bounds(r)
        o, l = out[ts].double().cpu().numpy(), lse[ts].double().cpu().numpy()
        assert np.array_equal(np.isnan(o), np.isnan(r["out"][ts])) and np.array_equal(np.isneginf(l), np.isneginf(r["lse"][ts]))
        fine = np.isfinite(r["out"][ts]) & np.isfinite(bo[ts])
        assert (np.abs(o - r["out"][ts])[fine] <= bo[ts][fine]).all()
        fine = np.isfinite(r["lse"][ts])
        assert (np.abs(l - r["lse"][ts])[fine] <= bl[ts][fine]).all()


@pytest.mark.parametrize("dtype", [E4, I8], ids=["e4m3", "i8"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hkv,G,n_sel", [(8, 5, 8), (2, 8, 31), (4, 1, 1)])
def test_many_lists(Hkv, G, n_sel, D, dtype):
    """At least 384 listed blocks an SM; lists with tails of -1, empty ones, blocks past the
    token's own, tokens at negative positions and padding rows."""
    new = -(-384 * sms() // (Hkv * n_sel)) // 3 + 1
    c = wide_case([new + 900, 700, new - 5], [new] * 3, G * Hkv, Hkv, D, dtype, D + G, 24, pad=7)
    assert c.T * Hkv * n_sel >= 384 * sms()
    nb = 1 + (c.max_len - 1) // 64
    key = torch.rand(c.T, Hkv, nb, generator=c.gen)
    top = key.topk(min(n_sel, nb), -1).indices.sort(-1).values.int()
    cut = torch.randint(0, n_sel + 1, (c.T, Hkv, 1), generator=c.gen)
    blocks = torch.full((c.T, Hkv, n_sel), -1, dtype=torch.int32)
    blocks[..., :top.shape[-1]] = torch.where(torch.arange(top.shape[-1]) < cut, top, -1)
    d = Dev(c)
    got = d.attend(0.11, blocks.to(DEV))
    assert _lib.dsa_get_error(d.ws) == 0
    n = sum(c.new)
    assert torch.isfinite(got[0][:n]).all() and (got[0][n:] == 7.0).all() and (got[1][n:] == 7.0).all()
    same_rows(c, sampled(c, 60, (0, n - 1, 2 * new, 2 * new + 4, 2 * new + 5)), got, 0.11, blocks)
    again = d.attend(0.11, blocks.to(DEV))
    assert all(torch.equal(a, b) for a, b in zip(got, again))


@pytest.mark.parametrize("dtype", [E4, I8], ids=["e4m3", "i8"])
@pytest.mark.parametrize("new,G", [(1, 2), (2, 8), (4, 7)])
def test_long_contexts_in_long_runs(new, G, dtype):
    lens = [50000 + 777 * i for i in range(8)]
    c = wide_case(lens, [new] * 8, 8 * G, 8, 64, dtype, 3, 40)
    units = 8 * sum(-(-n // 64) for n in lens)
    assert units > 33 * 8 * sms()                       # of a warp
    d = Dev(c)
    got = d.attend(0.125)
    assert _lib.dsa_get_error(d.ws) == 0
    same_rows(c, sampled(c, 3, (0,)), got, 0.125)


def test_prompt_of_many_rows():
    """More than 4096 rows a request (no prefetch), more than 32 blocks an SM within items."""
    c = wide_case([9001], [1100], 16, 2, 128, E4, 5, 30)
    kb, vb = c.k.view(torch.uint8), c.v.view(torch.uint8)
    c.block_table[0, -18:] = torch.arange(12, 30)        # the new tokens' pages, each there once
    c.block_table[0, :-18] %= 12
    vb[int(c.block_table[0, 8500 // 64]), 0, 8500 % 64, 77] = 0x7F
    d = Dev(c)
    got = d.attend(0.09)
    assert _lib.dsa_get_error(d.ws) == 0
    start = 9001 - 1100
    nan = torch.isnan(got[0].float())
    want = torch.zeros_like(nan)
    want[8500 - start:, :8, 77] = True
    assert torch.equal(nan, want)
    same_rows(c, sampled(c, 12, (0, 599, 598, 1099)), got, 0.09)


@pytest.mark.parametrize("D", [64, 128])
def test_nan_notes_come_round(D):
    """Hundreds of requests an SM's tiles go through in turn, some with NaN values in the block
    that their rows see in part: NaN in the columns and rows that see them, and in no other's."""
    B, H, Hkv = 3 * sms(), 16, 4
    c = ref.Case([70] * B, [70] * B, H, Hkv, D, E4, seed=D)
    vb = c.v.view(torch.uint8)
    want = torch.zeros(c.T, H, D, dtype=torch.bool)
    for b in range(0, B, 7):
        for i in range(1 + b % 3):
            pos, h, col = (11 * b + 29 * i) % 70, (b + i) % Hkv, (5 * b + 31 * i) % D
            vb[int(c.block_table[b, pos // 64]), h, pos % 64, col] = 0x7F if i else 0xFF
            want[70 * b + pos:70 * b + 70, 4 * h:4 * h + 4, col] = True
    d = Dev(c)
    got = d.attend(0.1)
    assert _lib.dsa_get_error(d.ws) == 0
    assert torch.equal(torch.isnan(got[0].float()).cpu(), want)
    assert torch.isfinite(got[1]).all()
    same_rows(c, sampled(c, 80, (0, 69, 70, c.T - 1)), got, 0.1)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("nb,n", [(200, 9), (300, 32), (300, 298), (700, 40), (700, 697), (1650, 64), (1650, 1000), (5000, 17)])
def test_selection_of_prompts(nb, n, D):
    """Rows of scores that a lane holds in 8 or 16 registers or not at all, tiles of 16 and of 8
    tokens: with ties (pages that repeat), NaN scores, negative scales, a query of zeros."""
    new = 16 * sms() // 4 + 41
    c = wide_case([64 * nb - 9, 64 * nb - 700], [new - 30, 30], 8, 4, D, E4, nb + n, 150, pad=5)
    assert c.T // 2 >= 8 and c.T * 4 >= 16 * sms()
    c.k_mean_scale[3] = math.nan
    c.k_mean_scale[4] *= -1
    c.k_mean[5] = 0
    c.q[7] = 0
    c.q[-9, 2] = 0
    d = Dev(c)
    got = d.select(n, 2, 3)
    assert _lib.dsa_get_error(d.ws) == 0
    ts = sampled(c, 25, (0, 7, new - 31, new - 30, new - 4, new - 1))
    with np.errstate(invalid="ignore"):
        want = ref.select(c, n, 2, 3)
    assert np.array_equal(got[ts].cpu().numpy(), want[ts])
    assert (got[new:] == -9).all()


@pytest.mark.parametrize("dtype", [E4, I8], ids=["e4m3", "i8"])
def test_stored_bytes(dtype):
    """Codes as bytes: zeros keep their sign in e4m3, when written and when a growing scale
    rounds them again; a NaN is 0x7F, and int8 0."""
    c = ref.Case([20], [20], 2, 2, 64, dtype, seed=4, max_len=64)
    c.block_table[0, 0] = 1
    d = Dev(c)
    ws = _lib.workspace(256, DEV)
    qmax = ref.QMAX[dtype]

    def code(x):
        if dtype == I8:
            return np.where(np.isnan(x), 0, np.clip(np.rint(x), -127, 127)).astype(np.int8).view(np.uint8)
        b = torch.from_numpy(np.clip(x, -qmax, qmax).astype(np.float32)).to(E4).view(torch.uint8).numpy()
        return np.where(np.isnan(x), np.uint8(0x7F), b)

    x = torch.randn(20, 4, 64, generator=c.gen)
    x[3], x[4, :, ::2], x[4, :, 1::2] = 0.0, -0.0, -1e-9
    x[5, 1, 7], x[6, 2, 9] = math.nan, -math.nan
    x[12:] *= 40                                           # a second call, with a scale that grows
    x = x.bfloat16()
    values, scale = {}, {}
    for lo, hi in ((0, 12), (12, 20)):
        geom = _lib.Geometry(torch.tensor([hi], dtype=torch.int32, device=DEV), torch.tensor([0, hi - lo], dtype=torch.int32, device=DEV),
                             d.block_table, c.P, 64, hi - lo)
        part = x[lo:hi].to(DEV)
        _lib.dsa_gqa_append(geom, d.cache, part[:, :2], part[:, 2:], ws=ws)
        assert _lib.dsa_get_error(ws) == 0
        for name, at in (("k", 0), ("v", 2)):
            for h in range(2):
                y = x[lo:hi, at + h].float().numpy()
                big = np.abs(y[np.isfinite(y)]).max() / qmax
                s = max(big, scale.get((name, h), np.float32(0)))
                old = values.get((name, h), np.zeros((0, 64), np.uint8))
                was = torch.from_numpy(old.copy()).view(dtype).float().numpy()
                values[name, h] = np.concatenate([code(was * (scale.get((name, h), np.float32(0)) / s)), code(y / s)])
                scale[name, h] = s
                got = getattr(d, name)[1, h].view(torch.uint8).cpu().numpy()
                assert np.array_equal(got[:hi], values[name, h]), (name, h, lo)
                assert float(getattr(d, name + "_scale")[1, h]) == float(s)
    if dtype == E4:
        assert (values["k", 0] == 0x80).any() and (values["k", 0] == 0).any() and (values["k", 1] == 0x7F).any()
