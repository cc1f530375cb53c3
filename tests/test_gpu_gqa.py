"""The grouped-query operators against their plain definitions: append bit for bit (its
operations are defined one by one), attention within bounds derived from its roundings,
block lists equal."""
import math

import numpy as np
import pytest
import torch

import gqa_reference as ref
from dsa_sparse_attention_02_gb300 import _lib

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E4, I8 = torch.float8_e4m3fn, torch.int8


class Dev:
    """A Case on the GPU."""

    def __init__(self, c):
        self.c = c
        up = lambda x: x.to(DEV)  # noqa: E731
        self.k, self.v = (x.view(torch.uint8).to(DEV).view(c.dtype) for x in (c.k, c.v))
        self.k_scale, self.v_scale, self.k_mean, self.k_mean_scale = map(up, (c.k_scale, c.v_scale, c.k_mean, c.k_mean_scale))
        self.seq_lens, self.cu_q, self.block_table, self.q = map(up, (c.seq_lens, c.cu_q, c.block_table, c.q))
        self.geom = _lib.Geometry(self.seq_lens, self.cu_q, self.block_table, c.P, c.max_len, c.T)
        self.cache = _lib.GqaCache(self.k, self.v, self.k_scale, self.v_scale, self.k_mean, self.k_mean_scale)

    def attend(self, sm_scale, blocks=None, q=None, ws=None, lse=True, stream=None):
        c = self.c
        q = self.q if q is None else q
        out = torch.full((c.T, c.H, c.D), 7.0, dtype=torch.bfloat16, device=DEV)
        le = torch.full((c.T, c.H), 7.0, device=DEV) if lse else None
        if blocks is None:
            ws = _lib.workspace(_lib.dsa_gqa_attend_workspace_size(self.geom, self.cache, c.H), DEV) if ws is None else ws
            _lib.dsa_gqa_attend(self.geom, self.cache, q, sm_scale, out, le, ws, stream)
        else:
            n = blocks.shape[2]
            ws = _lib.workspace(_lib.dsa_gqa_attend_blocks_workspace_size(self.geom, self.cache, c.H, n), DEV) if ws is None else ws
            _lib.dsa_gqa_attend_blocks(self.geom, self.cache, q, blocks, sm_scale, out, le, ws, stream)
        self.ws = ws
        return out, le

    def select(self, n_sel, first, last, stream=None):
        c = self.c
        blocks = torch.full((c.T, c.Hkv, n_sel), -9, dtype=torch.int32, device=DEV)
        self.ws = _lib.workspace(_lib.dsa_block_select_workspace_size(self.geom, self.cache, n_sel), DEV)
        _lib.dsa_block_select(self.geom, self.cache, self.q, n_sel, first, last, blocks, self.ws, stream)
        return blocks


def tables(c, rope):
    r = rope // 2
    if not r:
        return None, None
    ang = np.arange(c.max_len)[:, None] * 10000.0 ** (-np.arange(r) / r)
    return np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)


def check_attend(d, sm_scale, blocks=None, err=0, **kw):
    c = d.c
    out, lse = d.attend(sm_scale, None if blocks is None else blocks.to(DEV), **kw)
    assert _lib.dsa_get_error(d.ws) == err
    r = ref.attend(c, sm_scale, blocks)
    bo, bl = ref.attend_bounds(r)
    n = sum(c.new)
    got = out.double().cpu().numpy()[:n]
    off = np.abs(got - r["out"][:n])
    assert np.isfinite(got).all()
    assert (off <= bo[:n]).all(), float((off / bo[:n]).max())
    if lse is not None:
        le, want = lse.double().cpu().numpy()[:n], r["lse"][:n]
        assert (np.isneginf(le) == np.isneginf(want)).all()
        ok = np.isfinite(want)
        assert (np.abs(le - want)[ok] <= bl[:n][ok]).all(), float((np.abs(le - want)[ok] / bl[:n][ok]).max())
        assert (lse[n:] == 7.0).all()
    assert (out[n:] == 7.0).all()           # rows behind the last request
    return out, lse


# ---------------------------------------------------------------- append

def run_append(c, k_new, v_new, q_in, rope, mean=True, dev=None):
    d = dev or Dev(c)
    cos, sin = tables(c, rope)
    up = lambda x: None if x is None else torch.from_numpy(x).to(DEV)  # noqa: E731
    cache = d.cache if mean else _lib.GqaCache(d.k, d.v, d.k_scale, d.v_scale)
    q_out = None if q_in is None else torch.full((c.T, c.H, c.D), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = _lib.workspace(_lib.dsa_gqa_append_workspace_size(d.geom, cache), DEV)
    _lib.dsa_gqa_append(d.geom, cache, k_new, v_new, q_in, q_out, rope, up(cos), up(sin), ws)
    d.ws = ws
    want = ref.append(c, k_new.cpu(), v_new.cpu(), None if q_in is None else q_in.cpu(), rope, cos, sin, mean)
    return d, q_out, want


def same_state(d, want, q_out=None, T=None):
    for name in ("k", "v"):
        got = getattr(d, name).float().cpu().numpy()
        assert np.array_equal(got, want[name], equal_nan=True), (name, int((got != want[name]).sum()))
    for name in ("k_scale", "v_scale", "k_mean", "k_mean_scale"):
        assert np.array_equal(getattr(d, name).cpu().numpy(), want[name]), name
    if q_out is not None:
        assert torch.equal(q_out[:T].cpu(), want["q"][:T])
        assert (q_out[T:] == 7.0).all()


APPEND = [   # lens, new, H, Hkv, D, rope
    ([1], [1], 1, 1, 128, 0), ([1], [1], 3, 3, 64, 8), ([64], [1], 8, 2, 128, 64), ([65], [1], 8, 2, 64, 64),
    ([200, 256, 63], [1, 1, 1], 16, 4, 128, 128), ([130, 64, 5, 300], [4, 64, 5, 129], 5, 1, 128, 24),
    ([130, 64, 5, 300], [3, 1, 2, 66], 32, 2, 64, 40), ([700], [700], 8, 8, 128, 128), ([1000] * 40, [2] * 40, 7, 1, 64, 32),
]


@pytest.mark.parametrize("dtype", [E4, I8], ids=["e4m3", "i8"])
@pytest.mark.parametrize("lens,new,H,Hkv,D,rope", APPEND)
def test_append_bit_for_bit(lens, new, H, Hkv, D, rope, dtype):
    c = ref.Case(lens, new, H, Hkv, D, dtype, seed=len(lens) + D, pad=3)
    # one projection's output: queries, keys and values side by side; magnitudes that grow some scales and not others
    qkv = torch.randn(c.T, H + 2 * Hkv, D, generator=c.gen) * torch.exp(torch.randn(c.T, 1, 1, generator=c.gen))
    qkv = qkv.bfloat16().to(DEV)
    q, k, v = qkv[:, :H], qkv[:, H:H + Hkv], qkv[:, H + Hkv:]
    d, q_out, want = run_append(c, k, v, q, rope)
    assert _lib.dsa_get_error(d.ws) == 0
    same_state(d, want, q_out, sum(new))


def test_append_within_half_a_step_of_64_bits():
    """Dequantised new tokens against the rotation in 64 bits: a code is off by half a step
    (e4m3 2^-4 of the value, or 2^-10 of the scale below its normal range), the fp32
    rotation, scale and quotient by a few 2^-24 of the block's largest value."""
    c = ref.Case([300], [170], 8, 2, 128, E4, seed=5)
    x = torch.randn(c.T, 12, 128, generator=c.gen).bfloat16()
    d, _, _ = run_append(c, x[:, :2].to(DEV), x[:, 2:4].to(DEV), None, 128)
    ang = np.arange(300)[:, None] * 10000.0 ** (-np.arange(64) / 64)
    cos, sin = np.cos(ang).astype(np.float32).astype(np.float64), np.sin(ang).astype(np.float32).astype(np.float64)
    for t, _, pos in c.tokens():
        page = int(c.block_table[0, pos // 64])
        for h in range(2):
            y = x[t, h].double().numpy()
            turned = np.concatenate([y[:64] * cos[pos] - y[64:] * sin[pos], y[64:] * cos[pos] + y[:64] * sin[pos]])
            for name, want in (("k", turned), ("v", x[t, 2 + h].double().numpy())):
                s = float(getattr(d, name + "_scale")[page, h])
                got = getattr(d, name)[page, h, pos % 64].double().cpu().numpy() * s
                assert (np.abs(got - want) <= np.abs(want) * 2.0 ** -4 + s * (2.0 ** -10 + 448 * 2.0 ** -21)).all()


@pytest.mark.parametrize("dtype", [E4, I8], ids=["e4m3", "i8"])
def test_append_token_by_token(dtype):
    """Ninety tokens one at a time across a page border, magnitudes rising and falling."""
    c = ref.Case([40], [1], 4, 2, 64, dtype, seed=9, max_len=192)
    c.block_table[0, :3] = torch.tensor([2, 0, 1], dtype=torch.int32)
    d = Dev(c)
    for i in range(90):
        c.lens = [41 + i]
        c.seq_lens = torch.tensor(c.lens, dtype=torch.int32)
        d.seq_lens.copy_(c.seq_lens)
        x = (torch.randn(1, 4, 64, generator=c.gen) * math.exp(2 * math.sin(i / 9.0))).bfloat16().to(DEV)
        d, _, want = run_append(c, x[:, :2], x[:, 2:], None, 32, dev=d)
        same_state(d, want)
        c.k, c.v = (torch.from_numpy(want[n]).to(dtype) for n in ("k", "v"))
        c.k_scale, c.v_scale, c.k_mean, c.k_mean_scale = (torch.from_numpy(want[n]) for n in ("k_scale", "v_scale", "k_mean", "k_mean_scale"))


@pytest.mark.parametrize("dtype", [E4, I8], ids=["e4m3", "i8"])
def test_append_odd_values(dtype):
    c = ref.Case([70, 130, 64, 10], [3, 66, 64, 10], 2, 2, 128, dtype, seed=3)
    x = torch.randn(c.T, 4, 128, generator=c.gen)
    x[0, 0, 5], x[0, 1, 6], x[1, 2, 7] = math.nan, math.inf, -math.inf
    x[3:10] = 0
    x[10, :, :] = 3.0e38
    x[69:133] = 0                      # the third request's whole block: scale at its floor
    x[133:] = 1e-38
    x = x.bfloat16().to(DEV)
    with np.errstate(over="ignore", invalid="ignore"):
        d, _, want = run_append(c, x[:, :2], x[:, 2:], None, 0)
    same_state(d, want)


def test_append_without_means_leaves_them():
    c = ref.Case([100, 3], [5, 3], 4, 4, 128, E4, seed=4)
    x = torch.randn(c.T, 8, 128, generator=c.gen).bfloat16().to(DEV)
    d, _, want = run_append(c, x[:, :4], x[:, 4:], None, 0, mean=False)
    same_state(d, want)


def test_append_empty_requests_padding_and_bad_pages():
    """Padding requests (seq_lens 0, or no new token), tokens at negative positions, and a
    request whose page does not exist: everything else is stored, the last is reported."""
    c = ref.Case([0, 90, 2, 70, 33], [1, 0, 4, 2, 1], 2, 2, 64, E4, seed=8, pad=2)
    c.block_table[3, 1] = c.P
    x = torch.randn(c.T, 6, 64, generator=c.gen).bfloat16().to(DEV)
    d, q_out, want = run_append(c, x[:, 2:4], x[:, 4:], x[:, :2], 16)
    assert _lib.dsa_get_error(d.ws) == _lib.DSA_ERR_BAD_INDEX
    same_state(d, want)
    real = [t for t, _, pos in c.tokens() if pos >= 0]
    assert torch.equal(q_out[real].cpu(), want["q"][real])
    rest = [t for t in range(c.T) if t not in real]
    assert (q_out[rest] == 7.0).all()


def test_append_bad_lengths_are_reported():
    c = ref.Case([100, 50], [2, 1], 2, 2, 64, E4, seed=8)
    d0 = Dev(c)
    for seq, cu in (([2000, 50], [0, 2, 3]), ([100, 50], [0, 2, 4]), ([100, 50], [0, 2, 1])):
        d0.seq_lens.copy_(torch.tensor(seq))
        d0.cu_q.copy_(torch.tensor(cu))
        x = torch.zeros(3, 4, 64, dtype=torch.bfloat16, device=DEV)
        ws = _lib.workspace(256, DEV)
        _lib.dsa_gqa_append(d0.geom, d0.cache, x[:, :2], x[:, 2:], ws=ws)
        assert _lib.dsa_get_error(ws) == _lib.DSA_ERR_BAD_INDEX


# ---------------------------------------------------------------- attention

ATTEND = [   # lens, new, H, Hkv, D
    ([1], [1], 1, 1, 128), ([2], [1], 16, 1, 64), ([63, 64, 65], [1, 1, 1], 8, 1, 128), ([127, 128, 129], [1, 2, 3], 6, 2, 64),
    ([200, 256], [1, 1], 12, 4, 64), ([1000, 37, 511], [4, 1, 3], 40, 8, 128), ([300], [17], 7, 1, 128), ([300], [130], 16, 2, 64),
    ([500, 90], [33, 90], 24, 8, 128), ([5000], [1], 8, 1, 128), ([2111], [2], 5, 5, 64), ([640] * 33, [1] * 33, 16, 1, 128),
    ([260, 1, 70], [260, 1, 70], 8, 2, 128), ([400, 600], [129, 5], 16, 1, 128),
]


@pytest.mark.parametrize("dtype", [E4, I8], ids=["e4m3", "i8"])
@pytest.mark.parametrize("lens,new,H,Hkv,D", ATTEND)
def test_attend(lens, new, H, Hkv, D, dtype):
    c = ref.Case(lens, new, H, Hkv, D, dtype, seed=sum(lens) % 97, pad=2)
    check_attend(Dev(c), D ** -0.5)


@pytest.mark.parametrize("new", [1, 4, 40, 200])
def test_attend_empty_rows_and_padding(new):
    """Requests of length 0 (with a token, as padded batches have), of fewer keys than new
    tokens, and without new tokens."""
    c = ref.Case([0, 70, new - 1, 130, 64], [1, 0, new, 2, 1], 8, 2, 128, E4, seed=2, pad=5)
    out, lse = check_attend(Dev(c), 0.1)
    empty = [t for t, _, pos in c.tokens() if pos < 0]
    assert len(empty) >= 2 and (out[empty] == 0).all() and torch.isneginf(lse[empty]).all()


@pytest.mark.parametrize("new", [1, 3, 20, 70])
@pytest.mark.parametrize("dtype", [E4, I8], ids=["e4m3", "i8"])
def test_attend_does_not_see_what_it_must_not(new, dtype):
    """NaN codes behind every row's last key, in unused pages, and in keys and values of
    newer tokens of the same request that only later rows see."""
    c = ref.Case([150, 200], [new, new], 16, 2, 128, dtype, seed=6)
    used = {int(c.block_table[b, i]): (b, i) for b, n in enumerate(c.lens) for i in range(-(-n // 64))}
    kb, vb = c.k.view(torch.uint8), c.v.view(torch.uint8)
    for p in range(c.P):
        lo = 0 if p not in used else max(0, min(64, c.lens[used[p][0]] - 64 * used[p][1]))
        kb[p, :, lo:], vb[p, :, lo:] = 0x7F, 0xFF
        if p not in used:
            c.k_scale[p], c.v_scale[p] = math.nan, math.inf
    check_attend(Dev(c), 128 ** -0.5)
    if dtype == I8 or new == 1:
        return
    d = Dev(c)
    clean, clean_lse = d.attend(128 ** -0.5)
    # the last token of each request: its value is NaN in column 3, its key in column 9
    for b, n in enumerate(c.lens):
        p = int(c.block_table[b, (n - 1) // 64])
        vb[p, :, (n - 1) % 64, 3] = 0x7F
    d2 = Dev(c)
    out, lse = d2.attend(128 ** -0.5)
    last = torch.zeros(c.T, dtype=torch.bool)
    last[[new - 1, 2 * new - 1]] = True
    first = ~last
    assert torch.isfinite(out[first]).all() and torch.equal(lse, clean_lse)
    bound = 2.0 ** -7 * clean.float().abs() + 2.0 ** -9
    assert ((out.float() - clean.float()).abs()[first] <= bound[first]).all()
    assert torch.isnan(out[last][:, :, 3]).all()
    rest = torch.ones(128, dtype=torch.bool)
    rest[3] = False
    assert ((out.float() - clean.float()).abs()[last][:, :, rest] <= bound[last][:, :, rest]).all()
    for b, n in enumerate(c.lens):
        p = int(c.block_table[b, (n - 1) // 64])
        kb[p, :, (n - 1) % 64, 9] = 0x7F
    out, lse = Dev(c).attend(128 ** -0.5)
    assert ((out.float() - clean.float()).abs()[first] <= bound[first]).all()
    assert torch.isnan(out[last]).all()


@pytest.mark.parametrize("new", [1, 30])
def test_attend_wide_ranges(new):
    """Scores that rise from page to page by large steps, scales of pages that differ by
    2^30, queries far below and above the normal range, an attention scale of 0."""
    c = ref.Case([700, 333], [new, new], 8, 2, 128, E4, seed=12)
    c.k_scale *= torch.exp(1.5 * torch.randn(c.P, 2, generator=c.gen))
    c.v_scale *= torch.exp2(30 * (torch.rand(c.P, 2, generator=c.gen) - 0.5))
    check_attend(Dev(c), 128 ** -0.5)
    check_attend(Dev(c), 0.0)
    c.q = (c.q.float() * 1e-20).bfloat16()
    c.k_scale *= 1e20
    check_attend(Dev(c), 0.05)
    c.q = (c.q.float() * 1e20 * 1e20).bfloat16()
    c.k_scale *= 1e-30
    c.k_scale *= 1e-10
    check_attend(Dev(c), 0.05)
    c.q[:, ::3] = 0
    check_attend(Dev(c), 0.05)


@pytest.mark.parametrize("new", [1, 2, 50])
def test_attend_strided_queries_no_lse(new):
    c = ref.Case([120, 77], [new, new], 6, 2, 64, I8, seed=1)
    d = Dev(c)
    wide = torch.full((c.T, 11, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    wide[:, :6] = d.q
    a, la = check_attend(d, 0.125)
    b, lb = d.attend(0.125, q=wide[:, :6])
    assert torch.equal(a, b) and torch.equal(la, lb)
    e, _ = d.attend(0.125, lse=False)
    assert torch.equal(a, e)


def test_attend_bad_pages_and_lengths():
    c = ref.Case([300, 200], [2, 1], 8, 2, 128, E4, seed=4)
    c.block_table[0, 2] = c.P + 5
    c.block_table[1, 0] = -1
    check_attend(Dev(c), 0.09, err=_lib.DSA_ERR_BAD_INDEX)
    c = ref.Case([300, 200], [2, 1], 8, 2, 128, E4, seed=4)
    d = Dev(c)
    d.seq_lens[0] = 100000
    out, lse = d.attend(0.09)
    assert _lib.dsa_get_error(d.ws) == _lib.DSA_ERR_BAD_INDEX
    assert (out[:2] == 0).all() and torch.isneginf(lse[:2]).all() and torch.isfinite(lse[2]).all()


@pytest.mark.parametrize("blocks", [False, True])
def test_attend_repeats_bit_for_bit(blocks):
    c = ref.Case([900, 4000, 100, 2500], [1, 1, 3, 2], 16, 2, 128, E4, seed=7)
    d = Dev(c)
    li = d.select(5, 1, 2) if blocks else None
    a, la = d.attend(0.1, li)
    ws = d.ws
    ws[256:] = 0xA5                      # a workspace holds nothing from call to call
    for _ in range(3):
        b, lb = d.attend(0.1, li, ws=ws)
        assert torch.equal(a, b) and torch.equal(la, lb)


# ---------------------------------------------------------------- listed blocks

def lists(c, n, kind):
    """Ascending lists: random subsets, empty ones, blocks past the token's own."""
    nb = -(-c.max_len // 64)
    out = torch.full((c.T, c.Hkv, n), -1, dtype=torch.int32)
    for t in range(c.T):
        for h in range(c.Hkv):
            m = min(n, nb) if kind == "full" else int(torch.randint(0, min(n, nb) + 1, (1,), generator=c.gen))
            out[t, h, :m] = torch.randperm(nb, generator=c.gen)[:m].sort().values.int()
    return out


@pytest.mark.parametrize("dtype", [E4, I8], ids=["e4m3", "i8"])
@pytest.mark.parametrize("kind", ["full", "random"])
@pytest.mark.parametrize("lens,new,H,Hkv,D,n", [
    ([300, 1, 90], [1, 1, 2], 8, 2, 128, 3), ([1000, 700], [1, 1], 16, 1, 64, 12), ([400], [40], 5, 1, 128, 4),
    ([129, 640], [3, 20], 24, 8, 64, 1), ([2000] * 5, [1] * 5, 14, 2, 128, 31)])
def test_attend_blocks(lens, new, H, Hkv, D, n, kind, dtype):
    c = ref.Case(lens, new, H, Hkv, D, dtype, seed=n + D, pad=1)
    check_attend(Dev(c), D ** -0.5, blocks=lists(c, n, kind))


def test_attend_all_blocks_is_attend():
    c = ref.Case([300, 70, 513], [4, 1, 2], 16, 2, 128, E4, seed=3)
    d = Dev(c)
    li = torch.arange(9, dtype=torch.int32, device=DEV).expand(c.T, 2, 9).contiguous()
    a, la = check_attend(d, 0.1)
    b, lb = d.attend(0.1, li)
    assert _lib.dsa_get_error(d.ws) == 0
    r = ref.attend(c, 0.1)
    bo, bl = ref.attend_bounds(r)
    assert (np.abs(b.double().cpu().numpy() - r["out"]) <= bo).all()
    assert (np.abs(lb.double().cpu().numpy() - r["lse"]) <= bl).all()


def test_attend_blocks_lists_out_of_order():
    """Entries that repeat or fall back, or that follow -1, are skipped and reported."""
    c = ref.Case([400], [1], 8, 2, 128, E4, seed=3)
    d = Dev(c)
    want = torch.tensor([[[0, 2, 5, -1], [1, -1, -1, -1]]], dtype=torch.int32)
    a, la = d.attend(0.1, want.to(DEV))
    assert _lib.dsa_get_error(d.ws) == 0
    bad = torch.tensor([[[0, 2, 2, 5], [1, -1, 3, -1]]], dtype=torch.int32)
    b, lb = d.attend(0.1, bad.to(DEV))
    assert _lib.dsa_get_error(d.ws) == _lib.DSA_ERR_BAD_INDEX
    r = ref.attend(c, 0.1, want)
    bo, bl = ref.attend_bounds(r)
    for o, l in ((a, la), (b, lb)):
        assert (np.abs(o.double().cpu().numpy() - r["out"]) <= bo).all()
        assert (np.abs(l.double().cpu().numpy() - r["lse"]) <= bl).all()
    far = torch.tensor([[[6, 7, 100000, 2 ** 31 - 1], [-5, -1, -1, -1]]], dtype=torch.int32)
    o, l = d.attend(0.1, far.to(DEV))       # block 6 is the token's own
    assert torch.isfinite(o).all() and torch.isneginf(l[0, 4:]).all() and (o[0, 4:] == 0).all()


# ---------------------------------------------------------------- selection

SELECT = [   # lens, new, H, Hkv, D, n_sel, first, last
    ([1, 64, 65], [1, 1, 1], 4, 2, 128, 1, 0, 1), ([3000], [1], 8, 1, 128, 8, 1, 2), ([3000, 900], [2, 3], 5, 1, 64, 4, 0, 1),
    ([5000, 70, 0, 640], [1, 1, 1, 2], 16, 2, 64, 9, 2, 3), ([9000], [1], 16, 4, 128, 70, 1, 1), ([2500], [700], 16, 4, 128, 8, 1, 2),
    ([2000, 1200, 700], [300, 400, 33], 9, 3, 64, 5, 1, 1), ([70000], [1], 2, 1, 128, 1000, 3, 5), ([6000], [900], 8, 8, 128, 24, 0, 2),
]


@pytest.mark.parametrize("lens,new,H,Hkv,D,n,first,last", SELECT)
def test_select(lens, new, H, Hkv, D, n, first, last):
    c = ref.Case(lens, new, H, Hkv, D, E4, seed=n + D, pad=2)
    d = Dev(c)
    got = d.select(n, first, last)
    assert _lib.dsa_get_error(d.ws) == 0
    want = ref.select(c, n, first, last)
    m = sum(new)
    assert np.array_equal(got[:m].cpu().numpy(), want[:m])
    assert (got[m:] == -9).all()


@pytest.mark.parametrize("new", [1, 600])
def test_select_ties_zeros_and_nan(new):
    c = ref.Case([6000], [new], 4, 4, 64, E4, seed=1)
    for i in range(94):                       # few distinct means: ties everywhere
        p = int(c.block_table[0, i])
        c.k_mean[p] = c.k_mean[int(c.block_table[0, i % 3])]
        c.k_mean_scale[p] = 1.0
    c.k_mean[int(c.block_table[0, 40]), 1] = 0
    c.k_mean_scale[int(c.block_table[0, 41]), 2] = math.nan
    c.k_mean_scale[int(c.block_table[0, 42]), 2] = -1.0
    c.q[0, 0] = 0                             # every score 0
    c.q[0, 2, 5] = math.nan
    c.q[-1, 3] = math.inf
    d = Dev(c)
    for n, f, l in ((7, 1, 2), (33, 0, 1), (93, 4, 4)):
        with np.errstate(invalid="ignore", over="ignore"):
            want = ref.select(c, n, f, l)
        assert np.array_equal(d.select(n, f, l).cpu().numpy()[:, :3], want[:, :3])
        got = d.select(n, f, l)[:, 3]         # an infinite query: some list of n blocks, in order
        assert ((got[:, 1:] > got[:, :-1]) | (got[:, 1:] < 0)).all()


def test_select_bad_page_ranks_last_and_is_reported():
    c = ref.Case([3000], [1], 4, 2, 128, E4, seed=1)
    c.block_table[0, 11] = c.P
    d = Dev(c)
    got = d.select(46, 1, 1)
    assert _lib.dsa_get_error(d.ws) == _lib.DSA_ERR_BAD_INDEX
    assert np.array_equal(got.cpu().numpy(), ref.select(c, 46, 1, 1))


# ---------------------------------------------------------------- together

def test_steps_together_on_a_stream_and_in_a_graph():
    """Append, selection and attention over the selected blocks, as a decode step uses them,
    on a stream of their own; then captured once and replayed with new tokens and lengths."""
    H, Hkv, D, n = 16, 2, 128, 6
    c = ref.Case([700, 90, 1500], [1, 1, 1], H, Hkv, D, E4, seed=21, max_len=2048, spare=40)
    for b in range(3):                         # pages for 2048 tokens each
        c.block_table[b] = -7
    P = c.P = 96
    g = c.gen
    order = torch.randperm(P, generator=g).int()
    c.block_table = order.view(3, 32).contiguous()
    c2 = ref.Case([64 * P], [1], H, Hkv, D, E4, seed=22, spare=0)
    c.k, c.v, c.k_scale, c.v_scale, c.k_mean, c.k_mean_scale = c2.k, c2.v, c2.k_scale, c2.v_scale, c2.k_mean, c2.k_mean_scale
    d = Dev(c)
    cos, sin = tables(c, 64)
    dcos, dsin = torch.from_numpy(cos).to(DEV), torch.from_numpy(sin).to(DEV)
    qkv = torch.zeros(3, H + 2 * Hkv, D, dtype=torch.bfloat16, device=DEV)
    q_out = torch.zeros(3, H, D, dtype=torch.bfloat16, device=DEV)
    blocks = torch.zeros(3, Hkv, n, dtype=torch.int32, device=DEV)
    out, lse = torch.zeros(3, H, D, dtype=torch.bfloat16, device=DEV), torch.zeros(3, H, device=DEV)
    ws = _lib.workspace(max(_lib.dsa_gqa_append_workspace_size(d.geom, d.cache), _lib.dsa_block_select_workspace_size(d.geom, d.cache, n),
                            _lib.dsa_gqa_attend_blocks_workspace_size(d.geom, d.cache, H, n)), DEV)

    def step():
        _lib.dsa_gqa_append(d.geom, d.cache, qkv[:, H:H + Hkv], qkv[:, H + Hkv:], qkv[:, :H], q_out, 64, dcos, dsin, ws)
        _lib.dsa_block_select(d.geom, d.cache, q_out, n, 1, 2, blocks, ws)
        _lib.dsa_gqa_attend_blocks(d.geom, d.cache, q_out, blocks, D ** -0.5, out, lse, ws)

    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    for i in range(4):
        new = (1.5 * torch.randn(3, H + 2 * Hkv, D, generator=g)).bfloat16()
        if i == 3:
            c.lens[1] = 0                      # a request that left: its slot is padding now
        c.seq_lens = torch.tensor(c.lens, dtype=torch.int32)
        want = ref.append(c, new[:, H:H + Hkv], new[:, H + Hkv:], new[:, :H], 64, cos, sin)
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            d.seq_lens.copy_(c.seq_lens)
            qkv.copy_(new)
            if i < 2:
                step()
        torch.cuda.synchronize()
        if i == 2:
            with torch.cuda.graph(graph):
                step()
        if i >= 2:
            graph.replay()
        torch.cuda.synchronize()
        assert _lib.dsa_get_error(ws) == 0
        same_state(d, want)
        real = [t for t, _, pos in c.tokens() if pos >= 0]
        assert torch.equal(q_out[real].cpu(), want["q"][real])
        c.k, c.v = (torch.from_numpy(want[x]).to(E4) for x in ("k", "v"))
        c.k_scale, c.v_scale, c.k_mean, c.k_mean_scale = (torch.from_numpy(want[x]) for x in ("k_scale", "v_scale", "k_mean", "k_mean_scale"))
        c.q = q_out.cpu()
        sel = ref.select(c, n, 1, 2)
        assert np.array_equal(blocks.cpu().numpy(), sel)
        r = ref.attend(c, D ** -0.5, torch.from_numpy(sel))
        bo, bl = ref.attend_bounds(r)
        assert (np.abs(out.double().cpu().numpy() - r["out"]) <= bo).all()
        ok = np.isfinite(r["lse"])
        assert (np.abs(lse.double().cpu().numpy() - r["lse"])[ok] <= bl[ok]).all()
        c.lens = [x + 1 for x in c.lens]


def test_prompt_in_chunks_then_decode():
    """A prompt appended and attended chunk by chunk gives what one pass over the stored
    cache gives for its rows (the blocks' scales may have grown in between, so each chunk is
    compared with the cache as it was)."""
    H, Hkv, D = 8, 2, 128
    c = ref.Case([500], [500], H, Hkv, D, I8, seed=31)
    x = torch.randn(500, H + 2 * Hkv, D, generator=c.gen).bfloat16()
    at = 0
    for m in (300, 129, 70, 1):
        c.new, c.lens, c.T = [m], [at + m], m
        c.seq_lens, c.cu_q = torch.tensor([at + m], dtype=torch.int32), torch.tensor([0, m], dtype=torch.int32)
        part = x[at:at + m].to(DEV)
        d, q_out, want = run_append(c, part[:, H:H + Hkv], part[:, H + Hkv:], part[:, :H], 128)
        same_state(d, want, q_out, m)
        c.k, c.v = (torch.from_numpy(want[n]).to(I8) for n in ("k", "v"))
        c.k_scale, c.v_scale, c.k_mean, c.k_mean_scale = (torch.from_numpy(want[n]) for n in ("k_scale", "v_scale", "k_mean", "k_mean_scale"))
        c.q = q_out.cpu()
        check_attend(Dev(c), D ** -0.5)
        at += m


def test_no_work():
    c = ref.Case([10], [1], 2, 2, 64, E4)
    d = Dev(c)
    geom = _lib.Geometry(d.seq_lens, d.cu_q, d.block_table, c.P, c.max_len, 0)
    none = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device=DEV)
    ws = _lib.workspace(256, DEV)
    _lib.dsa_gqa_append(geom, d.cache, none, none, none, none, ws=ws)
    _lib.dsa_gqa_attend(geom, d.cache, none, 0.1, none, None, ws)
    _lib.dsa_block_select(geom, d.cache, none, 2, 0, 1, torch.zeros(0, 2, 2, dtype=torch.int32, device=DEV), ws)
    _lib.dsa_gqa_attend_blocks(geom, d.cache, none, torch.zeros(0, 2, 2, dtype=torch.int32, device=DEV), 0.1, none, None, ws)
    assert _lib.dsa_get_error(ws) == 0


# ---------------------------------------------------------------- batches and sizes at the edges

def test_attend_rows_between_warps_and_tiles():
    """33 to 64 query rows per request and key head under long tables (the declared lengths
    choose the kernel), with short contexts in them."""
    for dtype in (E4, I8):
        c = ref.Case([700, 90, 6], [6, 4, 5], 16, 2, 128, dtype, seed=17, pad=2, max_len=64 * 2600)
        check_attend(Dev(c), 0.09)


@pytest.mark.parametrize("dtype", [E4, I8], ids=["e4m3", "i8"])
@pytest.mark.parametrize("lens,new,H,Hkv,D", [
    ([1558, 143], [75, 3], 40, 8, 128), ([700, 249, 60], [40, 90, 8], 14, 2, 64), ([64], [16], 8, 1, 128),
    ([1500, 700, 64, 900], [9, 14, 1, 40], 24, 4, 128), ([3000, 5, 2000], [12, 5, 8], 16, 2, 64),
    ([90 + 7 * i % 170 for i in range(70)], [1 + 3 * i % 10 for i in range(70)], 21, 3, 128)])
def test_attend_sharp_softmax(lens, new, H, Hkv, D, dtype):
    """Weights on few keys: the running maximum moves often and at different units for the
    rows of one tile, so that its warps drift apart. The same bits every time."""
    c = ref.Case(lens, new, H, Hkv, D, dtype, seed=71, pad=1, max_len=max(lens) if len(lens) < 9 else 64 * 300)
    d = Dev(c)
    a, la = check_attend(d, 0.5)
    for _ in range(5):
        b, lb = d.attend(0.5)
        assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("lens,new,H,Hkv,D", [
    ([900] + [70 + 5 * i for i in range(40)], [500] + [1] * 40, 16, 2, 128),     # a prompt among decoding requests
    ([150] + [40 + i for i in range(120)], [100] + [1] * 120, 8, 1, 64),
    ([33] * 700 + [200, 9], [0] * 700 + [3, 1], 4, 2, 64),                       # slots without tokens
    ([0, 65, 0] * 200 + [130], [1, 0, 1] * 200 + [2], 2, 1, 128), ([65] * 2, [2] * 2, 128, 128, 64), ([70], [2], 2048, 128, 64)])
def test_uneven_batches(lens, new, H, Hkv, D):
    c = ref.Case(lens, new, H, Hkv, D, E4, seed=len(lens), pad=3)
    d = Dev(c)
    check_attend(d, D ** -0.5)
    got = d.select(3, 1, 1)
    assert _lib.dsa_get_error(d.ws) == 0
    n = sum(new)
    assert np.array_equal(got[:n].cpu().numpy(), ref.select(c, 3, 1, 1)[:n])
    check_attend(d, D ** -0.5, blocks=got.cpu())


@pytest.mark.parametrize("new", [1, 3, 40])
def test_far_pages(new):
    """Codes beyond 2^32 bytes: the same answers, bit for bit, as from a small cache."""
    c = ref.Case([400, 130], [new, new], 16, 1, 64, E4, seed=14)
    near, far = Dev(c), Dev(c)
    P = 2 ** 20 + 4096
    at = [(i + 1) * (P // c.P) - 1 for i in range(c.P)]
    assert at[-1] * 64 * 64 > 2 ** 32
    for name in ("k", "v", "k_scale", "v_scale", "k_mean", "k_mean_scale"):
        x = getattr(near, name)
        big = torch.empty((P,) + tuple(x.shape[1:]), dtype=x.dtype, device=DEV)
        for i, p in enumerate(at):
            big[p].view(torch.uint8).copy_(x[i].view(torch.uint8))
        setattr(far, name, big)
    bt = c.block_table.clone()
    for i, p in enumerate(at):
        bt[c.block_table == i] = p
    far.block_table = bt.to(DEV)
    far.geom = _lib.Geometry(far.seq_lens, far.cu_q, far.block_table, P, c.max_len, c.T)
    far.cache = _lib.GqaCache(far.k, far.v, far.k_scale, far.v_scale, far.k_mean, far.k_mean_scale)
    x = torch.randn(c.T, 18, 64, generator=c.gen).bfloat16().to(DEV)
    got = []
    for d in (near, far):
        q = torch.zeros(c.T, 16, 64, dtype=torch.bfloat16, device=DEV)
        ws = _lib.workspace(256, DEV)
        _lib.dsa_gqa_append(d.geom, d.cache, x[:, 16:17], x[:, 17:], x[:, :16], q, 0, ws=ws)
        sel = d.select(4, 1, 1)
        a, la = d.attend(0.125)
        b, lb = d.attend(0.125, sel)
        assert _lib.dsa_get_error(ws) == 0 and _lib.dsa_get_error(d.ws) == 0
        pages = list(range(c.P)) if d is near else at
        held = [torch.stack([getattr(d, n)[p].view(torch.uint8) for p in pages]) for n in ("k", "v", "k_scale", "v_scale", "k_mean", "k_mean_scale")]
        got.append([q, sel, a, la, b, lb] + held)
    for u, w in zip(*got):
        assert torch.equal(u, w)


@pytest.mark.parametrize("new", [1, 64])
def test_many_rows(new):
    """Queries and outputs of more than 2^32 elements: the first and the last request."""
    H, Hkv, D, n = 64, 4, 128, 1
    B = 2 ** 32 // (H * D * new) + 3
    c = ref.Case([64], [new], H, Hkv, D, I8, seed=15)
    d = Dev(c)
    T = B * new
    seq = torch.full((B,), 64, dtype=torch.int32, device=DEV)
    cu = torch.arange(B + 1, dtype=torch.int32, device=DEV) * new
    bt = d.block_table.expand(B, 1).contiguous()
    geom = _lib.Geometry(seq, cu, bt, c.P, 64, T)
    q = torch.zeros(T, H, D, dtype=torch.bfloat16, device=DEV)
    q[:new], q[-new:] = d.q, d.q
    out, lse = torch.full_like(q, 7.0), torch.full((T, H), 7.0, device=DEV)
    r = ref.attend(c, 0.09)
    bo, bl = ref.attend_bounds(r)
    blocks = torch.full((T, Hkv, n), -9, dtype=torch.int32, device=DEV)
    for listed in (False, True):
        if listed:
            ws = _lib.workspace(max(_lib.dsa_block_select_workspace_size(geom, d.cache, n),
                                    _lib.dsa_gqa_attend_blocks_workspace_size(geom, d.cache, H, n)), DEV)
            _lib.dsa_block_select(geom, d.cache, q, n, 0, 1, blocks, ws)
            assert (blocks == 0).all()
            _lib.dsa_gqa_attend_blocks(geom, d.cache, q, blocks, 0.09, out, lse, ws)
        else:
            ws = _lib.workspace(_lib.dsa_gqa_attend_workspace_size(geom, d.cache, H), DEV)
            _lib.dsa_gqa_attend(geom, d.cache, q, 0.09, out, lse, ws)
        assert _lib.dsa_get_error(ws) == 0
        for part in (slice(0, new), slice(T - new, T)):
            assert (np.abs(out[part].double().cpu().numpy() - r["out"]) <= bo).all()
            assert (np.abs(lse[part].double().cpu().numpy() - r["lse"]) <= bl).all()
        assert torch.isfinite(lse).all()
        out.fill_(7.0), lse.fill_(7.0)


def test_two_graphs_share_a_workspace():
    """A decode step and a prompt's step, captured with one workspace and replayed in turn."""
    a = Dev(ref.Case([700, 3000], [1, 1], 16, 2, 128, E4, seed=18))
    b = Dev(ref.Case([300, 250], [200, 90], 16, 2, 128, I8, seed=19))
    want = [x.attend(0.09) for x in (a, b)]
    ws = _lib.workspace(max(_lib.dsa_gqa_attend_workspace_size(x.geom, x.cache, 16) for x in (a, b)), DEV)
    graphs, got = [], []
    for x in (a, b):
        out, lse = torch.zeros_like(want[len(got)][0]), torch.zeros_like(want[len(got)][1])
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            _lib.dsa_gqa_attend(x.geom, x.cache, x.q, 0.09, out, lse, ws)
        graphs.append(g), got.append((out, lse))
    for i in (0, 1, 1, 0, 1):
        got[i][0].fill_(7.0), got[i][1].fill_(7.0)
        graphs[i].replay()
        assert torch.equal(got[i][0], want[i][0]) and torch.equal(got[i][1], want[i][1])
    assert _lib.dsa_get_error(ws) == 0


def test_two_streams_at_once():
    """Calls on two streams, each with a workspace of its own, over one cache."""
    c = ref.Case([5000, 3000, 900], [1, 2, 1], 16, 2, 128, E4, seed=20)
    d = Dev(c)
    li = d.select(6, 1, 2)
    want, listed = d.attend(0.09), d.attend(0.09, li)
    size = max(_lib.dsa_gqa_attend_workspace_size(d.geom, d.cache, 16), _lib.dsa_gqa_attend_blocks_workspace_size(d.geom, d.cache, 16, 6))
    wss = [_lib.workspace(size, DEV) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, (s, ws) in enumerate(zip(streams, wss)):
            with torch.cuda.stream(s):
                out, lse = torch.zeros_like(want[0]), torch.zeros_like(want[1])
                if i:
                    _lib.dsa_gqa_attend_blocks(d.geom, d.cache, d.q, li, 0.09, out, lse, ws)
                else:
                    _lib.dsa_gqa_attend(d.geom, d.cache, d.q, 0.09, out, lse, ws)
                got[i].append((out, lse))
    torch.cuda.synchronize()
    for i, right in enumerate((want, listed)):
        assert all(torch.equal(o, right[0]) and torch.equal(l, right[1]) for o, l in got[i])
        assert _lib.dsa_get_error(wss[i]) == 0


@pytest.mark.parametrize("lens,new,H,Hkv,D", [
    ([130, 64, 5, 300, 1], [1, 1, 2, 3, 1], 8, 1, 64), ([200, 90, 700], [20, 33, 64], 16, 2, 128), ([75] * 30, [70] * 30, 12, 3, 64)])
def test_attend_nan_reaches_those_who_see_it(lens, new, H, Hkv, D):
    """NaN codes at random visible places: a value's reaches its column of the rows that see
    it, a key's the whole row, and nothing else changes."""
    c = ref.Case(lens, new, H, Hkv, D, E4, seed=23, pad=1)
    kb, vb = c.k.view(torch.uint8), c.v.view(torch.uint8)
    for b, m in enumerate(lens):
        for i in range(3):
            pos = m - 1 - int(torch.randint(0, min(m, 100), (1,), generator=c.gen))
            (kb if b % 3 == 2 and i == 0 else vb)[int(c.block_table[b, pos // 64]), (b + i) % Hkv, pos % 64, (37 * b + i) % D] = 0x7F if i else 0xFF
    d = Dev(c)
    li = lists(c, 3, "random")
    n = sum(new)
    for blocks in (None, li):
        out, lse = d.attend(0.2, None if blocks is None else blocks.to(DEV))
        with np.errstate(invalid="ignore"):
            r = ref.attend(c, 0.2, blocks)
            bo, bl = ref.attend_bounds(r)
        got, want = out.double().cpu().numpy()[:n], r["out"][:n]
        assert np.isnan(want).any() and np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(np.isnan(lse[:n].cpu().numpy()), np.isnan(r["lse"][:n]))
        ok = np.isfinite(want) & np.isfinite(bo[:n])       # (a NaN value has no bound for its key head's rows: `top`)
        assert (np.abs(got - want)[ok] <= bo[:n][ok]).all()
