"""Expanded latent attention over ragged keys against its definition in 64 bits: prompts of one
token and of thousands, heads, strides, queries without keys, values that are not finite."""
import math

import numpy as np
import pytest
import torch

import latent_reference as ref
from dsa_sparse_attention_02_gb300 import _lib
from test_gpu_latent_attend import compare

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
SM = 192 ** -0.5


class Batch:
    def __init__(self, lens, new, H, seed=0, pad_q=0, pad_k=0, fused=True):
        g = self.gen = torch.Generator().manual_seed(seed)
        self.lens, self.new, self.H = lens, new, H
        self.cu_q = [0] + np.cumsum(new).tolist()
        self.cu_k = [0] + np.cumsum(lens).tolist()
        self.T, self.S = sum(new) + pad_q, sum(lens) + pad_k
        self.q = torch.randn(self.T, H, 192, generator=g).bfloat16()
        self.kv = torch.randn(self.S, H, 256, generator=g).bfloat16()
        self.rows = torch.randn(self.S, 576, generator=g).bfloat16()
        self.k, self.v, self.rope = self.kv[..., :128], self.kv[..., 128:], self.rows[:, 512:]
        if not fused:
            self.k, self.v, self.rope = self.k.contiguous(), self.v.contiguous(), self.rope.contiguous()
        self.upload()

    def upload(self):
        kv, rows = self.kv.to(DEV), self.rows.to(DEV)
        self.d = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in (self.cu_q, self.cu_k)] + [self.q.to(DEV)]
        self.d += [kv[..., :128], kv[..., 128:], rows[:, 512:]] if self.k.stride(-2) != 128 else [x.to(DEV) for x in (self.k, self.v, self.rope)]

    def attend(self, sm=SM, lse=True, ws=None, stream=None, **kw):
        names = ("cu_q", "cu_k", "q", "k", "v", "k_rope")
        a = {n: kw.get(n, x) for n, x in zip(names, self.d)}
        out = torch.full((self.T, self.H, 128), 7.0, dtype=torch.bfloat16, device=DEV)
        le = torch.full((self.T, self.H), 7.0, device=DEV) if lse else None
        self.ws = ws if ws is not None else _lib.workspace(
            _lib.dsa_latent_attend_expanded_workspace_size(len(self.lens), self.T, self.S, self.H), DEV)
        _lib.dsa_latent_attend_expanded(*a.values(), sm, out, le, self.ws, stream)
        return out, le

    def check(self, sm=SM, ts=None):
        out, lse = self.attend(sm)
        assert _lib.dsa_get_error(self.ws) == 0
        n = sum(self.new)
        assert (out[n:] == 7.0).all() and (lse[n:] == 7.0).all()
        compare(ref.expanded(self.q, self.k, self.v, self.rope, self.cu_q, self.cu_k, sm, ts), out, lse)
        again = self.attend(sm)
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
        return out, lse


@pytest.mark.parametrize("lens,new,H,pad_q,pad_k", [
    ([1], [1], 1, 0, 0), ([128], [128], 2, 0, 0), ([129], [1], 16, 2, 3), ([257, 256], [257, 255], 3, 0, 0), ([70, 1, 300], [70, 1, 5], 5, 1, 0),
    ([0, 5, 127], [2, 9, 127], 4, 3, 1), ([640], [300], 1, 0, 0), ([64, 0, 65], [1, 0, 1], 20, 0, 200), ([200], [2], 128, 0, 0)])
@pytest.mark.parametrize("fused", [True, False])
def test_expanded(lens, new, H, pad_q, pad_k, fused):
    Batch(lens, new, H, sum(lens) + H, pad_q, pad_k, fused).check()


def test_expanded_without_keys():
    b = Batch([0, 0], [3, 1], 2)
    out, lse = b.check()
    assert (out == 0).all() and torch.isneginf(lse).all()


@pytest.mark.parametrize("lens,new,H", [([5000], [1500], 4), ([3001, 17, 900], [3001, 17, 1], 2), ([30000], [3], 3), ([2048], [2048], 32)])
def test_expanded_long(lens, new, H):
    b = Batch(lens, new, H, 7)
    n = sum(new)
    b.check(ts={0, n - 1, n // 2, n // 3, 255, 256} & set(range(n)))


def test_expanded_many_requests():
    lens = [(91 * i) % 300 for i in range(500)]
    new = [min((7 * i) % 40, n + 2) for i, n in enumerate(lens)]
    b = Batch(lens, new, 2, 8)
    b.check(ts=set(range(0, b.T, 97)))


def test_expanded_scales():
    b = Batch([300, 40], [40, 40], 3, 9)
    b.check(0.0)
    b.q *= 16
    b.upload()
    b.check(1.0)                                  # the reference maximum moves
    b = Batch([1024], [2], 2, 10)                 # rising and falling scores
    b.q.zero_()
    b.q[0, :, 128], b.q[1, :, 128] = 1.0, -1.0
    b.rows[:, 512] = torch.arange(1024) / 4
    b.upload()
    b.check(1.0)


@pytest.mark.parametrize("what", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("where", ["v", "k", "rope"])
def test_expanded_values_that_are_not_finite(where, what):
    """Keys of no request, of other requests and behind a row's own change nothing; those seen
    reach the head (or all heads, by the rotated part) and rows from theirs on."""
    b = Batch([200, 300], [200, 140], 3, 11, pad_k=70)
    clean = b.attend()

    def spoil(s):
        (b.rows[s] if where == "rope" else b.kv[s, 1])[{"v": 128 + 17, "k": 9, "rope": 512 + 3}[where]] = what

    for s in range(500, 570):
        spoil(s)
    b.upload()
    got = b.attend()
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
    spoil(90)
    spoil(200 + 160 + 70)                          # seen by request 1's rows from 70 on
    b.upload()
    got = b.attend()
    sees = torch.zeros(b.T, b.H, dtype=torch.bool)
    sees[90:200] = sees[200 + 70:] = True
    if where != "rope":
        sees[:, [0, 2]] = False
    assert torch.equal(got[0][~sees], clean[0][~sees]) and torch.equal(got[1][~sees], clean[1][~sees])
    if where == "v":
        assert not torch.isfinite(got[0][sees][:, 17].float()).any() and torch.equal(got[1], clean[1])
        keep = torch.arange(128) != 17
        assert torch.equal(got[0][sees][:, keep], clean[0][sees][:, keep])
    elif math.isnan(what):
        assert torch.isnan(got[0][sees].float()).all()


def test_expanded_bad_requests():
    b = Batch([100, 80, 64], [3, 2, 4], 2, 12)
    want = b.attend()
    for name, i, v in (("cu_k", 2, 90), ("cu_k", 3, 10 ** 6), ("cu_k", 1, -4), ("cu_q", 3, b.T + 1)):
        bad = (b.d[0] if name == "cu_q" else b.d[1]).clone()
        bad[i] = v
        out, lse = b.attend(**{name: bad})
        assert _lib.dsa_get_error(b.ws) == _lib.DSA_ERR_BAD_INDEX
        hit = {("cu_k", 2): [1], ("cu_k", 3): [2], ("cu_k", 1): [0, 1], ("cu_q", 3): [2]}[name, i]
        for r in range(3):
            sl = slice(b.cu_q[r], b.cu_q[r + 1])
            if r in hit:
                assert (out[sl] == 0).all() and torch.isneginf(lse[sl]).all(), (name, i, r)
            elif not (name == "cu_k" and (i == r or i == r + 1)):
                assert torch.equal(out[sl], want[0][sl]) and torch.equal(lse[sl], want[1][sl])


def test_expanded_streams_graphs_and_strides():
    b = Batch([300, 70], [33, 70], 3, 13)
    want = b.attend()
    assert torch.equal(b.attend(lse=False)[0], want[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = [torch.zeros_like(b.ws) for _ in range(2)]
    got = b.attend(ws=ws[0], stream=side) + b.attend(ws=ws[1])
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(got, want + want))
    wide = torch.randn(b.T, 5, 256, device=DEV).bfloat16()
    wide[:, 1:4, 64:] = b.d[2]
    got = b.attend(q=wide[:, 1:4, 64:])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    heads_first = b.d[3].transpose(0, 1).contiguous().transpose(0, 1)
    got = b.attend(k=heads_first)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        o, l = torch.empty_like(want[0]), torch.empty_like(want[1])
        _lib.dsa_latent_attend_expanded(*b.d, SM, o, l, ws[0])
    for cu_q, cu_k in (([0, 1, 103], [0, 299, 370]), ([0, 33, 40], [0, 0, 64]), ([0, 50, 103], [0, 300, 370])):
        b.d[0].copy_(torch.tensor(cu_q))
        b.d[1].copy_(torch.tensor(cu_k))
        b.d[2].copy_(torch.randn(b.q.shape, generator=b.gen).bfloat16())
        o.fill_(7.0)
        l.fill_(7.0)
        g.replay()
        want = b.attend(ws=ws[1])
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])


def test_expanded_refusals_of_the_binding():
    b = Batch([10], [10], 2, 14)
    b.attend()
    for bad in (dict(q=b.d[2][..., :128]), dict(k=b.d[3][:, :1]), dict(v=b.d[4].float()), dict(k_rope=b.rows[:, :64]), dict(cu_q=b.d[0].long()),
                dict(cu_k=b.d[1][:1]), dict(v=None)):
        with pytest.raises(TypeError):
            b.attend(**bad)
    with pytest.raises(_lib.DsaError):
        b.attend(ws=_lib.workspace(256, DEV))


@pytest.mark.parametrize("lens,new,H", [([1000], [1], 1), ([129, 128, 127], [3, 128, 1], 2), ([2000, 900, 40], [128, 100, 40], 16), ([600], [128], 3)])
def test_expanded_few_rows(lens, new, H):
    """At most 128 rows a request in the mean: units of an item alternate between two places; items
    of one unit, cut items, items longer than the mean."""
    b = Batch(lens, new, H, 21)
    n = sum(new)
    b.check(ts={0, n - 1, n // 2, n // 3})
    b = Batch([700, 64, 64, 64], [300, 1, 1, 1], H, 22)
    b.check(ts={0, 127, 128, 255, 256, 299, 300, 302})


def test_expanded_few_rows_nan():
    """A NaN among the first of many units, whose weight is nothing beside later ones, is still seen."""
    b = Batch([1024, 1024], [2, 2], 2, 23)
    b.q.zero_()
    b.q[:, :, 128] = 8.0
    b.rows[:, 512] = torch.arange(2048) % 1024 / 4
    b.kv[5, 0, 128 + 9] = math.nan
    b.upload()
    out, lse = b.attend(1.0)
    want = torch.zeros(4, 2, 128, dtype=torch.bool)
    want[:2, 0, 9] = True
    assert torch.equal(torch.isnan(out.float()).cpu(), want) and torch.isfinite(lse).all()
