"""Refusals of the dense latent entry points and of their binding, before anything reaches a
GPU (the C functions take dummy addresses here and return without a launch), the rotary
frequencies, and the plain definitions the GPU tests compare with."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

import latent_reference as ref
from dsa_sparse_attention_02_gb300 import _lib
from test_gqa_abi import BAD_GEOM, BIG, INV, OK, UNS, WSP, geom, lib  # noqa: F401
from test_gqa_abi import ref as by

BF16, E4, I8 = _lib.DSA_BF16, _lib.DSA_E4M3, _lib.DSA_I8


def rope(**kw):
    r = _lib.Rope().c
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def check_common(call):
    for kw, want in BAD_GEOM:
        assert call(g=geom(**kw)) == want, kw
    assert call(g=None) == INV
    assert call(ws=None) == WSP and call(ws=264) == WSP and call(wb=255) == WSP
    assert call(dt=3) == INV and call(dt=-1) == INV


def test_append_refusals(lib):  # noqa: F811
    def call(g=geom(), dt=E4, kv=16, ks=576, gm=16, eps=1e-6, r=rope(), cache=16, ko=16, H=8, q=16, qt=1536, qh=192, qo=32, ot=512,
             oh=64, ws=256, wb=BIG):
        return lib.dsa_latent_append(by(g), dt, kv, ks, gm, eps, by(r), cache, ko, H, q, qt, qh, qo, ot, oh, ws, wb, None)
    check_common(call)
    for kw in (dict(kv=8), dict(ks=575), dict(ks=568), dict(ks=580), dict(gm=8), dict(eps=-1e-6), dict(eps=math.nan), dict(eps=math.inf),
               dict(r=None), dict(r=rope(dim=0)), dict(r=rope(dim=8)), dict(r=rope(dim=80)), dict(r=rope(dim=24)), dict(r=rope(scale=math.nan)),
               dict(cache=None), dict(cache=24), dict(ko=8), dict(H=0), dict(H=129), dict(q=None), dict(qo=None), dict(q=24), dict(qo=8),
               dict(qt=56), dict(qt=68), dict(qh=56), dict(qh=66), dict(ot=60), dict(oh=60), dict(kv=None), dict(kv=None, cache=None),
               dict(kv=None, cache=None, ko=None, q=None, qo=None)):
        assert call(**kw) == INV, kw
    assert call(g=geom(T=0)) == OK and call(g=geom(T=0, B=0)) == OK
    assert call(g=geom(T=(1 << 31) - 1), H=128) == UNS


def test_attend_refusals(lib):  # noqa: F811
    def call(g=geom(), dt=E4, H=16, q=16, cache=16, sm=0.1, out=16, lse=16, ws=256, wb=BIG):
        return lib.dsa_latent_attend(by(g), dt, H, q, cache, sm, out, lse, ws, wb, None)
    check_common(call)
    for kw in (dict(H=0), dict(H=129), dict(H=-1), dict(q=None), dict(q=8), dict(cache=None), dict(cache=8), dict(out=None), dict(out=8),
               dict(lse=18), dict(sm=math.nan), dict(sm=math.inf), dict(sm=-0.1), dict(sm=3e38)):
        assert call(**kw) == INV, kw
    assert call(wb=lib.dsa_latent_attend_workspace_size(by(geom()), 16) - 1) == WSP
    assert call(g=geom(T=(1 << 31) - 1), H=2) == UNS
    assert call(g=geom(T=0)) == OK


def test_gather_refusals(lib):  # noqa: F811
    def call(g=geom(), dt=E4, cache=16, first=16, cu=16, S=5, out=16, st=576, ws=256, wb=BIG):
        return lib.dsa_latent_gather(by(g), dt, cache, first, cu, S, out, st, ws, wb, None)
    check_common(call)
    for kw in (dict(cache=None), dict(cache=8), dict(first=18), dict(cu=None), dict(cu=18), dict(S=-1), dict(out=None), dict(out=8),
               dict(st=575), dict(st=568), dict(st=580), dict(g=geom(T=0, B=0))):
        assert call(**kw) == INV, kw
    assert call(S=0) == OK


def test_expanded_refusals(lib):  # noqa: F811
    def call(B=2, T=4, S=8, cq=16, ck=16, H=2, q=16, qt=384, qh=192, k=16, kt=512, kh=256, v=16, vt=512, vh=256, r=16, rt=64, sm=0.1,
             out=16, lse=16, ws=256, wb=BIG):
        return lib.dsa_latent_attend_expanded(B, T, S, cq, ck, H, q, qt, qh, k, kt, kh, v, vt, vh, r, rt, sm, out, lse, ws, wb, None)
    for kw in (dict(B=-1), dict(B=0), dict(T=-1), dict(S=-1), dict(cq=None), dict(ck=None), dict(cq=18), dict(ck=18), dict(H=0), dict(H=129),
               dict(q=None), dict(q=8), dict(qt=184), dict(qt=388), dict(qh=184), dict(qh=196), dict(k=None), dict(k=8), dict(kt=120),
               dict(kt=516), dict(kh=120), dict(v=None), dict(v=24), dict(vt=124), dict(vh=64), dict(r=None), dict(r=8), dict(rt=56),
               dict(rt=68), dict(out=None), dict(out=8), dict(lse=18), dict(sm=-1.0), dict(sm=math.nan), dict(sm=3e38)):
        assert call(**kw) == INV, kw
    assert call(ws=None) == WSP and call(ws=264) == WSP
    assert call(wb=lib.dsa_latent_attend_expanded_workspace_size(2, 4, 8, 2) - 1) == WSP
    assert call(T=(1 << 31) - 1) == UNS and call(S=(1 << 31) - 1) == UNS
    assert call(T=0) == OK and call(T=0, B=0) == OK


def test_workspace_sizes(lib):  # noqa: F811
    assert lib.dsa_latent_attend_workspace_size(None, 16) == 256 and lib.dsa_latent_attend_workspace_size(by(geom(T=0)), 16) == 256
    for B, H in ((1, 1), (1, 16), (7, 5), (64, 128)):
        got = [lib.dsa_latent_attend_workspace_size(by(geom(B=B, T=T)), H) for T in list(range(1, 40 * B)) + [10 ** 4, 10 ** 6]]
        assert got == sorted(got) and got[0] > 256


@pytest.mark.parametrize("bad", [dict(dim=0), dict(dim=8), dict(dim=20), dict(dim=80), dict(base=1.0), dict(base=math.nan), dict(base=math.inf),
                                 dict(factor=0.5), dict(factor=math.nan), dict(original_len=-1), dict(attn_factor=math.inf),
                                 dict(original_len=4096, beta_slow=0.0), dict(original_len=4096, beta_fast=0.5),
                                 dict(original_len=4096, beta_fast=math.inf)])
def test_rope_refusals(lib, bad):  # noqa: F811
    with pytest.raises(_lib.DsaError, match="dsa_rope_init"):
        _lib.Rope(**bad)


@pytest.mark.parametrize("kw", [dict(), dict(dim=16), dict(dim=48, base=500.0), dict(factor=4.0), dict(dim=32, base=1e6, factor=40.0, original_len=4096),
                                dict(factor=8.0, original_len=1 << 20), dict(factor=40.0, original_len=2), dict(dim=64, factor=2.0, original_len=100, beta_fast=4.0, beta_slow=4.0)])
def test_rope_frequencies(lib, kw):  # noqa: F811
    """As fractions of 2^64 of a turn: off by one of those and the roundings of a few operations in 64 bits."""
    r = _lib.Rope(**kw)
    dim, base = kw.get("dim", 64), kw.get("base", 10000.0)
    f = ref.frequencies(dim, base, kw.get("factor", 1.0), kw.get("original_len", 0), kw.get("beta_fast", 32.0), kw.get("beta_slow", 1.0))
    if not kw.get("original_len"):
        f = base ** (-np.arange(0, dim, 2) / dim) / kw.get("factor", 1.0)
    got = np.array([r.c.turns[i] / 2.0 ** 64 for i in range(32)])
    assert np.abs(got[:dim // 2] - f / (2 * math.pi)).max() <= 2.0 ** -50 and (got[dim // 2:] == 0).all()
    assert r.c.dim == dim and r.c.interleaved == 1 and r.c.scale == 1.0


class Handle:
    """A geometry without a device."""
    T, B, num_pages = 3, 1, 2
    seq_lens = torch.zeros(1, dtype=torch.int32)


def test_binding_refuses_what_is_missing_or_does_not_fit():
    g, rows, ws = Handle(), torch.zeros(3, 576, dtype=torch.bfloat16), torch.zeros(256, dtype=torch.uint8)
    q = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="go together"):
        _lib.dsa_latent_append(g, BF16, rows, None, None, q_in=q, ws=ws)
    with pytest.raises(TypeError, match="go with kv_in"):
        _lib.dsa_latent_append(g, BF16, None, None, None, kv_out=rows, ws=ws)
    for bad in (None, torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros(512, dtype=torch.uint8)[::2]):
        with pytest.raises(TypeError, match="ws"):
            _lib.dsa_latent_append(g, BF16, rows, None, None, ws=bad)
        with pytest.raises(TypeError, match="ws"):
            _lib.dsa_latent_attend(g, BF16, q, rows, 0.1, q, None, bad)
        with pytest.raises(TypeError, match="ws"):
            _lib.dsa_latent_gather(g, BF16, rows, None, rows, rows, bad)
        with pytest.raises(TypeError, match="ws"):
            _lib.dsa_latent_attend_expanded(Handle.seq_lens, Handle.seq_lens, q, q, q, rows, 0.1, q, None, bad)
    with pytest.raises(ValueError):                   # CPU tensors
        _lib.dsa_latent_attend(g, BF16, q, rows, 0.1, q, None, ws)


def test_tensor_check():
    t = torch.zeros(4, 3, 64, dtype=torch.bfloat16)
    dt, i = torch.bfloat16, -1
    assert _lib._tensor("x", t, dt, (4, 3, 64), i)[1:] == (192, 64)
    assert _lib._tensor("x", t, dt, (4, 3, 64), i, 3)[1:] == ()
    wide = torch.zeros(4, 3, 192, dtype=dt)[..., 128:]
    assert _lib._tensor("x", wide, dt, (4, 3, 64), i)[1:] == (576, 192)
    one = torch.zeros(1, 1, 64, dtype=dt).as_strided((1, 1, 64), (1, 1, 1))     # strides that say nothing
    assert _lib._tensor("x", one, dt, (1, 1, 64), i)[1:] == (64, 64)
    for bad, inner in ((t.float(), 1), (t[:3], 1), (t.transpose(0, 1).contiguous(), 1), (torch.zeros(4, 3, 128, dtype=dt)[..., ::2], 1),
                       (wide, 2), (torch.zeros(8, 3, 64, dtype=dt)[::2], 3), (3, 1), (None, 1)):
        with pytest.raises(TypeError, match="x"):
            _lib._tensor("x", bad, dt, (4, 3, 64), i, inner)
    with pytest.raises(TypeError, match="cuda:0"):
        _lib._tensor("x", t, dt, (4, 3, 64), 0)


def test_cache_check():
    g = Handle()
    for dt, shape, kind in ((BF16, (2, 64, 576), torch.bfloat16), (E4, (2, 41984), torch.uint8), (I8, (2, 41984), torch.uint8)):
        t = torch.zeros(shape, dtype=kind)
        assert _lib._latent_cache(dt, t, g, -1) == t.data_ptr()
        for bad in (t[..., :-8], t.view(torch.int8 if kind is torch.uint8 else torch.float16), None, torch.zeros((4,) + shape[1:], dtype=kind)[::2]):
            with pytest.raises(TypeError, match="kv_cache"):
                _lib._latent_cache(dt, bad, g, -1)
        with pytest.raises(ValueError, match="pages"):
            _lib._latent_cache(dt, t[:1], g, -1)
    with pytest.raises(ValueError, match="kv_dtype"):
        _lib._latent_cache(7, t, g, -1)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "i8"])
def test_the_plain_definition(kind):
    """Attention of one key is that key; of a zero query the mean; a token at a negative position sees none."""
    c = ref.Case([1, 70, 2], [1, 2, 3], H=2, kind=kind)
    c.q[1:3] = 0
    r = ref.attend(c, 0.2)
    x, _ = c.rows(0)
    assert np.allclose(r[0][0], x[0, :512].numpy(), rtol=1e-12)
    assert np.allclose(r[0][1], 0.2 * (c.q[0].double() @ x[0]).numpy(), rtol=1e-12)
    y, _ = c.rows(1)
    assert np.allclose(r[1][0], y[:69, :512].mean(0).numpy()) and np.allclose(r[2][1], math.log(70))
    assert np.isneginf(r[3][1]).all() and (r[3][0] == 0).all() and np.isfinite(r[4][1]).all()
    f = ref.frequencies(64, 10000.0)
    v = np.random.default_rng(0).standard_normal((3, 64))
    for inter in (True, False):
        u, _ = ref.rotate(v, 1234, f, inter)
        assert np.allclose((u * u).sum(-1), (v * v).sum(-1)) and np.allclose(ref.rotate(u, -1234, f, inter)[0], v)
