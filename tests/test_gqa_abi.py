"""Refusals of the grouped-query entry points, before anything reaches a GPU (the C
functions take dummy addresses here and return without a launch)."""
import ctypes as C
import os

import pytest
import torch

from dsa_sparse_attention_02_gb300 import _lib

INV, UNS, WSP, OK = _lib.DSA_ERR_INVALID_ARG, _lib.DSA_ERR_UNSUPPORTED, _lib.DSA_ERR_WORKSPACE, _lib.DSA_OK
BIG = 1 << 40


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_lib.LIB_PATH):
        from dsa_sparse_attention_02_gb300 import build
        build.build()
    return _lib.load()


def geom(**kw):
    g = dict(B=1, T=1, max_seq_len=128, num_pages=4, page_size=64, bt_stride=2, seq_lens=16, cu_q=16, block_table=16)
    g.update(kw)
    return _lib.dsa_geom_t(*g.values())


def cache(**kw):
    c = dict(dtype=_lib.DSA_E4M3, Hkv=2, D=128, k=16, v=16, k_scale=16, v_scale=16, k_mean=16, k_mean_scale=16)
    c.update(kw)
    return _lib.dsa_gqa_cache_t(*c.values())


BAD_GEOM = [(dict(page_size=32), UNS), (dict(T=-1), INV), (dict(B=0), INV), (dict(bt_stride=1), INV), (dict(max_seq_len=0), INV),
            (dict(seq_lens=None), INV), (dict(cu_q=None), INV), (dict(block_table=None), INV), (dict(num_pages=0), INV)]
BAD_CACHE = [(dict(dtype=_lib.DSA_BF16), INV), (dict(dtype=9), INV), (dict(Hkv=0), INV), (dict(Hkv=129), INV), (dict(D=96), UNS),
             (dict(D=256), UNS), (dict(D=0), UNS)]
BAD_CODES = [dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(k=24), dict(v=8), dict(k_scale=18), dict(v_scale=17)]


def sweep(call, with_codes=True):
    for kw, want in BAD_GEOM:
        assert call(g=geom(**kw)) == want, kw
    for kw, want in BAD_CACHE:
        assert call(c=cache(**kw)) == want, kw
    if with_codes:
        for kw in BAD_CODES:
            assert call(c=cache(**kw)) == INV, kw
    assert call(g=None) == INV and call(c=None) == INV
    assert call(ws=None) == WSP and call(ws=264) == WSP and call(wb=255) == WSP
    assert call(g=geom(T=0)) == OK and call(g=geom(T=0, B=0)) == OK


def ref(x):
    return None if x is None else C.byref(x)


def test_append_refusals(lib):
    def call(g=geom(), c=cache(), k=16, ks=256, v=16, vs=256, H=8, q=16, qs=1024, qo=16, rope=64, cos=16, sin=16, ws=256, wb=BIG):
        return lib.dsa_gqa_append(ref(g), ref(c), k, ks, v, vs, H, q, qs, qo, rope, cos, sin, ws, wb, None)
    sweep(call)
    for kw in (dict(k=None), dict(v=None), dict(k=8), dict(v=20), dict(ks=255), dict(vs=248), dict(ks=257), dict(qs=1016), dict(qs=1028),
               dict(q=None), dict(qo=None), dict(qo=24), dict(q=18), dict(H=7), dict(H=0), dict(H=34), dict(rope=-8), dict(rope=12),
               dict(rope=136), dict(cos=None), dict(sin=None), dict(cos=24), dict(sin=8), dict(c=cache(k_mean=None)),
               dict(c=cache(k_mean_scale=None)), dict(c=cache(k_mean=24)), dict(c=cache(k_mean_scale=18))):
        assert call(**kw) == INV, kw
    assert call(c=cache(D=64), rope=72) == INV


def test_attend_refusals(lib):
    def call(g=geom(), c=cache(k_mean=None, k_mean_scale=None), H=8, q=16, qs=1024, sm=0.1, out=16, lse=16, ws=256, wb=BIG):
        return lib.dsa_gqa_attend(ref(g), ref(c), H, q, qs, sm, out, lse, ws, wb, None)
    sweep(call)
    for kw in (dict(H=0), dict(H=3), dict(H=34), dict(q=None), dict(q=8), dict(qs=1000), dict(qs=1025), dict(sm=float("nan")), dict(sm=3e38),
               dict(sm=float("inf")), dict(sm=-0.5), dict(out=None), dict(out=8), dict(lse=18)):
        assert call(**kw) == INV, kw
    assert call(wb=lib.dsa_gqa_attend_workspace_size(ref(geom()), ref(cache()), 8) - 1) == WSP
    assert call(g=geom(num_pages=1 << 24), c=cache(Hkv=128), H=128) == UNS


def test_attend_blocks_refusals(lib):
    def call(g=geom(), c=cache(k_mean=None, k_mean_scale=None), H=8, q=16, qs=1024, bl=16, n=3, sm=0.1, out=16, lse=None, ws=256, wb=BIG):
        return lib.dsa_gqa_attend_blocks(ref(g), ref(c), H, q, qs, bl, n, sm, out, lse, ws, wb, None)
    sweep(call)
    for kw in (dict(bl=None), dict(bl=18), dict(n=0), dict(n=-1), dict(n=32769), dict(H=5), dict(q=None), dict(out=None)):
        assert call(**kw) == INV, kw
    assert call(wb=lib.dsa_gqa_attend_blocks_workspace_size(ref(geom()), ref(cache()), 8, 3) - 1) == WSP


def test_select_refusals(lib):
    def call(g=geom(), c=cache(k=None, v=None, k_scale=None, v_scale=None), H=8, q=16, qs=1024, n=4, f=1, la=2, bl=16, ws=256, wb=BIG):
        return lib.dsa_block_select(ref(g), ref(c), H, q, qs, n, f, la, bl, ws, wb, None)
    sweep(call, with_codes=False)
    for kw in (dict(n=0), dict(n=1025), dict(f=-1), dict(la=0), dict(f=3, la=2), dict(f=2 ** 31 - 1, la=2), dict(la=2 ** 31 - 1),
               dict(bl=None), dict(bl=18), dict(q=None), dict(H=6, c=cache(Hkv=4)), dict(c=cache(k_mean=None)),
               dict(c=cache(k_mean_scale=None)), dict(c=cache(k_mean=8))):
        assert call(**kw) == INV, kw
    assert call(g=geom(max_seq_len=(1 << 21) + 1, bt_stride=1 << 16)) == UNS


def test_workspace_sizes_of_refused_arguments(lib):
    for fn, more in ((lib.dsa_gqa_attend_workspace_size, (8,)), (lib.dsa_gqa_attend_blocks_workspace_size, (8, 4))):
        assert fn(None, ref(cache()), *more) == 256 and fn(ref(geom()), None, *more) == 256
        assert fn(ref(geom(T=0)), ref(cache()), *more) == 256


@pytest.mark.parametrize("B,H,Hkv,D,max_len", [(1, 8, 8, 128, 4096), (32, 40, 8, 128, 16384), (7, 16, 1, 64, 300), (64, 128, 8, 64, 131072)])
def test_workspace_sizes_grow_with_the_tokens(lib, B, H, Hkv, D, max_len):
    c = cache(Hkv=Hkv, D=D)
    for size in (lambda g: lib.dsa_gqa_attend_workspace_size(ref(g), ref(c), H),
                 lambda g: lib.dsa_gqa_attend_blocks_workspace_size(ref(g), ref(c), H, 16)):
        got = [size(geom(B=B, T=T, max_seq_len=max_len, bt_stride=max_len // 64 + 1)) for T in list(range(1, 40 * B)) + [10 ** 4, 10 ** 6]]
        assert got == sorted(got) and got[0] > 256


def test_binding_refuses_tensors_that_do_not_fit():
    k = torch.zeros(3, 2, 64, 64, dtype=torch.int8)
    sc = torch.zeros(3, 2)
    for bad in ((k.float(), k, sc, sc), (k[:, :, :32], k, sc, sc), (k, k[:2], sc, sc), (k, k.view(torch.float8_e4m3fn), sc, sc),
                (k, k, sc[:, :1], sc), (k, k, sc.double(), sc), (k, k, sc, sc.t()), (k, k, sc, sc, torch.zeros(3, 2, 64, dtype=torch.int8)),
                (k, k, sc, sc, torch.zeros(3, 2, 32, dtype=torch.int8), sc),
                (k, k, sc, sc)):                      # the last fits, but is on the host
        with pytest.raises(TypeError):
            _lib.GqaCache(*bad)

    class Handle:                                     # a cache and a geometry without a device
        D, Hkv, T, num_pages, device, index = 64, 2, 5, 3, torch.device("cpu"), -1

    h = Handle()
    for bad in (torch.zeros(5, 4, 64), torch.zeros(4, 4, 64, dtype=torch.bfloat16), torch.zeros(5, 4, 32, dtype=torch.bfloat16),
                torch.zeros(5, 64, 4, dtype=torch.bfloat16).transpose(1, 2), torch.zeros(5, 8, 64, dtype=torch.bfloat16)[:, ::2]):
        with pytest.raises(TypeError):
            _lib._heads("q", bad, h, h)
    with pytest.raises(TypeError):
        _lib._heads("out", torch.zeros(5, 8, 64, dtype=torch.bfloat16)[:, :4], h, h, 4, False)
    with pytest.raises(TypeError):
        _lib._plain("blocks", torch.zeros(5, 2, 3, dtype=torch.int64), torch.int32, (5, 2, 3), h)
    h.device, h.index = torch.device("cuda", 0), 0    # now a cache on a GPU: host tensors do not fit
    with pytest.raises(ValueError):
        _lib._plain("blocks", torch.zeros(5, 2, 3, dtype=torch.int32), torch.int32, (5, 2, 3), h)
    with pytest.raises(ValueError):
        _lib._heads("q", torch.zeros(5, 4, 64, dtype=torch.bfloat16), h, h)
