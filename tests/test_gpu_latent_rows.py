"""Latent rows into the paged cache and out of it, against their definitions in 64 bits: norm,
rotation in both layouts at near and far positions, records' codes and scales, strides, rows that
are not to be touched; and a prompt and its decode through all four latent operators."""
import math

import numpy as np
import pytest
import torch

import latent_reference as ref
from dsa_sparse_attention_02_gb300 import _lib
from test_gpu_latent_attend import DEV, KIND, KINDS, Dev, compare

pytestmark = pytest.mark.gpu
EPS = 1e-6


def inputs(c, scale=1.5):
    g = c.gen
    return ((scale * torch.randn(c.T, 576, generator=g)).bfloat16(), 1 + 0.1 * torch.randn(512, generator=g),
            torch.randn(c.T, c.H, 64, generator=g).bfloat16())


def append(d, rope, kv, gamma, q, eps=EPS, keep=True, q_out=None, stream=None):
    c = d.c
    up = lambda x: None if x is None else x.to(DEV)  # noqa: E731
    rows = torch.full((c.T, 576), 7.0, dtype=torch.bfloat16, device=DEV) if keep else None
    qo = q_out if q_out is not None else torch.full((c.T, c.H, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    d.ws = _lib.workspace(_lib.dsa_latent_append_workspace_size(d.geom), DEV)
    _lib.dsa_latent_append(d.geom, d.kind, up(kv), d.cache, rope, gamma=up(gamma), eps=eps, q_in=up(q), q_out=qo, kv_out=rows, ws=d.ws,
                           stream=stream)
    return rows, qo


def verify(d, kv, gamma, q, f, inter, attn, rows, qo, eps=EPS, skip=()):
    """The append's outputs and the pages it wrote; every other byte of the cache as before."""
    c = d.c
    before, after = c.cache, d.cache.cpu()
    g = np.ones(512) if gamma is None else gamma.double().numpy()
    want = before.clone()
    for t, b, pos in c.tokens():
        x = kv[t].double().numpy()
        y, rel = ref.normed(x[:512], g, eps)
        k, bk = ref.rotate(x[512:], max(pos, 0), f, inter, attn)
        u, bu = ref.rotate(q[t].double().numpy(), max(pos, 0), f, inter, attn)
        assert (np.abs(qo[t].double().cpu().numpy() - u) <= bu).all(), t
        if rows is not None:
            r = rows[t].double().cpu().numpy()
            assert (np.abs(r[:512] - y) <= (ref.HALF + rel) * np.abs(y)).all() and (np.abs(r[512:] - k) <= bk).all(), t
        if pos < 0 or b in skip:
            continue
        p, s = c.slot(b, pos)
        if c.kind == "bf16":
            r = after[p, s].double().numpy()
            assert (np.abs(r[:512] - y) <= (ref.HALF + rel) * np.abs(y)).all() and (np.abs(r[512:] - k) <= bk).all(), t
            if rows is not None:
                assert torch.equal(after[p, s], rows[t].cpu())
            want[p, s] = after[p, s]
            continue
        (code, scale, rope), w = ref.planes(after), ref.planes(want)
        assert (np.abs(rope[p, s].double().numpy() - k) <= bk).all(), t
        amax = np.abs(y.reshape(4, 128)).max(1)
        sc = scale[p, s].double().numpy()
        assert (np.abs(sc - np.where(amax > 0, amax / ref.QMAX[c.kind], 1.0)) <= 2.0 ** -21 * sc).all(), t
        v = code[p, s].view(ref.CODE[c.kind]).double().numpy().reshape(4, 128)
        n = y.reshape(4, 128) / sc[:, None]
        step = 0.5 if c.kind == "i8" else np.maximum(2.0 ** -4 * np.abs(n), 2.0 ** -10)
        assert (np.abs(v - n) <= step + 2.0 ** -20 * np.abs(n)).all(), t
        for a, z in zip(w, (code, scale, rope)):
            a[p, s] = z[p, s]
    assert torch.equal(want.view(torch.uint8), after.view(torch.uint8))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,new,H,dim,inter,kw,pad", [
    ([1], [1], 1, 64, True, {}, 0), ([100, 64, 7], [3, 1, 7], 5, 64, False, {}, 2), ([70, 0, 2], [70, 1, 4], 16, 32, True, dict(base=500.0), 1),
    ([200, 65], [2, 65], 64, 16, False, dict(factor=4.0), 0), ([130], [130], 20, 48, True, dict(base=1e6, factor=40.0, original_len=4096, attn_factor=1.37), 0),
    ([90, 91], [1, 1], 128, 48, False, dict(factor=8.0, original_len=1024), 3)])
def test_append(lens, new, H, dim, inter, kw, pad, kind):
    c = ref.Case(lens, new, H, kind, seed=H + dim, pad=pad)
    kv, gamma, q = inputs(c)
    d = Dev(c)
    rows, qo = append(d, _lib.Rope(dim, interleaved=inter, **kw), kv, gamma, q)
    assert _lib.dsa_get_error(d.ws) == 0
    n = sum(new)
    assert (rows[n:] == 7.0).all() and (qo[n:] == 7.0).all()
    f = ref.frequencies(dim, kw.get("base", 10000.0), kw.get("factor", 1.0), kw.get("original_len", 0))
    verify(d, kv, gamma, q, f, inter, kw.get("attn_factor", 1.0), rows, qo)


@pytest.mark.parametrize("kind", KINDS)
def test_append_far_positions_and_sizes_of_values(kind):
    """Positions up to 2^20 (a block table whose front is no page); rows of zeros, of one value,
    tiny and large ones; gamma left out; eps 0."""
    c = ref.Case([128, 100], [66, 5], 3, kind, seed=3)
    far = 1 << 20
    table = torch.full((2, far // 64 + 2), -7, dtype=torch.int32)
    table[:, far // 64 - 2:] = c.block_table[:, :1].expand(2, 4)
    table[:, far // 64 - 2:far // 64] = c.block_table[:, :2]
    c.block_table, c.lens, c.max_len = table, [far, far - 28], far
    c.seq_lens = torch.tensor(c.lens, dtype=torch.int32)
    kv, _, q = inputs(c)
    kv[0, :512] = 0
    kv[1, :512] = 0
    kv[1, 5] = 2.0
    kv[2, :512] *= 2.0 ** -40
    kv[3, :512] *= 2.0 ** 40
    kv[4, 128:256] = 0
    d = Dev(c)
    rows, qo = append(d, _lib.Rope(), kv, None, q, eps=1e-12)
    assert _lib.dsa_get_error(d.ws) == 0
    verify(d, kv, None, q, ref.frequencies(64, 10000.0), True, 1.0, rows, qo, eps=float(np.float32(1e-12)))
    d = Dev(c)
    rows, qo = append(d, _lib.Rope(), kv[1:2].repeat(c.T, 1), None, q, eps=0.0)
    verify(d, kv[1:2].repeat(c.T, 1), None, q, ref.frequencies(64, 10000.0), True, 1.0, rows, qo, eps=0.0)


def test_append_strides_in_place_and_parts():
    """Columns of a projection's output, queries rotated where they lie, rows alone, queries alone, another stream."""
    c = ref.Case([300, 64], [40, 1], 6, "e4m3", seed=4)
    kv, gamma, q = inputs(c)
    r = _lib.Rope(interleaved=False)
    a = Dev(c)
    rows, qo = append(a, r, kv, gamma, q)
    b = Dev(c)
    wide = torch.randn(c.T, 1024, device=DEV).bfloat16()
    wide[:, 64:640] = kv.to(DEV)
    heads = torch.randn(c.T, c.H, 192, device=DEV).bfloat16()
    heads[..., 128:] = q.to(DEV)
    kept = heads.clone()
    ws = _lib.workspace(256, DEV)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    _lib.dsa_latent_append(b.geom, b.kind, wide[:, 64:640], b.cache, r, gamma=gamma.to(DEV), eps=EPS, q_in=heads[..., 128:], q_out=heads[..., 128:],
                           ws=ws, stream=side)
    side.synchronize()
    assert torch.equal(b.cache, a.cache) and torch.equal(heads[..., 128:], qo) and torch.equal(heads[..., :128], kept[..., :128])
    e = Dev(c)
    _lib.dsa_latent_append(e.geom, e.kind, kv.to(DEV), e.cache, r, gamma=gamma.to(DEV), eps=EPS, ws=ws)
    assert torch.equal(e.cache, a.cache)
    alone = torch.zeros_like(qo)
    _lib.dsa_latent_append(e.geom, e.kind, None, None, r, q_in=kept[..., 128:], q_out=alone, ws=ws)
    assert torch.equal(alone, qo) and torch.equal(e.cache, a.cache) and _lib.dsa_get_error(ws) == 0
    with pytest.raises(_lib.DsaError):
        _lib.dsa_latent_append(e.geom, e.kind, kv[:1].to(DEV).expand(c.T, 576), e.cache, r, ws=ws)


@pytest.mark.parametrize("kind", KINDS)
def test_append_bad_pages_and_requests(kind):
    c = ref.Case([100, 80, 64], [2, 3, 1], 4, kind, seed=5)
    kv, gamma, q = inputs(c)
    d = Dev(c)
    d.block_table[1, 1] = c.P
    rows, qo = append(d, _lib.Rope(), kv, gamma, q)
    assert _lib.dsa_get_error(d.ws) == _lib.DSA_ERR_BAD_INDEX
    verify(d, kv, gamma, q, ref.frequencies(64, 10000.0), True, 1.0, rows, qo, skip={1})
    d = Dev(c)
    d.seq_lens[1] = c.max_len + 64
    append(d, _lib.Rope(), kv, gamma, q)
    assert _lib.dsa_get_error(d.ws) == _lib.DSA_ERR_BAD_INDEX
    keep = c.cache.view(torch.uint8).reshape(c.P, -1)
    now = d.cache.cpu().view(torch.uint8).reshape(c.P, -1)
    for i in range(2):
        assert torch.equal(now[int(c.block_table[1, i])], keep[int(c.block_table[1, i])])


def gathered(c, first, counts):
    """The rows, in fp32 steps: code times scale, rounded to bf16."""
    out = []
    for b, (p0, n) in enumerate(zip(first, counts)):
        for pos in range(p0, p0 + n):
            p, s = c.slot(b, pos)
            if c.kind == "bf16":
                out.append(c.cache[p, s])
                continue
            code, scale, rope = ref.planes(c.cache)
            x = code[p, s].view(ref.CODE[c.kind]).float().view(4, 128) * scale[p, s][:, None]
            out.append(torch.cat([x.view(512).bfloat16(), rope[p, s]]))
    return torch.stack(out) if out else torch.zeros(0, 576, dtype=torch.bfloat16)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,first,counts", [([1], None, [1]), ([100, 64, 3], [3, 0, 1], [97, 64, 0]), ([200, 0, 65, 1], [63, 0, 64, 0], [2, 0, 1, 1]),
                                               ([1000, 77], None, [1000, 77])])
def test_gather(lens, first, counts, kind):
    c = ref.Case(lens, [0] * len(lens), 1, kind, seed=7)
    d = Dev(c)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)
    S = sum(counts)
    wide = torch.full((S + 5, 640), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = _lib.workspace(_lib.dsa_latent_gather_workspace_size(d.geom), DEV)
    f = None if first is None else torch.tensor(first, dtype=torch.int32, device=DEV)
    _lib.dsa_latent_gather(d.geom, d.kind, d.cache, f, cu, wide[:, 32:608], ws)
    assert _lib.dsa_get_error(ws) == 0
    assert torch.equal(wide[:S, 32:608].cpu(), gathered(c, first or [0] * len(lens), counts))
    assert (wide[S:] == 7.0).all() and (wide[:, :32] == 7.0).all() and (wide[:, 608:] == 7.0).all()


@pytest.mark.parametrize("kind", KINDS)
def test_gather_refuses_positions_and_pages(kind):
    c = ref.Case([100, 130], [0, 0], 1, kind, seed=8)
    for first, counts, zero in (([90, 0], [20, 5], range(10, 20)), ([0, -2], [3, 5], (3, 4)), ([0, 120], [1, 20], range(11, 21))):
        d = Dev(c)
        cu = torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int32, device=DEV)
        out = torch.full((sum(counts), 576), 7.0, dtype=torch.bfloat16, device=DEV)
        ws = _lib.workspace(256, DEV)
        _lib.dsa_latent_gather(d.geom, d.kind, d.cache, torch.tensor(first, dtype=torch.int32, device=DEV), cu, out, ws)
        assert _lib.dsa_get_error(ws) == _lib.DSA_ERR_BAD_INDEX
        assert (out[list(zero)] == 0).all() and not (out == 7.0).all(1).any()
    d = Dev(c)
    d.block_table[1, 1] = -1
    out = torch.full((230, 576), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = _lib.workspace(256, DEV)
    _lib.dsa_latent_gather(d.geom, d.kind, d.cache, None, torch.tensor([0, 100, 230], dtype=torch.int32, device=DEV), out, ws)
    assert _lib.dsa_get_error(ws) == _lib.DSA_ERR_BAD_INDEX
    want = gathered(c, [0, 0], [100, 130])
    want[164:228] = 0
    assert torch.equal(out.cpu(), want)


def test_rows_past_32_bits():
    """Cache rows and gathered rows whose byte offsets pass 2^32."""
    c = ref.Case([130, 64], [130, 1], 2, "bf16", seed=9)
    kv, gamma, q = inputs(c)
    a = Dev(c)
    rows, _ = append(a, _lib.Rope(), kv, gamma, q)
    P = 2 ** 32 // (64 * 1152) + c.P + 3
    b = Dev(c)
    b.cache = torch.empty(P, 64, 576, dtype=torch.bfloat16, device=DEV)
    b.cache[P - c.P:] = c.cache.to(DEV)
    b.block_table = torch.where(b.block_table >= 0, b.block_table + (P - c.P), b.block_table)
    b.geom = _lib.Geometry(b.seq_lens, b.cu_q, b.block_table, P, c.max_len, c.T)
    again, _ = append(b, _lib.Rope(), kv, gamma, q)
    assert torch.equal(again, rows) and torch.equal(b.cache[P - c.P:], a.cache)
    out = torch.empty(130, 576, dtype=torch.bfloat16, device=DEV)
    _lib.dsa_latent_gather(b.geom, b.kind, b.cache, None, torch.tensor([0, 130, 130], dtype=torch.int32, device=DEV), out, b.ws)
    assert torch.equal(out, rows[:130]) and _lib.dsa_get_error(b.ws) == 0


@pytest.mark.parametrize("kind", KINDS)
def test_a_prompt_and_its_decode(kind):
    """As a layer without an index runs them: a prompt's second chunk is appended, its context
    gathered, expanded and attended; then a token is appended and attended in the absorbed form."""
    H, scale = 4, 192 ** -0.5
    c = ref.Case([300, 131], [100, 131], H, kind, seed=10, max_len=400)
    for b, n in enumerate(c.lens):                      # room for one token more
        if n % 64 == 0:
            c.block_table[b, n // 64] = c.P - 1 - b
    kv, gamma, q = inputs(c)
    d = Dev(c)
    rope = _lib.Rope(base=10000.0, factor=4.0, original_len=128, attn_factor=1.1)
    g = torch.Generator(device=DEV).manual_seed(1)
    w = (torch.randn(512, H * 256, device=DEV, generator=g) * 512 ** -0.5).bfloat16()
    S = sum(c.lens)
    cu_k = torch.tensor([0, c.lens[0], S], dtype=torch.int32, device=DEV)
    qn = torch.randn(c.T, H, 192, device=DEV, generator=g).bfloat16()
    qr, ws = qn.clone(), _lib.workspace(1 << 26, DEV)
    _lib.dsa_latent_append(d.geom, d.kind, kv.to(DEV), d.cache, rope, gamma=gamma.to(DEV), eps=EPS, q_in=qr[..., 128:], q_out=qr[..., 128:], ws=ws)
    rows = torch.empty(S, 576, dtype=torch.bfloat16, device=DEV)
    _lib.dsa_latent_gather(d.geom, d.kind, d.cache, None, cu_k, rows, ws)
    both = (rows[:, :512] @ w).view(S, H, 256)
    out, lse = torch.empty(c.T, H, 128, dtype=torch.bfloat16, device=DEV), torch.empty(c.T, H, device=DEV)
    _lib.dsa_latent_attend_expanded(d.cu_q, cu_k, qr, both[..., :128], both[..., 128:], rows[:, 512:], scale, out, lse, ws)
    ts = {0, 50, 99, 100, c.T - 1}
    compare(ref.expanded(qr.cpu(), both[..., :128].cpu(), both[..., 128:].cpu(), rows[:, 512:].cpu(), [0, 100, 231], cu_k.tolist(), scale, ts), out, lse)
    # the next token of both requests
    lens = torch.tensor([301, 132], dtype=torch.int32, device=DEV)
    geom = _lib.Geometry(lens, torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV), d.block_table, c.P, c.max_len, 2)
    q1 = torch.randn(2, H, 576, device=DEV, generator=g).bfloat16()
    new = (1.5 * torch.randn(2, 576, device=DEV, generator=g)).bfloat16()
    _lib.dsa_latent_append(geom, d.kind, new, d.cache, rope, gamma=gamma.to(DEV), eps=EPS, q_in=q1[..., 512:], q_out=q1[..., 512:], ws=ws)
    o1, l1 = torch.empty(2, H, 512, dtype=torch.bfloat16, device=DEV), torch.empty(2, H, device=DEV)
    _lib.dsa_latent_attend(geom, d.kind, q1, d.cache, scale, o1, l1, ws)
    assert _lib.dsa_get_error(ws) == 0
    c.lens, c.new, c.cache, c.q = [301, 132], [1, 1], d.cache.cpu(), q1.cpu()
    compare(ref.attend(c, scale), o1, l1)
    assert math.isfinite(l1.sum().item())
