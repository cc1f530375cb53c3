"""Dense absorbed attention over the paged latent cache against its definition in 64 bits:
every cache type, one head to 128, one new token to hundreds, contexts of no token, one and
many; keys that a row does not see, values that are not finite, bad pages and requests."""
import math

import numpy as np
import pytest
import torch

import latent_reference as ref
from dsa_sparse_attention_02_gb300 import _lib

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
KIND = {"bf16": _lib.DSA_BF16, "e4m3": _lib.DSA_E4M3, "i8": _lib.DSA_I8}
KINDS = list(KIND)
SM = 192 ** -0.5


class Dev:
    """A Case on the GPU."""

    def __init__(self, c):
        self.c, self.kind = c, KIND[c.kind]
        self.cache, self.seq_lens, self.cu_q, self.block_table, self.q = (
            x.to(DEV) for x in (c.cache, c.seq_lens, c.cu_q, c.block_table, c.q))
        self.geom = _lib.Geometry(self.seq_lens, self.cu_q, self.block_table, c.P, c.max_len, c.T)

    def attend(self, sm=SM, ws=None, lse=True, stream=None):
        c = self.c
        out = torch.full((c.T, c.H, 512), 7.0, dtype=torch.bfloat16, device=DEV)
        le = torch.full((c.T, c.H), 7.0, device=DEV) if lse else None
        self.ws = ws if ws is not None else _lib.workspace(_lib.dsa_latent_attend_workspace_size(self.geom, c.H), DEV)
        _lib.dsa_latent_attend(self.geom, self.kind, self.q, self.cache, sm, out, le, self.ws, stream)
        return out, le


def compare(res, out, lse):
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    with np.errstate(invalid="ignore"):
        for t, (ro, rl, bo, bl) in res.items():
            assert np.array_equal(np.isnan(o[t]), np.isnan(ro)) and np.array_equal(np.isneginf(l[t]), np.isneginf(rl)), t
            fine = np.isfinite(ro)
            assert (np.abs(o[t] - ro) <= bo)[fine].all(), (t, np.nanmax((np.abs(o[t] - ro) / bo)[fine]))
            fine = np.isfinite(rl)
            assert (np.abs(l[t] - rl) <= bl)[fine].all(), (t, np.nanmax((np.abs(l[t] - rl) / bl)[fine]))


def check(c, sm=SM, error=0, ts=None):
    d = Dev(c)
    out, lse = d.attend(sm)
    assert _lib.dsa_get_error(d.ws) == error
    n = sum(c.new)
    assert (out[n:] == 7.0).all() and (lse[n:] == 7.0).all()
    compare(ref.attend(c, sm, ts), out, lse)
    again = d.attend(sm)
    assert torch.equal(out.view(torch.int16), again[0].view(torch.int16)) and torch.equal(lse.view(torch.int32), again[1].view(torch.int32))
    return d, out, lse


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,new,H,pad", [
    ([1], [1], 1, 0), ([64], [1], 16, 2), ([65], [1], 16, 0), ([63, 1, 200], [1, 1, 1], 5, 3), ([0, 3, 128], [1, 2, 1], 3, 0),
    ([130], [130], 2, 0), ([70, 2], [70, 5], 20, 4), ([257, 500, 64], [4, 1, 3], 16, 0), ([300, 90], [2, 1], 64, 0),
    ([500, 129, 64, 65], [1, 1, 1, 1], 128, 1), ([333, 1000], [7, 30], 40, 0), ([190], [3], 128, 0), ([0, 0], [2, 1], 12, 1)])
def test_attend(lens, new, H, pad, kind):
    check(ref.Case(lens, new, H, kind, seed=sum(lens) + H, pad=pad))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("lens,new,H", [([20000], [1], 16), ([9000, 11000], [1, 2], 64), ([30001], [1], 128), ([3000], [150], 24), ([2500], [65], 128)])
def test_attend_long(lens, new, H, kind):
    """Items cut into many runs; hundreds of new tokens. Tokens are sampled."""
    c = ref.Case(lens, new, H, kind, seed=H)
    n = sum(new)
    check(c, ts={0, n - 1, n // 2, n // 3})


@pytest.mark.parametrize("kind", KINDS)
def test_attend_many_requests(kind):
    lens = [(37 * b) % 400 for b in range(700)]
    new = [b % 3 for b in range(700)]
    c = ref.Case(lens, new, 16, kind, seed=2)
    check(c, ts=set(range(0, c.T, 23)) | {c.T - 1})


@pytest.mark.parametrize("kind", KINDS)
def test_scale_zero_and_large_scores(kind):
    c = ref.Case([200, 77], [3, 1], 16, kind, seed=5)
    check(c, 0.0)
    c.q *= 12                                   # scores in the hundreds: the reference maximum moves within a request
    check(c, 1.0)
    # rising and falling scores along the context
    c = ref.Case([640, 640], [1, 1], 16, kind, seed=6)
    c.q.zero_()
    c.q[..., 512] = 1.0
    for b, sign in ((0, 1), (1, -1)):
        for pos in range(640):
            p, s = c.slot(b, pos)
            if kind == "bf16":
                c.cache[p, s, 512] = sign * pos / 2
            else:
                ref.planes(c.cache)[2][p, s, 0] = sign * pos / 2
    check(c, 1.0)


def spoil(c, page, slot, what):
    """A value of this kind in the row: in its latent part, rotated part or scale."""
    bad = math.nan if what.startswith("nan") else math.inf
    if c.kind == "bf16":
        c.cache[page, slot, 520 if what.endswith("rope") else 3] = bad
        return
    code, scale, rope = ref.planes(c.cache)
    if what.endswith("rope"):
        rope[page, slot, 8] = bad
    elif what.endswith("scale"):
        scale[page, slot, 2] = bad
    else:
        code[page, slot, 77] = 0x7F               # (the e4m3 NaN; int8 has none)


@pytest.mark.parametrize("kind,what", [("bf16", "nan"), ("bf16", "inf"), ("bf16", "nan rope"), ("bf16", "inf rope"), ("e4m3", "nan"), ("e4m3", "nan rope"),
                                       ("e4m3", "nan scale"), ("e4m3", "inf scale"), ("i8", "nan scale"), ("i8", "inf rope"), ("i8", "inf scale")])
@pytest.mark.parametrize("H", [2, 16, 64])
def test_values_that_are_not_finite(kind, what, H):
    """Behind a request's last token, in pages of no request and in other requests they change
    nothing; a row that sees one is NaN (or infinite in its column)."""
    c = ref.Case([100, 130, 64], [3, 66, 1], H, kind, seed=9)
    clean = Dev(c).attend()
    used = {int(c.block_table[b, i]) for b, n in enumerate(c.lens) for i in range(-(-n // 64))}
    for page in set(range(c.P)) - used:
        for s in (0, 5, 63):
            spoil(c, page, s, what)
    for b, n in enumerate(c.lens):
        for s in range(n % 64, 64 if n % 64 else 0):
            spoil(c, int(c.block_table[b, n // 64]), s, what)
    d = Dev(c)
    got = d.attend()
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1], clean[1])
    spoil(c, *c.slot(1, 100), what)               # seen from position 100 on: token 3 + 36 of request 1
    d = Dev(c)
    got = d.attend()
    assert _lib.dsa_get_error(d.ws) == 0
    sees = torch.zeros(c.T, dtype=torch.bool)
    sees[3 + 36:3 + 66] = True
    assert torch.equal(got[0][~sees], clean[0][~sees]) and torch.equal(got[1][~sees], clean[1][~sees])
    if what != "inf rope":                        # (an infinite rotated part may also make a weight of 0)
        assert (~torch.isfinite(got[0][sees].float())).any(-1).all()
    if "nan" in what:
        assert torch.isnan(got[0][sees].float()).all()


@pytest.mark.parametrize("kind", KINDS)
def test_bad_pages_and_requests(kind):
    c = ref.Case([300, 200, 64, 90], [2, 1, 1, 2], 16, kind, seed=11)
    c.block_table[0, 1] = -1
    c.block_table[1, 2] = c.P
    c.block_table[3, 0] = 2 ** 30
    check(c, error=_lib.DSA_ERR_BAD_INDEX)
    # a length past the host's: its rows see no key, the others are as they were
    c = ref.Case([300, 200, 64], [2, 1, 1], 16, kind, seed=12)
    d = Dev(c)
    d.seq_lens[1] = c.max_len + 1
    out, lse = d.attend()
    assert _lib.dsa_get_error(d.ws) == _lib.DSA_ERR_BAD_INDEX
    assert (out[2] == 0).all() and torch.isneginf(lse[2]).all()
    r = ref.attend(c, SM)
    compare({t: r[t] for t in (0, 1, 3)}, out, lse)
    # offsets that decrease
    d = Dev(c)
    d.cu_q[1] = 4
    d.attend()
    assert _lib.dsa_get_error(d.ws) == _lib.DSA_ERR_BAD_INDEX


@pytest.mark.parametrize("kind", KINDS)
def test_without_lse_on_another_stream_and_captured(kind):
    c = ref.Case([700, 130, 1], [1, 2, 1], 16, kind, seed=13)
    d = Dev(c)
    want = d.attend()
    assert torch.equal(d.attend(lse=False)[0], want[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = [_lib.workspace(_lib.dsa_latent_attend_workspace_size(d.geom, c.H), DEV) for _ in range(2)]
    a, b = d.attend(ws=ws[0], stream=side), d.attend(ws=ws[1])       # two at a time
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a + b, want + want))
    # captured once, replayed for other lengths and queries; two graphs share a workspace
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o, l = torch.empty_like(want[0]), torch.empty_like(want[1])
            _lib.dsa_latent_attend(d.geom, d.kind, d.q, d.cache, SM, o, l, ws[0])
        graphs.append(g)
        outs.append((o, l))
    for lens in ([700, 130, 1], [5, 64, 0], [699, 2, 1]):
        d.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        d.q.copy_(torch.randn(c.q.shape, generator=c.gen).bfloat16())
        want = d.attend(ws=ws[1])
        for g, got in zip(graphs, outs):
            g.replay()
        torch.cuda.synchronize()
        for got in outs:
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("kind", ["bf16", "i8"])
def test_pages_past_32_bits(kind):
    """Pages whose byte offsets pass 2^32, and whose rows' element offsets pass 2^31."""
    c = ref.Case([130, 64], [1, 2], 16, kind, seed=15)
    page_bytes = 64 * 1152 if kind == "bf16" else ref.PAGE_BYTES
    P = 2 ** 32 // page_bytes + c.P + 9
    want = Dev(c).attend()
    big = torch.empty((P,) + c.cache.shape[1:], dtype=c.cache.dtype, device=DEV)
    big[P - c.P:] = c.cache.to(DEV)
    d = Dev(c)
    d.cache = big
    d.block_table = torch.where(d.block_table >= 0, d.block_table + (P - c.P), d.block_table)
    d.geom = _lib.Geometry(d.seq_lens, d.cu_q, d.block_table, P, c.max_len, c.T)
    got = d.attend()
    assert _lib.dsa_get_error(d.ws) == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_workspace_of_a_larger_step_serves():
    c = ref.Case([300, 200], [1, 1], 16, seed=16)
    d = Dev(c)
    want = d.attend()
    more = _lib.Geometry(d.seq_lens, d.cu_q, d.block_table, c.P, c.max_len, 4000)
    ws = _lib.workspace(_lib.dsa_latent_attend_workspace_size(more, c.H), DEV).fill_(0xA5)
    ws[:256] = 0
    got = d.attend(ws=ws)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_refusals_of_the_binding():
    d = Dev(ref.Case([100], [1], 16, seed=17))
    o, ws = torch.empty(1, 16, 512, dtype=torch.bfloat16, device=DEV), _lib.workspace(1 << 24, DEV)
    call = lambda q=d.q, cache=d.cache, out=o, lse=None, ws=ws: _lib.dsa_latent_attend(d.geom, d.kind, q, cache, SM, out, lse, ws)  # noqa: E731
    for bad in (dict(q=d.q[..., :512]), dict(q=d.q.float()), dict(q=d.q.cpu()), dict(cache=d.cache.cpu()), dict(cache=d.cache[:, :, :512]),
                dict(out=o[:, :8]), dict(out=None), dict(lse=torch.empty(16, device=DEV))):
        with pytest.raises(TypeError):
            call(**bad)
    with pytest.raises(_lib.DsaError):
        call(ws=_lib.workspace(256, DEV))
    call()


@pytest.mark.parametrize("lens,new,H", [([700, 64, 129], [1, 1, 1], 100), ([300, 1, 0], [8, 1, 3], 16), ([90, 5000], [5, 3], 24), ([200, 77], [1, 1], 65),
                                        ([130, 130, 130], [3, 1, 0], 64)])
def test_pairs_of_items(lens, new, H):
    """65 to 128 rows a request in the mean: two items of 64 rows share their pages' loads; requests with
    fewer rows, with more, and without any; NaN behind the last token and in a page seen in part."""
    c = ref.Case(lens, new, H, "bf16", seed=31 + H)
    for b, n in enumerate(lens):
        for s in range(n % 64, 64 if n % 64 else 0):
            spoil(c, int(c.block_table[b, n // 64]), s, "nan")
    check(c)
    c.block_table[0, 0] = -3
    check(c, error=_lib.DSA_ERR_BAD_INDEX)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B,n,new,H", [(22, 5500, 2, 12), (7, 9000, 1, 32), (60, 1300, 1, 20), (8, 4000, 1, 16), (10, 4000, 3, 16), (3, 9000, 1, 128)])
def test_long_runs_of_each_row_count(B, n, new, H, kind):
    """Runs of tens of pages with 16, 17 to 32 and up to 64 rows an item, many times over: rings come
    round many times, and nothing depends on which load is first."""
    lens = [n - 37 * b for b in range(B)]
    c = ref.Case([64 * 40], [1], H, kind, seed=B, spare=0)          # a small cache whose pages repeat
    c.lens, c.new, c.T, c.max_len = lens, [new] * B, new * B, n
    c.seq_lens = torch.tensor(lens, dtype=torch.int32)
    c.cu_q = torch.arange(B + 1, dtype=torch.int32) * new
    c.block_table = torch.randint(0, c.P, (B, -(-n // 64)), generator=c.gen, dtype=torch.int32)
    c.q = torch.randn(c.T, H, 576, generator=c.gen).bfloat16()
    d, out, lse = check(c, ts={0, c.T - 1, c.T // 2})
    for _ in range(30):
        again = d.attend()
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    assert _lib.dsa_get_error(d.ws) == 0
