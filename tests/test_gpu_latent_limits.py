"""Ends of the dense latent operators' ranges on the GPU: offsets that do not begin at 0, scales too
small to matter over long contexts, runs of many pages."""
import math

import numpy as np
import pytest
import torch

import latent_reference as ref
from dsa_sparse_attention_02_gb300 import _lib
from test_gpu_latent_attend import DEV, KINDS, Dev, check, compare
from test_gpu_latent_rows import gathered

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("at", [1, 3, 70])
def test_gather_leaves_rows_before_the_first_request(kind, at):
    """Rows cu_k[0] .. cu_k[B]-1 are the requests'; those before are nobody's, as those behind."""
    c = ref.Case([100, 0, 130], [0, 0, 0], 1, kind, seed=21)
    d = Dev(c)
    cu = torch.tensor([at, at + 100, at + 100, at + 230], dtype=torch.int32, device=DEV)
    out = torch.full((at + 237, 576), 7.0, dtype=torch.bfloat16, device=DEV)
    ws = _lib.workspace(_lib.dsa_latent_gather_workspace_size(d.geom), DEV)
    _lib.dsa_latent_gather(d.geom, d.kind, d.cache, None, cu, out, ws)
    assert _lib.dsa_get_error(ws) == 0
    assert (out[:at] == 7.0).all() and (out[at + 230:] == 7.0).all()
    assert torch.equal(out[at:at + 230].cpu(), gathered(c, [0, 0, 0], [100, 0, 130]))


def repeated(lens, new, H, kind, seed, pages):
    """Requests whose block tables repeat a few pages."""
    c = ref.Case([64 * pages], [1], H, kind, seed=seed, spare=0)
    B, n = len(lens), max(lens)
    c.lens, c.new, c.T, c.max_len = list(lens), list(new), sum(new), n
    c.seq_lens = torch.tensor(c.lens, dtype=torch.int32)
    c.cu_q = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32)
    c.block_table = torch.randint(0, c.P, (B, -(-n // 64)), generator=c.gen, dtype=torch.int32)
    c.q = torch.randn(c.T, H, 576, generator=c.gen).bfloat16()
    return c


@pytest.mark.parametrize("kind", ["e4m3", "i8"])
def test_small_scales_over_long_runs(kind):
    """Scales of 2^-100 and scores that rise by e^5 behind the first page: the weights' sum, 40000 keys
    in one run, stays finite."""
    B, n = torch.cuda.get_device_properties(0).multi_processor_count, 40000
    c = repeated([n] * B, [1] * B, 16, kind, 22, 2)
    c.block_table[:, 0], c.block_table[:, 1:] = 0, 1
    _, scale, rope = ref.planes(c.cache)
    scale[...] = 2.0 ** -100
    rope.zero_()
    rope[1, :, 0] = 5.0
    c.q[..., 512] = 1.0
    d = Dev(c)
    out, lse = d.attend(1.0)
    assert _lib.dsa_get_error(d.ws) == 0
    res = ref.attend(c, 1.0, {0, B - 1})
    for r in res.values():
        r[2][...] -= 1e-30                        # (an absolute term, as large as these values)
    compare(res, out, lse)
    want = math.log(64 + (n - 64) * math.exp(5.0))
    assert (lse.double() - want).abs().max() < 1e-4


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("H,new,tile,blocks", [(16, 1, 16, 1), (5, 3, 16, 1), (20, 1, 32, 1), (12, 2, 32, 1), (64, 1, 64, 1), (20, 3, 64, 1),
                                               (128, 1, 64, 2), (24, 4, 64, 2), (128, 2, 64, 1)])
def test_runs_of_thirty_pages_and_more(kind, H, new, tile, blocks):
    """Every row count and form: each run has 30 pages at least, so that rings of places come round
    seven times or more; 30 repeats give the same bits."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    runs = sms // blocks if kind == "bf16" else sms
    rows = tile * blocks if kind == "bf16" else tile
    B, items = 24, -(-H * new // rows)
    n = 64 * (-(-36 * runs // (B * items)))
    lens = [n - 37 * (b % 8) for b in range(B)]
    assert min(lens) > new and sum(items * -(-x // 64) for x in lens) >= 30 * runs
    c = repeated(lens, [new] * B, H, kind, H + new, 40)
    d, out, lse = check(c, ts={0, c.T - 1, c.T // 2})
    assert torch.isfinite(lse).all()
    for _ in range(30):
        again = d.attend()
        assert torch.equal(out, again[0]) and torch.equal(lse, again[1])
    assert _lib.dsa_get_error(d.ws) == 0
