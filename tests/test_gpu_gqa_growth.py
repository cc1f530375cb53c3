"""A block filled token by token: each growth of its scale rounds the older codes once more,
and no value is further off than those roundings together allow."""
import numpy as np
import pytest
import torch

import gqa_reference as ref
from dsa_sparse_attention_02_gb300 import _lib
from test_gpu_gqa import DEV, E4, I8, Dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [E4, I8], ids=["e4m3", "i8"])
@pytest.mark.parametrize("rise", [1.0, 2.0, 30.0])
def test_growing_scales_round_once_each(rise, dtype):
    """Bounds carried along: writing a token, and each growth of its block's scale s, adds half a
    step (e4m3: 2^-4 of the value, or 2^-10 of s below its normal range; int8: s / 2) and three
    fp32 operations' 2^-24 of the value. (A value at the block's largest may be cut at the largest
    code where the scale was rounded down: 2^-24 of it, in the last term.)"""
    c = ref.Case([64], [1], 2, 2, 64, dtype, seed=11)
    c.block_table[0, 0] = 1
    d = Dev(c)
    ws = _lib.workspace(256, DEV)
    x = (torch.randn(64, 4, 64, generator=c.gen) * rise ** (torch.arange(64) / 63.0)[:, None, None]).bfloat16()
    cu, seq = torch.tensor([0, 1], dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    geom = _lib.Geometry(seq, cu, d.block_table, c.P, 64, 1)
    want = x.double().numpy()
    bound, scale, growths = np.zeros((64, 4, 64)), np.zeros(4), np.zeros(4)
    for i in range(64):
        seq.fill_(i + 1)
        part = x[i:i + 1].to(DEV)
        _lib.dsa_gqa_append(geom, d.cache, part[:, :2], part[:, 2:], ws=ws)
        now = torch.cat([d.k_scale[1], d.v_scale[1]]).double().cpu().numpy()
        grew = now > scale
        assert (now >= scale).all()
        growths += grew & (i > 0)
        for h in range(4):
            lo = 0 if grew[h] else i                      # which codes are rounded now
            size = np.abs(want[lo:i + 1, h]) + bound[lo:i + 1, h]
            half = now[h] / 2 if dtype == I8 else np.maximum(size * 2.0 ** -4, now[h] * 2.0 ** -10)
            bound[lo:i + 1, h] += half + 4 * 2.0 ** -24 * size
        scale = now
    assert _lib.dsa_get_error(ws) == 0
    assert (growths >= 2).all()
    got = torch.cat([d.k[1].double() * d.k_scale[1].double()[:, None, None], d.v[1].double() * d.v_scale[1].double()[:, None, None]])
    off = np.abs(got.transpose(0, 1).cpu().numpy() - want)
    assert (off <= bound).all(), float((off / bound).max())
