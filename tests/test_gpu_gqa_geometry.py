"""Inconsistent requests among good ones, and bad pages, are reported by every grouped-query
operator, wherever they stand in the batch."""
import numpy as np
import pytest
import torch

import gqa_reference as ref
from dsa_sparse_attention_02_gb300 import _lib
from test_gpu_gqa import DEV, E4, Dev

pytestmark = pytest.mark.gpu
BAD = _lib.DSA_ERR_BAD_INDEX


def call_all(d, T):
    """The error word of each operator, called on d's geometry."""
    c = d.c
    x = torch.zeros(T, c.H + 2 * c.Hkv, c.D, dtype=torch.bfloat16, device=DEV)
    ws = _lib.workspace(max(_lib.dsa_gqa_attend_workspace_size(d.geom, d.cache, c.H),
                            _lib.dsa_gqa_attend_blocks_workspace_size(d.geom, d.cache, c.H, 3)), DEV)
    out, lse = torch.zeros(T, c.H, c.D, dtype=torch.bfloat16, device=DEV), torch.zeros(T, c.H, device=DEV)
    blocks = torch.full((T, c.Hkv, 3), -1, dtype=torch.int32, device=DEV)
    got = {}
    _lib.dsa_gqa_append(d.geom, d.cache, x[:, c.H:c.H + c.Hkv], x[:, c.H + c.Hkv:], x[:, :c.H], out, ws=ws)
    got["append"] = _lib.dsa_get_error(ws)
    _lib.dsa_gqa_append(d.geom, d.cache, x[:, c.H:c.H + c.Hkv], x[:, c.H + c.Hkv:], ws=ws)
    got["append without queries"] = _lib.dsa_get_error(ws)
    _lib.dsa_gqa_attend(d.geom, d.cache, d.q, 0.1, out, lse, ws)
    got["attend"] = _lib.dsa_get_error(ws)
    _lib.dsa_block_select(d.geom, d.cache, d.q, 3, 0, 1, blocks, ws)
    got["select"] = _lib.dsa_get_error(ws)
    blocks.fill_(-1)
    _lib.dsa_gqa_attend_blocks(d.geom, d.cache, d.q, blocks, 0.1, out, lse, ws)
    got["attend_blocks"] = _lib.dsa_get_error(ws)
    return got


@pytest.mark.parametrize("op", ["append", "append without queries", "attend", "select", "attend_blocks"])
@pytest.mark.parametrize("cu", [
    [0, 5, 3, 8], [0, 3, 2, 2, 8], [0, 8, 1, 8, 8], [0, 1, 0, 1, 2, 3, 4, 5, 6, 7, 8], [0, 2, 7, 6], [0, -1, 4, 8],
    list(range(0, 8)) + [6] + [8] * 70, [0] * 2000 + [8, 2] + [8] * 300, [0, 1000, 10, 40], [0, 64, 700, 20, 30, 800, 1000]])
def test_decreasing_offsets_are_reported(cu, op):
    B, T = len(cu) - 1, max(cu)
    c = ref.Case([1000 if B < 9 else 70] * B, [0] * B, 4, 2, 64, E4, seed=3, pad=T)
    d = Dev(c)
    assert set(call_all(d, T).values()) == {0}           # (no request has tokens)
    d.cu_q.copy_(torch.tensor(cu))
    assert call_all(d, T)[op] == BAD


@pytest.mark.parametrize("new", [1, 700])
@pytest.mark.parametrize("n_sel", [3, 40])
def test_selection_reports_bad_pages_it_lists(n_sel, new):
    """Also where every visible block is taken and nothing has to be scored."""
    c = ref.Case([new + 63, 1100], [new, new], 8, 4, 64, E4, seed=2)
    for block in (0, (new + 62) // 64):
        bt = c.block_table.clone()
        c.block_table[0, block] = c.P
        d = Dev(c)
        got = d.select(n_sel, 1, 2)
        assert _lib.dsa_get_error(d.ws) == BAD
        c.tokens = lambda: [x for x in ref.Case.tokens(c) if x[0] % 97 == 0]
        ts = [t for t, _, _ in c.tokens()]
        assert np.array_equal(got[ts].cpu().numpy(), ref.select(c, n_sel, 1, 2)[ts])
        c.block_table = bt
    d = Dev(c)
    d.select(n_sel, 1, 2)
    assert _lib.dsa_get_error(d.ws) == 0                             # entries behind the last block are no pages: not read
