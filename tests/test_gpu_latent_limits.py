"""Ends of the dense latent operators' ranges on the GPU: offsets that do not begin at 0."""
import pytest
import torch

import latent_reference as ref
from dsa_sparse_attention_02_gb300 import _lib
from test_gpu_latent_attend import DEV, KINDS, Dev
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
