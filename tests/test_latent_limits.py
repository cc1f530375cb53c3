"""Limits of the dense latent operators that need no GPU: what their sources must not hold, and
refusals at the ends of their ranges."""
import glob
import os

import pytest

from dsa_sparse_attention_02_gb300 import _lib, build
from test_gqa_abi import UNS, WSP, geom, lib, ref  # noqa: F401


def test_loads_go_to_the_own_block_alone():
    """Any rank of a run on several GPUs loads the library, and caches lie wherever a caller put them: no load
    or commit in it goes to several blocks' shared memory at once."""
    sources = [f for d in (build.CSRC, build.INCLUDE) for f in glob.glob(os.path.join(d, "**", "*"), recursive=True) if os.path.isfile(f)]
    assert any(f.endswith("ptx.cuh") for f in sources)
    for f in sources:
        with open(f, encoding="utf-8") as h:
            assert "multicast" not in h.read().lower(), f


@pytest.mark.parametrize("H,least", [(1, (1 << 31) - 127), (2, (1 << 30) - 63), (128, (1 << 24))])
def test_attend_refuses_rows_that_do_not_round_up_to_items(lib, H, least):  # noqa: F811
    """T * H up to 2^31 - 128: rounded up to items of 128 rows it still fits 32 bits."""
    def call(T):                                     # (workspace too small: what comes behind the refusal)
        return lib.dsa_latent_attend(ref(geom(T=T)), _lib.DSA_BF16, H, 16, 16, 0.1, 16, None, 256, 256, None)
    assert call(least - 1) == WSP
    for T in (least, least + 1, (1 << 31) - 1):
        assert call(T) == UNS
        assert b"2^31" in lib.dsa_last_error()
