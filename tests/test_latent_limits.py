"""Limits of the dense latent operators that need no GPU: what their sources must not hold, and
refusals at the ends of their ranges."""
import glob
import os

from dsa_sparse_attention_02_gb300 import build


def test_loads_go_to_the_own_block_alone():
    """Any rank of a run on several GPUs loads the library, and caches lie wherever a caller put them: no load
    or commit in it goes to several blocks' shared memory at once."""
    sources = [f for d in (build.CSRC, build.INCLUDE) for f in glob.glob(os.path.join(d, "**", "*"), recursive=True) if os.path.isfile(f)]
    assert any(f.endswith("ptx.cuh") for f in sources)
    for f in sources:
        with open(f, encoding="utf-8") as h:
            assert "multicast" not in h.read().lower(), f
