"""Limits of the dense latent operators that need no GPU: what their sources must not hold, and
refusals at the ends of their ranges."""
import glob
import os

import pytest
import torch

from dsa_sparse_attention_02_gb300 import _lib, build
from test_gqa_abi import INV, OK, UNS, WSP, geom, lib, ref  # noqa: F401


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


def test_binding_names_a_tensor_that_is_missing_or_has_other_dimensions(monkeypatch):
    """Also those whose sizes the calls go by: a TypeError with their name, not one about an attribute or index."""
    class Handle:                                    # a geometry without a device
        T, B, num_pages, max_seq_len = 3, 1, 2, 128
        seq_lens = torch.zeros(1, dtype=torch.int32)

    monkeypatch.setattr(_lib, "_latent_call", lambda ws, stream, index: 0)
    g, ws, cu = Handle(), torch.zeros(256, dtype=torch.uint8), torch.zeros(2, dtype=torch.int32)
    x = torch.zeros(3, 2, 576, dtype=torch.bfloat16)
    cache, part = torch.zeros(2, 64, 576, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    for bad in (None, 3, torch.zeros(3, dtype=torch.bfloat16), torch.zeros(3, 2, 1, 64, dtype=torch.bfloat16)):
        with pytest.raises(TypeError, match="^q must"):
            _lib.dsa_latent_attend(g, _lib.DSA_BF16, bad, cache, 0.1, x, None, ws)
        with pytest.raises(TypeError, match="^out must"):
            _lib.dsa_latent_gather(g, _lib.DSA_BF16, cache, None, cu, bad, ws)
        with pytest.raises(TypeError, match="^q must"):
            _lib.dsa_latent_attend_expanded(cu, cu, bad, x, x, x, 0.1, x, None, ws)
        with pytest.raises(TypeError, match="^k must"):
            _lib.dsa_latent_attend_expanded(cu, cu, x, bad, x, x, 0.1, x, None, ws)
        if bad is not None:
            with pytest.raises(TypeError, match="^q_in must"):
                _lib.dsa_latent_append(g, _lib.DSA_BF16, None, None, _lib.Rope(), q_in=bad, q_out=part, ws=ws)
    for bad in (None, 3, torch.zeros(2, 2, dtype=torch.int32), torch.tensor(2, dtype=torch.int32)):
        with pytest.raises(TypeError, match="^cu_q must"):
            _lib.dsa_latent_attend_expanded(bad, cu, x, x, x, x, 0.1, x, None, ws)
    for bad in (None, _lib.dsa_rope_t(), 64):
        with pytest.raises(TypeError, match="^rope must"):
            _lib.dsa_latent_append(g, _lib.DSA_BF16, None, None, bad, q_in=part, q_out=part, ws=ws)


@pytest.mark.parametrize("shape,strides,want", [((1, 2, 64), (130, 64, 1), (128, 64)), ((1, 1, 64), (577, 577, 1), (64, 64)), ((3, 1, 64), (72, 5, 1), (72, 64)),
                                                ((1, 576), (577, 1), (576,)), ((1, 1, 192), (1 << 40, 3, 1), (192, 192)), ((2, 1, 64), (0, 9, 1), (0, 64))])
def test_strides_over_a_single_element_say_nothing(shape, strides, want):
    """A single token, or head, may lie at any stride in its tensor: 577 or 130 is no multiple of 8, but never taken."""
    t = torch.zeros(4096, dtype=torch.bfloat16).as_strided(shape, strides)
    assert _lib._tensor("x", t, torch.bfloat16, shape, -1)[1:] == want


def test_a_geometry_passes_the_sizes_it_has_now():
    """`ref` follows `c`: a program that gives a geometry other sizes or tables by a new `c` is understood."""
    g = _lib.Geometry.__new__(_lib.Geometry)
    g.c = geom()
    assert g.ref._obj is g.c
    g.c = geom(T=7)
    assert g.ref._obj is g.c and g.ref._obj.T == 7


def test_an_empty_batch_is_no_error(lib):  # noqa: F811
    """Tensors without elements have no address, the cache has one."""
    rope = _lib.Rope().c

    def append(T, kv=None, cache=16, ko=None, H=4, q=None, qo=None):
        return lib.dsa_latent_append(ref(geom(T=T)), _lib.DSA_BF16, kv, 576, 16, 1e-6, ref(rope), cache, ko, H, q, 256, 64, qo, 256, 64, 256, 256, None)
    assert append(0) == OK and append(0, q=16) == OK and append(0, H=0) == OK
    assert append(1) == INV and append(1, kv=16, q=16) == INV
    assert lib.dsa_latent_attend(ref(geom(T=0)), _lib.DSA_BF16, 16, None, 16, 0.1, None, None, 256, 256, None) == OK
    assert lib.dsa_latent_gather(ref(geom()), _lib.DSA_BF16, 16, None, 16, 0, None, 576, 256, 256, None) == OK
    assert lib.dsa_latent_attend_expanded(1, 0, 0, 16, 16, 4, None, 768, 192, None, 512, 128, None, 512, 128, None, 64, 0.1, None, None, 256, 256,
                                          None) == OK
