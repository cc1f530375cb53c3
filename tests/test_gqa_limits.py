"""Sizes past what a launch can count are refused (C functions with dummy addresses, nothing
reaches a GPU), and so are calls of the binding that leave out or misfit a tensor."""
import pytest
import torch

from dsa_sparse_attention_02_gb300 import _lib
from test_gqa_abi import OK, UNS, cache, geom, lib, ref  # noqa: F401


@pytest.mark.parametrize("B,T,Hkv", [(1 << 24, 1, 128), (1 << 30, 1, 1), (1 << 30, 1, 2), ((1 << 31) - 1, 1, 1), (1 << 23, (1 << 31) - 1, 128)])
def test_append_refuses_more_blocks_than_a_launch_has(lib, B, T, Hkv):  # noqa: F811
    def call(**kw):
        c = cache(Hkv=Hkv)
        return lib.dsa_gqa_append(ref(geom(**kw)), ref(c), 16, 128 * Hkv, 16, 128 * Hkv, 0, None, 0, None, 0, None, None, 256, 1 << 20, None)
    assert call(B=B, T=T) == UNS
    assert b"2^31" in lib.dsa_last_error()
    assert call(B=B // (2 * Hkv) // 4, T=0) == OK


def test_binding_refuses_what_is_missing_or_does_not_fit():
    class Handle:                                     # a cache and a geometry without a device
        D, Hkv, T, num_pages, device, index = 64, 2, 5, 3, torch.device("cpu"), -1

    h = Handle()
    rows = torch.zeros(5, 2, 64, dtype=torch.bfloat16)
    for ws in (None, torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros(1 << 12, dtype=torch.uint8)[::2]):
        with pytest.raises(TypeError, match="ws"):    # (an expanded tensor has more elements than bytes)
            _lib.dsa_gqa_append(h, h, rows, rows, ws=ws)
        with pytest.raises(TypeError, match="ws"):
            _lib.dsa_gqa_attend(h, h, rows, 0.1, rows, None, ws)
    ws = torch.zeros(256, dtype=torch.uint8)
    for q_in, q_out in ((rows, None), (None, rows)):  # (queries that would be left out in silence)
        with pytest.raises(TypeError, match="go together"):
            _lib.dsa_gqa_append(h, h, rows, rows, q_in, q_out, ws=ws)
    with pytest.raises(TypeError, match="q is missing"):
        _lib._heads("q", None, h, h)
    with pytest.raises(TypeError, match="rope_cos is missing"):
        _lib._plain("rope_cos", None, torch.float32, (8, 4), h)


@pytest.mark.parametrize("n", [(1 << 31) - 1, (1 << 31) - 64, (1 << 31) - 65536])
def test_lengths_that_do_not_round_up_in_32_bits_are_refused(lib, n):  # noqa: F811
    """(2^31 - 64 tokens and more came out as a negative number of pages, which any table holds.)"""
    g, c = geom(max_seq_len=n, T=0), cache()
    assert lib.dsa_gqa_attend(ref(g), ref(c), 8, None, 0, 0.1, None, None, 256, 1 << 20, None) == UNS
    assert lib.dsa_gqa_append(ref(g), ref(c), None, 0, None, 0, 0, None, 0, None, 0, None, None, 256, 1 << 20, None) == UNS
    assert lib.dsa_topk_workspace_size(ref(g), 2048) == 256
    g = geom(max_seq_len=(1 << 31) - 65537, T=0, bt_stride=1 << 25)
    assert lib.dsa_gqa_attend(ref(g), ref(c), 8, None, 0, 0.1, None, None, 256, 1 << 20, None) == OK
