"""Sizes past what a launch can count are refused (C functions with dummy addresses, nothing
reaches a GPU), and so are calls of the binding that leave out or misfit a tensor."""
import pytest

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
