"""CPU checks of the edges of the 4-bit cache and the eviction: what the C entry points and the
build refuse (nothing reaches a GPU)."""

import ctypes

import pytest


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_top_hisa_b200 import build
    build.build()
    from sparse_attention_top_hisa_b200 import binding
    return binding.lib()


P, F = ctypes.c_void_p, ctypes.c_float
ODD = P(4096 + 2)  # never dereferenced


@pytest.mark.parametrize("k", [(1 << 20) + 1, 1 << 28])
def test_attention_rows_too_long_for_their_precision_are_refused(lib, k):
    D = P(4096)
    f = lib.hisa_sparse_attention_kv4
    assert f(D, D, D, D, D, D, 1, 4, 8, k, F(0.1), D, D, D, None) == 1
    # up to the limit the call goes on to the next check
    assert f(D, D, D, D, D, D, 1, 4, 8, 1 << 20, F(0.1), ODD, D, D, None) == 2
