"""CPU checks of the 4-bit cache and the eviction: the reference's quantiser on values
worked out by hand, and the refusals of the C entry points (nothing reaches a GPU)."""

import ctypes

import numpy as np
import pytest

import kv4_ref


@pytest.fixture(scope="module")
def lib():
    from sparse_attention_top_hisa_b200 import build
    build.build()
    from sparse_attention_top_hisa_b200 import binding
    return binding.lib()


def _row(*first):
    x = np.zeros((1, 128))
    x[0, :len(first)] = first
    return x


def test_reference_quantiser_by_hand():
    # amax 7: scale 1 (fp16 0x3C00 >> 7 = 0x78); halves round to even
    u, s = kv4_ref.quantise(_row(7, 0.5, 1.5, 2.5, -0.5, -1.5, -6.5, 6.5))
    assert s[0, 0] == 0x78 and not s[0, 1:].any()
    assert (u[0, :8].astype(int) - 8).tolist() == [7, 0, 2, 2, 0, -2, -6, 6]
    assert (u[0, 8:] == 8).all()
    # amax 7 * 1.0625: a tie between scales 1 and 1.125, the even one is 1; 7.4375 -> 7
    u, s = kv4_ref.quantise(_row(7 * 1.0625))
    assert s[0, 0] == 0x78 and u[0, 0] == 15
    # 7 * 1.1875: between 1.125 (odd) and 1.25 (even)
    u, s = kv4_ref.quantise(_row(7 * 1.1875, -1.25))
    assert s[0, 0] == 0x7A and u[0, 1] == 7
    # saturation, the smallest scales, zero
    u, s = kv4_ref.quantise(_row(1e30, -6720.0))
    assert kv4_ref.scale_grid()[s[0, 0]] == 896 and u[0, 0] == 15 and u[0, 1] == 1
    assert kv4_ref.quantise(_row(7 * 2.0 ** -18))[1][0, 0] == 0
    assert kv4_ref.quantise(_row(7 * 2.0 ** -17))[1][0, 0] == 1
    # an infinity marks its group
    u, s = kv4_ref.quantise(_row(np.inf, 1.0))
    assert s[0, 0] == 255 and (u[0] == 8).all()
    codes, scales = kv4_ref.pack(u, s, *kv4_ref.quantise(_row(7, -7)))
    k, v = kv4_ref.values(codes, scales)
    assert np.isnan(k[0, :16]).all() and not k[0, 16:].any()
    assert v[0, :3].tolist() == [7, -7, 0] and codes[0, 64] == 0x1F


def test_reference_attention_by_hand():
    q = np.zeros((1, 1, 128))
    q[0, 0, 0] = 1.0
    k = np.zeros((3, 128))
    k[1, 0] = np.log(3.0)
    v = np.zeros((3, 128))
    v[0, 5], v[1, 5] = 4.0, 8.0
    a = kv4_ref.Attention(q, k, v, np.array([[1, -1, 0]]), [0, 1], [0, 3], 1.0)
    assert a.out[0, 0, 5] == pytest.approx(7.0) and a.lse[0, 0] == pytest.approx(np.log(4))
    assert a.weight[0].tolist() == pytest.approx([0.75, 0.0, 0.25])


def test_reference_eviction_by_hand():
    w = [5, 0, 9, 9, 1, 9, 0, 3]
    assert kv4_ref.evict_select(w, 8, 4, 1, 1).tolist() == [0, 2, 3, 7]
    assert kv4_ref.evict_select(w, 8, 1, 2, 3).tolist() == [0]
    assert kv4_ref.evict_select(w, 8, 0, 2, 3).tolist() == []
    assert kv4_ref.evict_select(w, 8, 9, 0, 0).tolist() == list(range(8))


P, F = ctypes.c_void_p, ctypes.c_float
D, ODD = P(4096), P(4096 + 2)  # never dereferenced


def test_kv4_refusals(lib):
    for f in (lib.hisa_kv4_store, lib.hisa_kv4_load):
        ok = [D, D, D, D, None, 1, 4, D, D, None]
        for at, bad, want in ((5, -1, 1), (6, -1, 1), (5, 0, 1), (0, None, 1), (1, None, 1),
                              (2, None, 1), (3, None, 1), (7, None, 1), (8, None, 1),
                              (0, ODD, 2), (1, ODD, 2), (2, ODD, 2), (3, ODD, 2), (4, ODD, 2),
                              (7, ODD, 2), (8, ODD, 2)):
            a = list(ok)
            a[at] = bad
            assert f(*a) == want, (at, bad)
        assert f(None, None, None, None, None, 0, 0, None, None, None) == 0


def test_attention_kv4_refusals(lib):
    f = lib.hisa_sparse_attention_kv4
    ok = [D, D, D, D, D, D, 1, 4, 8, 16, F(0.1), D, D, D, None]
    for at, bad, want in ((6, -1, 1), (6, 0, 1), (7, -1, 1), (7, 1 << 25, 1), (8, 0, 1), (8, 33, 1),
                          (9, 0, 1), (10, F(float("nan")), 1), (0, None, 1), (1, None, 1),
                          (2, None, 1), (3, None, 1), (4, None, 1), (5, None, 1), (11, None, 1),
                          (12, None, 1),  # weights without lse
                          (0, ODD, 2), (1, ODD, 2), (2, ODD, 2), (3, ODD, 2), (11, P(4096 + 8), 2),
                          (12, ODD, 2), (13, P(4096 + 4), 2)):
        a = list(ok)
        a[at] = bad
        assert f(*a) == want, (at, bad)
    assert f(*([None] * 6), 0, 0, 8, 16, F(0.1), None, None, None, None) == 0


def test_token_weights_refusals(lib):
    f = lib.hisa_token_weights
    ok = [D, D, D, D, D, D, 1, 4, 8, 16, F(0.1), D, None]
    for at, bad, want in ((6, -1, 1), (6, 0, 1), (7, -1, 1), (8, 0, 1), (8, 33, 1), (9, 0, 1),
                          (10, F(float("nan")), 1), (3, None, 1), (11, None, 1), (0, ODD, 2),
                          (1, ODD, 2), (3, ODD, 2), (11, P(4096 + 4), 2)):
        a = list(ok)
        a[at] = bad
        assert f(*a) == want, (at, bad)
    assert f(*([None] * 6), 0, 0, 8, 16, F(0.1), None, None) == 0


def test_evict_refusals(lib):
    f = lib.hisa_evict_select
    ok = [D, D, None, D, 1, 128, 4, 4, D, D, None]
    for at, bad, want in ((4, -1, 1), (5, -1, 1), (6, -1, 1), (7, -1, 1), (0, None, 1),
                          (1, None, 1), (3, None, 1), (8, None, 1), (9, None, 1),
                          (0, P(4096 + 4), 2), (3, ODD, 2), (8, ODD, 2)):
        a = list(ok)
        a[at] = bad
        assert f(*a) == want, (at, bad)
    assert f(None, None, None, None, 0, 0, 0, 0, None, None, None) == 0

    from sparse_attention_top_hisa_b200.binding import _Rows
    f = lib.hisa_evict_rows

    def call(rows, n=None, s=1, most=8, cu=D):
        arr = (_Rows * max(1, len(rows)))(*[_Rows(*r) for r in rows])
        return f(arr, len(rows) if n is None else n, cu, D, D, D, s, most, None)
    good = (4096, 8192, 64)
    assert call([good], n=-1) == 1
    assert call([(4096 + 4096 * i, 65536 + 4096 * i, 64) for i in range(9)]) == 1
    assert call([good], s=-1) == 1 and call([good], s=65536) == 1 and call([good], most=-1) == 1
    assert call([(None, 8192, 64)]) == 1 and call([(4096, None, 64)]) == 1
    assert call([(4096, 8192, 0)]) == 1 and call([(4096, 8192, 6)]) == 1
    assert call([(4096, 8192, 4100)]) == 1
    assert call([(4098, 8192, 64)]) == 2 and call([(4096, 8194, 64)]) == 2
    assert call([good, (16384, 8192, 64)]) == 1  # the same destination twice
    assert call([good], cu=None) == 1 and call([good], cu=ODD) == 2
    assert call([]) == 0 and call([good], s=0) == 0 and call([good], most=0) == 0


def test_binding_refuses_host_tensors():
    import torch

    import sparse_attention_top_hisa_b200 as H
    cu = torch.tensor([0, 128], dtype=torch.int32)
    kv, sc = torch.zeros(128, 128, dtype=torch.uint8), torch.zeros(128, 16, dtype=torch.uint8)
    x = torch.zeros(128, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        H.hisa_kv4_store(x, x, cu, cu, None, kv, sc)
    with pytest.raises(ValueError, match="CUDA tensor"):
        H.hisa_sparse_attention_kv4(x.view(128, 1, 128), kv, sc, cu.view(1, 2), cu, cu, 1.0)
    with pytest.raises(ValueError, match="CUDA tensor"):
        H.hisa_evict_select(torch.zeros(128, dtype=torch.int64), cu, None, cu[1:], 128, 0, 0)


def test_index_rows_past_the_limit_are_refused(lib):
    big = (1 << 28) + 1
    assert lib.hisa_sparse_attention_kv4(D, D, D, D, D, D, 1, 4, 8, big, F(0.1), D, D, D, None) == 1
    assert lib.hisa_token_weights(D, D, D, D, D, D, 1, 4, 8, big, F(0.1), D, None) == 1
