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


def test_eviction_counts_over_an_input_are_refused(lib):
    """kept_len over seqlens_k, keep, the offsets or kept: the CTAs of a sequence read its length
    at different times."""
    f = lib.hisa_evict_select
    seqs = 4

    def call(weights=1 << 16, cu=2 << 16, lens=3 << 16, keep=4 << 16, kept=5 << 16, n=6 << 16,
             most=128):
        return f(P(weights), P(cu), P(lens) if lens else None, P(keep), seqs, most, 4, 4, P(kept),
                 P(n), None)
    assert call(most=-1) == 1  # the plain call is refused for other reasons only
    for change in (dict(n=3 << 16), dict(n=4 << 16), dict(n=2 << 16), dict(n=5 << 16),
                   dict(n=(3 << 16) + 4 * seqs - 4), dict(n=(4 << 16) - 4 * seqs + 4),
                   dict(n=(2 << 16) + 4 * seqs), dict(kept=1 << 16), dict(kept=2 << 16),
                   dict(kept=(3 << 16) + 4), dict(kept=4 << 16)):
        assert call(**change) == 1, change


def test_the_binding_is_built_again_for_another_torch(lib, monkeypatch):
    """Its accessors are compiled against the installed torch: newer than its sources is not
    enough to keep it."""
    import subprocess
    import types

    import torch

    from sparse_attention_top_hisa_b200 import build
    ran = []

    def run(cmd, **kw):
        ran.append(cmd)
        return types.SimpleNamespace(returncode=1, stdout="", stderr="not run")
    monkeypatch.setattr(subprocess, "run", run)
    assert build.build_binding() == build.BINDING and not ran  # up to date
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    with pytest.raises(RuntimeError, match="not run"):
        build.build_binding()
    assert len(ran) == 1 and any("torch 0.0.0" in x for x in ran[0])


def test_a_binding_of_another_torch_is_refused(lib, monkeypatch):
    import torch

    from sparse_attention_top_hisa_b200 import binding
    monkeypatch.setattr(binding, "_torch_binding", None)
    assert binding._native() is not None
    monkeypatch.setattr(binding, "_torch_binding", None)
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    with pytest.raises(ImportError, match="0.0.0"):
        binding._native()


def test_the_binding_refuses_calls_before_its_setup():
    import subprocess
    import sys

    code = ("import importlib.util as u, torch; from sparse_attention_top_hisa_b200 import build; "
            "s = u.spec_from_file_location('_hisa_torch', build.BINDING); m = u.module_from_spec(s); "
            "s.loader.exec_module(m); m.kv4_store(*[None] * 8)")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 1 and "setup() has not been called" in r.stderr
