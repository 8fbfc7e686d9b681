"""Refusals and sizes of the windowed, tree and cache calls (CPU only: every
call here returns before it launches anything)."""
import ctypes

import pytest
import torch

import moe_gqa_query_b200 as gq
from moe_gqa_query_b200 import _lib

lib = _lib.lib


def dims(**kw):
    base = dict(B=2, T=300, D=256, G=2, E=2, k=1, d=64)
    base.update(kw)
    return gq.make_dims(type("C", (), base)(), **{k: v for k, v in kw.items() if k in ("n_shared",)})


def prefill(d, window=64, sinks=4, q=256, qs=256, K=256, V=256, o=256, os_=256):
    return lib.gqe_attn_prefill_window(ctypes.byref(d), q, qs, K, V, window, sinks, o, os_, None, None)


def test_prefill_window_arguments():
    assert prefill(dims(), window=-1) == 1
    assert prefill(dims(), sinks=-3) == 1
    assert prefill(dims(), q=None) == 1
    assert prefill(dims(), qs=None) == 1
    assert prefill(dims(), K=264) == 1            # not 16-byte aligned
    assert prefill(dims(d=96)) == 2
    assert prefill(dims(k=3)) == 1


def test_prefill_window_bwd_arguments():
    d = dims()
    call = lambda w, s, ptrs, ws, n: lib.gqe_attn_prefill_window_bwd(  # noqa: E731
        ctypes.byref(d), *ptrs[:4], w, s, *ptrs[4:], ws, n, None)
    ok = [256] * 13
    need = gq.gqe_window_workspace_size(d, gq.GQE_OP_ATTN_WINDOW_BWD, 0, 64, 4)
    assert call(-1, 0, ok, 256, need) == 1
    assert call(64, -1, ok, 256, need) == 1
    assert call(64, 4, [None] + ok[1:], 256, need) == 1
    assert call(64, 4, ok, 256, need - 1) == 3
    assert call(64, 4, ok, None, need) == 3
    assert call(64, 4, ok, 128, need) == 3        # not 256-byte aligned


def test_prefill_window_bwd_row_count():
    # one-token sequences take a 128-row tile each: 2^24 of them are 2^31 rows
    size = lambda B: lib.gqe_window_workspace_size(  # noqa: E731
        ctypes.byref(dims(B=B, T=1, G=1, E=4, k=1, D=64, n_shared=0)), gq.GQE_OP_ATTN_WINDOW_BWD, 0, 0, 0,
        ctypes.byref(ctypes.c_size_t()))
    assert size((1 << 24) - 1) == 0
    assert size(1 << 24) == 2


def tree(d, L=100, q=256, Kt=256, parent=256, Kc=256, clen=256, window=0, sinks=0, o=256):
    return lib.gqe_attn_tree(ctypes.byref(d), q, 256, Kt, 256, parent, None, Kc, 256, L, clen, window, sinks, o, 256, None,
                             0, None)


def test_tree_arguments():
    d = dims(T=8)
    for bad in (dict(L=0), dict(q=None), dict(Kt=None), dict(parent=None), dict(Kc=None), dict(clen=None), dict(o=None),
                dict(window=-1), dict(sinks=-1), dict(Kt=260), dict(o=258)):
        assert tree(d, **bad) == 1, bad
    assert tree(dims(T=129)) == 2                 # at most 128 drafted tokens
    assert tree(dims(T=8, d=32)) == 2


def test_decode_window_arguments():
    call = lambda d, L=100, w=10, s=0, clen=256: lib.gqe_attn_decode_window(  # noqa: E731
        ctypes.byref(d), 256, 256, 256, 256, L, clen, w, s, 256, 256, None, 0, None)
    assert call(dims(T=2)) == 1                   # one token per sequence
    assert call(dims(T=1), L=0) == 1
    assert call(dims(T=1), w=-2) == 1
    assert call(dims(T=1), s=-2) == 1
    assert call(dims(T=1), clen=None) == 1


def test_commit_arguments():
    call = lambda d, L=100, Kt=256, path=256, new=256: lib.gqe_cache_commit(  # noqa: E731
        ctypes.byref(d), Kt, 256, path, 256, 256, 256, L, 256, new, None)
    assert call(dims(T=8), L=0) == 1
    assert call(dims(T=8), Kt=None) == 1
    assert call(dims(T=8), Kt=264) == 1
    assert call(dims(T=8), path=None) == 1
    assert call(dims(T=8), new=None) == 1
    assert call(dims(T=129)) == 2


def test_workspace_sizes():
    d = dims()
    plain = gq.gqe_workspace_size(d, gq.GQE_OP_ATTN_BWD)
    size = lambda *a: gq.gqe_window_workspace_size(*a)  # noqa: E731
    # two fp32 [2, 128, d] slots for each stretch of the walks, four stretches per SM at most
    for window in (0, 1, 64, 300, 10 ** 9):
        w = size(d, gq.GQE_OP_ATTN_WINDOW_BWD, 0, window, 5)
        assert plain < w <= plain + 255 + 4 * 148 * 2 * 2 * 128 * 64 * 4
    assert size(dims(T=1), gq.GQE_OP_ATTN_DECODE_WINDOW, 4096, 100, 4) == 0
    assert size(dims(T=128), gq.GQE_OP_ATTN_TREE, 4096, 0, 0) == 0
    for args, status in (((d, gq.GQE_OP_ATTN_TREE, 4096, 0, 0), 2), ((dims(T=8), gq.GQE_OP_ATTN_TREE, 0, 0, 0), 1),
                         ((d, gq.GQE_OP_ATTN_DECODE_WINDOW, 4096, 0, 0), 1), ((d, gq.GQE_OP_ATTN_BWD, 0, 5, 0), 1),
                         ((d, gq.GQE_OP_ATTN_WINDOW_BWD, 0, -5, 0), 1), ((d, gq.GQE_OP_ATTN_WINDOW_BWD, 0, 5, -1), 1)):
        with pytest.raises(gq.GQEError) as ei:
            size(*args)
        assert ei.value.status == status, args


def test_binding_refuses_host_and_wrong_tensors():
    """The binding looks at type, place and layout before it calls the library."""
    with pytest.raises(ValueError, match="must be torch.bfloat16|CUDA"):
        _lib._dev(torch.zeros(4), "x", torch.bfloat16, 0)
    with pytest.raises(ValueError, match="CUDA"):
        _lib._dev(torch.zeros(4, dtype=torch.bfloat16), "x", torch.bfloat16, 0)
    with pytest.raises(ValueError, match="required"):
        _lib._dev(None, "x", torch.bfloat16, 0)
    assert _lib._dev(None, "x", torch.bfloat16, 0, True) is None


def test_windowed_config_values():
    base = dict(B=1, T=8, D=64, G=1, E=1, k=1, d=64)
    assert gq.GQEConfig(**base).window == 0
    for bad in (dict(window=-1), dict(sinks=-1)):
        with pytest.raises(ValueError):
            gq.GQEConfig(**base, **bad)
