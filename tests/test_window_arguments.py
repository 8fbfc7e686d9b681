"""What the bindings of the windowed, tree and commit calls take and refuse (CPU: the
library is not reached, tensors are stand-ins)."""
import types

import pytest
import torch

import moe_gqa_query_b200 as gq
from moe_gqa_query_b200 import _lib


def test_binding_takes_device_pointers_for_lengths_too():
    assert _lib._lens(4096, "cache_len", 3, 0) == 4096
    assert _lib._lens(None, "tree_len", 3, 0, True) is None


B, T, G, k, d, L = 2, 3, 2, 2, 64, 10
BF16, I32, F32 = torch.bfloat16, torch.int32, torch.float32
ROWS, SH, KV, CACHE = (B, G, T, k, d), (B, T, d), (B, G, T, d), (B, G, L, d)

# call: tokens, arguments as the binding takes them, tensors as (shape, type)
CALLS = {
    "gqe_attn_prefill_window": (T, [(ROWS, BF16), (SH, BF16), (KV, BF16), (KV, BF16), 5, 1, (ROWS, BF16), (SH, BF16),
                                    ((B * T * (G * k + 1),), F32)]),
    "gqe_attn_prefill_window_bwd": (T, [(ROWS, BF16), (SH, BF16), (KV, BF16), (KV, BF16), 5, 1, (ROWS, BF16), (SH, BF16),
                                        ((B * T * (G * k + 1),), F32), (ROWS, BF16), (SH, BF16), (ROWS, BF16), (SH, BF16),
                                        (KV, BF16), (KV, BF16), None]),
    "gqe_attn_decode_window": (1, [((B, G, 1, k, d), BF16), ((B, 1, d), BF16), (CACHE, BF16), (CACHE, BF16), L,
                                   ((B,), I32), 5, 1, ((B, G, 1, k, d), BF16), ((B, 1, d), BF16)]),
    "gqe_attn_tree": (T, [(ROWS, BF16), (SH, BF16), (KV, BF16), (KV, BF16), ((B, T), I32), ((B,), I32), (CACHE, BF16),
                          (CACHE, BF16), L, ((B,), I32), 5, 1, (ROWS, BF16), (SH, BF16)]),
    "gqe_cache_commit": (T, [(KV, BF16), (KV, BF16), ((B, T), I32), ((B,), I32), (CACHE, BF16), (CACHE, BF16), L,
                             ((B,), I32), ((B,), I32)]),
}


@pytest.fixture
def call(monkeypatch):
    """The binding in front of a library that only counts: host tensors stand for the device's
    (their device number is -1)."""
    reached = []
    fns = {name: (lambda *a, name=name: reached.append(name) or 0) for name in CALLS}
    monkeypatch.setattr(_lib, "lib", types.SimpleNamespace(**fns))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)
    monkeypatch.setattr(_lib, "_stream", lambda *a: None)

    def run(name, change=None, n_shared=1):
        tokens, args = CALLS[name]
        dims = gq.gqe_dims(B=B, T=tokens, d_model=64, G=G, E=2, k=k, d_head=d, n_shared=n_shared, shared_kv_group=0,
                           renorm_scope=0, scale=0.0, output_mode=0)
        args = [torch.zeros(*a[0], dtype=a[1]) if isinstance(a, tuple) else a for a in args]
        for i, v in (change or {}).items():
            args[i] = v(args[i])
        del reached[:]
        getattr(_lib, name)(dims, *args)
        assert reached == [name]
    return run, reached


TENSORS = [(name, i) for name, (_, args) in CALLS.items() for i, a in enumerate(args) if isinstance(a, tuple)]


@pytest.mark.parametrize("name", list(CALLS))
def test_full_tensors_pass(call, name):
    run, _ = call
    run(name)
    run(name, {i: (lambda t: torch.cat([t, t])) for n, i in TENSORS                 # larger ones too, but for lengths
               if n == name and CALLS[name][1][i][1] != I32})


@pytest.mark.parametrize("name,i", TENSORS)
def test_a_tensor_too_small_for_the_call_is_refused(call, name, i):
    """One row, sequence or group short: the call would go past its end."""
    run, reached = call
    with pytest.raises(ValueError, match="elements|entries"):
        run(name, {i: lambda t: t.reshape(-1)[:-1]})
    with pytest.raises(ValueError, match="elements|entries"):
        run(name, {i: lambda t: t[:1] if t.dim() > 1 else t[:-1]})
    assert not reached


def test_without_a_shared_head_its_tensors_are_not_looked_at(call):
    run, _ = call
    for name in ("gqe_attn_prefill_window", "gqe_attn_tree"):
        sh = [i for n, i in TENSORS if n == name and CALLS[name][1][i][0] == SH]
        run(name, {i: lambda t: None for i in sh}, n_shared=0)
        run(name, {i: lambda t: t[:1] for i in sh}, n_shared=0)


def test_a_cache_length_past_32_bits_is_refused(call):
    """ctypes would cut it to its low 32 bits."""
    run, _ = call
    with pytest.raises(ValueError, match="elements"):
        run("gqe_attn_tree", {8: lambda v: v + 2 ** 32})
