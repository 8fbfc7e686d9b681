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


def test_layer_looks_at_its_cache():
    """decode_step, decode_tree and commit take L_max from the cache and the rest of its shape from
    the layer and the batch: the two must agree."""
    from moe_gqa_query_b200.layer import check_cache
    cfg = gq.GQEConfig(B=B, T=T, D=64, G=G, E=2, k=k, d=d)
    new = lambda *s: torch.zeros(*s, dtype=BF16)  # noqa: E731
    assert check_cache(cfg, B, new(*CACHE), new(*CACHE)) == L
    assert check_cache(cfg, B, new(B + 3, G, L, d), new(B + 3, G, L, d)) == L      # the first B sequences of a larger one
    for bad in ((B - 1, G, L, d), (B, G - 1, L, d), (B, G + 1, L, d), (B, G, L, 2 * d), (B, G * L, d)):
        with pytest.raises(ValueError, match="cache"):
            check_cache(cfg, B, new(*bad), new(*bad))
    with pytest.raises(ValueError, match="differ"):
        check_cache(cfg, B, new(*CACHE), new(B, G, L + 1, d))


@pytest.mark.parametrize("step", ["decode_step", "decode_tree", "commit"])
def test_layer_refuses_a_cache_before_it_launches_anything(monkeypatch, step):
    from moe_gqa_query_b200 import layer as mod
    for name in ("gqe_router_topk", "gqe_routed_qproj", "gqe_kv_append", "gqe_kv_proj", "gqe_cache_commit"):
        monkeypatch.setattr(mod.L, name, lambda *a: pytest.fail("launched"))
    self = object.__new__(mod.GQELayer)
    self.cfg = gq.GQEConfig(B=B, T=T, D=64, G=G, E=2, k=k, d=d, window=4)
    new = lambda *s: torch.zeros(*s, dtype=BF16)  # noqa: E731
    i32 = lambda *s: torch.zeros(*s, dtype=I32)  # noqa: E731
    Kc, Vc = new(B, G - 1, L, d), new(B, G - 1, L, d)
    with pytest.raises(ValueError, match="cache"):
        if step == "decode_step":
            self.decode_step(new(B, 64), Kc, Vc, i32(B))
        elif step == "decode_tree":
            self.decode_tree(new(B, T, 64), i32(B, T), Kc, Vc, i32(B))
        else:
            self.commit(dict(K=new(*KV), V=new(*KV)), i32(B, T), i32(B), Kc, Vc, i32(B))


def test_scratch_of_the_windowed_backward_is_4d_plus_8_bytes_a_row():
    """dq's fp32 sums, -LSE2 and -Delta of every row of the padded space; 2^31 rows, which are refused,
    would take 567 GB at d = 64."""
    for width, most in ((64, 570e9), (128, 1.12e12)):
        dims = gq.gqe_dims(B=(1 << 24) - 1, T=1, d_model=64, G=1, E=1, k=1, d_head=width, n_shared=0,
                           shared_kv_group=0, renorm_scope=0, scale=0.0, output_mode=0)
        need = gq.gqe_window_workspace_size(dims, gq.GQE_OP_ATTN_WINDOW_BWD, 0, 0, 0)
        assert 128 * dims.B * (4 * width + 8) <= need <= most
