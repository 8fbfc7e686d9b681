"""Parity of the windowed, tree and cache calls with the fp64 oracle (GPU).

Outputs are held to the worst-case error of their arithmetic
(oracle/gqe_window.py: bf16 rounding of the P and dS operands, fp32 sums, the
approximate exponential) plus the final bf16 rounding; no tolerance is fitted.
"""
import numpy as np
import pytest
import torch

import gqe_inputs as gi
from oracle import gqe_window as ow
from helpers import BF16_U, bf16_dev, to_f64

pytestmark = pytest.mark.gpu

gq = pytest.importorskip("moe_gqa_query_b200")

NAN = float("nan")
BF16 = torch.bfloat16


@pytest.fixture(autouse=True)
def _cuda_and_error_word():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield
    torch.cuda.synchronize()
    assert gq.gqe_device_error() == 0


def D(**kw):
    base = dict(B=1, T=128, D=64, G=2, E=2, k=1, d=64)
    base.update(kw)
    return gi.GQEDims(**base)


def close(got, ref, bound, what):
    """|err| <= 2^-8 |ref| + bound + 1e-6 (fp32 values near 0)."""
    got, ref = to_f64(got), np.asarray(ref)
    assert got.shape == ref.shape, what
    assert np.isfinite(got).all(), f"{what}: non-finite"
    r = np.abs(got - ref) / (BF16_U * np.abs(ref) + bound + 1e-6)
    assert r.size == 0 or r.max() <= 1.0, f"{what}: worst err/bound {r.max():.3f} at {np.unravel_index(r.argmax(), r.shape)}"


def i32(v):
    return torch.tensor(np.asarray(v), dtype=torch.int32, device="cuda")


def full(*shape, dtype=BF16):
    return torch.full(shape, NAN, dtype=dtype, device="cuda")


# ----------------------------------------------------------------------------
# prefill and its backward

def _prefill_inputs(dims, seed):
    B, G, T, k, d = dims.B, dims.G, dims.T, dims.k, dims.d
    return dict(q=gi.normal_bf16(seed, "q", (B, G, T, k, d)),
                qs=gi.normal_bf16(seed, "qsh", (B, T, d)) if dims.n_shared else None,
                K=gi.normal_bf16(seed, "K", (B, G, T, d)), V=gi.normal_bf16(seed, "V", (B, G, T, d)))


def _run_prefill(dims, x, window, sinks, stream=None):
    B, G, T, k, d = dims.B, dims.G, dims.T, dims.k, dims.d
    dev = {n: None if v is None else bf16_dev(v) for n, v in x.items()}
    o = full(B, G, T, k, d)
    os_ = full(B, T, d) if dims.n_shared else None
    lse = full(B * G * T * k + B * T * dims.n_shared, dtype=torch.float32)
    gq.gqe_attn_prefill_window(gq.make_dims(dims), dev["q"], dev["qs"], dev["K"], dev["V"], window, sinks, o, os_, lse,
                               stream)
    return dev, o, os_, lse


# (dims, window, sinks): tile borders at 128, windows shorter than a tile, rows
# that see nothing of a tile, sinks past the window start, k packing, d = 128 pairs
PREFILL = {
    "one_token": (D(T=1, B=2), 3, 1),
    "window_one": (D(T=130), 1, 0),
    "window_one_sink": (D(T=300, k=2), 1, 1),
    "half_tile": (D(T=128), 64, 4),
    "ragged_k2": (D(B=2, T=333, G=3, E=3, k=2, sg=1), 100, 7),
    "tile_window": (D(T=700, k=1), 128, 0),
    "window_past_tile": (D(T=700, k=1), 129, 128),
    "many_sinks": (D(T=700, k=1), 40, 300),
    "k3_no_shared": (D(B=2, T=400, G=1, E=3, k=3, n_shared=0), 130, 2),
    "k8": (D(T=150, G=1, E=8, k=8), 33, 5),
    "sinks_cover_all": (D(T=300), 10, 300),
    "d128_half_tile": (D(T=257, d=128), 64, 4),
    "d128_gap": (D(T=1000, d=128, G=1), 128, 1),
    "d128_gap_no_sink": (D(T=1000, d=128, G=1, sg=0), 200, 0),
    "d128_window_one": (D(T=600, d=128, G=1), 1, 0),
    "d128_k4": (D(T=500, d=128, E=4, k=4, sg=1), 77, 130),
    "d128_k3_many_sinks": (D(T=700, d=128, E=4, k=3, G=1), 150, 400),
    "window_over_T": (D(T=200, k=2), 500, 3),
    "no_window": (D(T=200, k=2), 0, 3),
}


@pytest.mark.parametrize("case", list(PREFILL))
def test_prefill_window(case):
    dims, window, sinks = PREFILL[case]
    x = _prefill_inputs(dims, 11)
    _, o, os_, lse = _run_prefill(dims, x, window, sinks)
    (ro, rs, rl), (bo, bs) = ow.attn_prefill_window(x["q"], x["qs"], x["K"], x["V"], dims, window, sinks)
    close(o, ro, bo, "o_routed")
    if dims.n_shared:
        close(os_, rs, bs, "o_sh")
    # lse: e = scale d 2^-24 |q||K| (< 3e-5 at these sizes) + 1e-4 of the sum + fp32 rounding of the value
    assert np.abs(to_f64(lse) - rl).max() <= 2e-4


@pytest.mark.parametrize("case", ["window_over_T", "no_window"])
def test_prefill_without_a_bound_is_the_causal_call(case):
    dims, window, sinks = PREFILL[case]
    x = _prefill_inputs(dims, 12)
    dev, o, os_, lse = _run_prefill(dims, x, window, sinks)
    o2, os2, lse2 = torch.empty_like(o), torch.empty_like(os_), torch.empty_like(lse)
    gq.gqe_attn_prefill(gq.make_dims(dims), dev["q"], dev["qs"], dev["K"], dev["V"], o2, os2, lse2)
    assert torch.equal(o, o2) and torch.equal(os_, os2) and torch.equal(lse, lse2)


def _run_bwd(dims, dev, window, sinks, o, os_, lse, do, dos):
    nan_ws = full(gq.gqe_window_workspace_size(gq.make_dims(dims), gq.GQE_OP_ATTN_WINDOW_BWD, 0, window, sinks) // 4,
                  dtype=torch.float32)
    dq, dK, dV = full(*o.shape), full(*dev["K"].shape), full(*dev["K"].shape)
    dqs = full(*os_.shape) if os_ is not None else None
    gq.gqe_attn_prefill_window_bwd(gq.make_dims(dims), dev["q"], dev["qs"], dev["K"], dev["V"], window, sinks, o, os_,
                                   lse, do, dos, dq, dqs, dK, dV, nan_ws)
    return dq, dqs, dK, dV


# few sequences: every stretch ends inside a walk, the sink tiles' walks span many; many sequences: most walks whole
BWD = dict(PREFILL, three_tokens=(D(T=3, B=4, G=1), 67, 0), ten_tokens=(D(T=10, B=2, G=4, sg=3), 594, 1),
           two_keys=(D(T=300, k=2), 2, 0), few_keys_d128=(D(T=300, d=128), 9, 6), few_and_many=(D(T=300), 16, 1),
           split_one_sink=(D(T=5000, G=1), 300, 1), split_two_tiles=(D(T=4500, G=1, E=4, k=2, sg=0), 64, 200),
           split_d128=(D(T=3000, G=1, E=4, k=2, d=128), 256, 5), sinks_unsplit=(D(B=8, T=2600, G=2, n_shared=0), 30, 2500))


@pytest.mark.parametrize("case", list(BWD))
def test_prefill_window_backward(case):
    dims, window, sinks = BWD[case]
    x = _prefill_inputs(dims, 13)
    do = gi.normal_bf16(13, "do", x["q"].shape)
    dos = gi.normal_bf16(13, "dosh", x["qs"].shape) if dims.n_shared else None
    dev, o, os_, lse = _run_prefill(dims, x, window, sinks)
    dq, dqs, dK, dV = _run_bwd(dims, dev, window, sinks, o, os_, lse, bf16_dev(do),
                               bf16_dev(dos) if dims.n_shared else None)
    if dims.B > 4:       # the large case: two sequences of the batch
        keep = [0, dims.B - 1]
        R = dims.G * dims.T * dims.k
        lse = torch.cat([lse[b * R:(b + 1) * R] for b in keep])
        dims = dims.replace(B=2)
        x = {n: None if v is None else v[keep] for n, v in x.items()}
        do, o, dq, dK, dV = do[keep], o[keep], dq[keep], dK[keep], dV[keep]
    ref, bnd = ow.attn_prefill_window_bwd(x["q"], x["qs"], x["K"], x["V"], window, sinks, to_f64(lse), do, dos, dims)
    for name, got, r, b in zip(("dq", "dq_sh", "dK", "dV"), (dq, dqs, dK, dV), ref, bnd):
        if got is not None:
            close(got, r, b, name)


def test_window_backward_dK_dV_are_deterministic():
    dims, window, sinks = BWD["split_two_tiles"]
    x = _prefill_inputs(dims, 14)
    do, dos = bf16_dev(gi.normal_bf16(14, "do", x["q"].shape)), bf16_dev(gi.normal_bf16(14, "dosh", x["qs"].shape))
    dev, o, os_, lse = _run_prefill(dims, x, window, sinks)
    a = _run_bwd(dims, dev, window, sinks, o, os_, lse, do, dos)
    b = _run_bwd(dims, dev, window, sinks, o, os_, lse, do, dos)
    assert torch.equal(a[2], b[2]) and torch.equal(a[3], b[3])


@pytest.mark.parametrize("window,sinks", [(700, 3), (0, 0)])
def test_window_backward_in_rounds(window, sinks):
    """A batch whose dq sums (69 MB) are worked on in two rounds of stretches:
    the sequences at both ends and on both sides of the rounds' border."""
    dims = D(B=32, T=1400, G=2, k=1, d=128)
    plain = gq.gqe_workspace_size(gq.make_dims(dims), gq.GQE_OP_ATTN_BWD)
    need = gq.gqe_window_workspace_size(gq.make_dims(dims), gq.GQE_OP_ATTN_WINDOW_BWD, 0, window, sinks)
    assert need > plain + 148 * 2 * 2 * 128 * 128 * 4 + 256
    x = _prefill_inputs(dims, 16)
    do, dos = gi.normal_bf16(16, "do", x["q"].shape), gi.normal_bf16(16, "dosh", x["qs"].shape)
    dev, o, os_, lse = _run_prefill(dims, x, window, sinks)
    got = _run_bwd(dims, dev, window, sinks, o, os_, lse, bf16_dev(do), bf16_dev(dos))
    for t in got:
        assert torch.isfinite(t).all()
    keep = [0, 15, 16, 31]
    R, R_sh = dims.G * dims.T, dims.B * dims.G * dims.T
    lse = torch.cat([lse[b * R:(b + 1) * R] for b in keep] + [lse[R_sh + b * 1400:R_sh + (b + 1) * 1400] for b in keep])
    x = {n: v[keep] for n, v in x.items()}
    ref, bnd = ow.attn_prefill_window_bwd(x["q"], x["qs"], x["K"], x["V"], window, sinks, to_f64(lse), do[keep],
                                          dos[keep], dims.replace(B=4))
    for name, t, r, b in zip(("dq", "dq_sh", "dK", "dV"), got, ref, bnd):
        close(t[keep], r, b, name)


def test_window_backward_replayed_from_one_graph():
    """The schedule travels with the launch: replays follow new inputs in the same tensors."""
    dims, window, sinks = BWD["few_and_many"]
    x, y = _prefill_inputs(dims, 18), _prefill_inputs(dims, 19)
    do, dos = bf16_dev(gi.normal_bf16(18, "do", x["q"].shape)), bf16_dev(gi.normal_bf16(18, "dosh", x["qs"].shape))
    dev, o, os_, lse = _run_prefill(dims, x, window, sinks)
    dq, dK, dV, dqs = (full(*t.shape) for t in (o, dev["K"], dev["K"], os_))
    ws = full(gq.gqe_window_workspace_size(gq.make_dims(dims), gq.GQE_OP_ATTN_WINDOW_BWD, 0, window, sinks) // 4,
              dtype=torch.float32)

    def step():
        gq.gqe_attn_prefill_window(gq.make_dims(dims), dev["q"], dev["qs"], dev["K"], dev["V"], window, sinks, o, os_,
                                   lse)
        gq.gqe_attn_prefill_window_bwd(gq.make_dims(dims), dev["q"], dev["qs"], dev["K"], dev["V"], window, sinks, o,
                                       os_, lse, do, dos, dq, dqs, dK, dV, ws)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for n in dev:
        dev[n].copy_(bf16_dev(y[n]))
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    dev2, o2, os2, lse2 = _run_prefill(dims, y, window, sinks)
    _, _, dK2, dV2 = _run_bwd(dims, dev2, window, sinks, o2, os2, lse2, do, dos)
    assert torch.equal(o, o2) and torch.equal(dK, dK2) and torch.equal(dV, dV2)


def test_bounds_past_32_bits_do_not_wrap():
    dims, _, _ = PREFILL["window_over_T"]
    x = _prefill_inputs(dims, 20)
    _, a, _, _ = _run_prefill(dims, x, 0, 0)
    _, b, _, _ = _run_prefill(dims, x, 2 ** 32 + 5, 2 ** 33)
    assert torch.equal(a, b)
    with pytest.raises(gq.GQEError):
        _run_prefill(dims, x, -2 ** 32 + 5, 0)
    dims, L, lens, _, _ = DECODE["no_window"]
    x = _cache_inputs(dims, L, 21)
    dev = {n: None if v is None else bf16_dev(v) for n, v in x.items()}
    outs = []
    for w, s in ((0, 0), (2 ** 31 - 1, 2 ** 31 - 1), (2 ** 32 + 5, 2 ** 40)):
        o, os_ = full(*dev["q"].shape), full(*dev["qs"].shape)
        gq.gqe_attn_decode_window(gq.make_dims(dims), dev["q"], dev["qs"], dev["Kc"], dev["Vc"], L, i32(lens), w, s, o,
                                  os_)
        outs.append(o)
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


@pytest.mark.parametrize("case", ["window_one", "one_token"])
def test_one_visible_key_has_no_score_gradient(case):
    dims, window, sinks = PREFILL[case]
    x = _prefill_inputs(dims, 15)
    dev, o, os_, lse = _run_prefill(dims, x, window, sinks)
    dq, dqs, dK, dV = _run_bwd(dims, dev, window, sinks, o, os_, lse, torch.ones_like(o), torch.ones_like(os_))
    assert not dq.any() and not dqs.any() and not dK.any()


# ----------------------------------------------------------------------------
# drafted trees and windowed decode

def random_parents(B, T, seed, chain=False):
    rng = np.random.default_rng(seed)
    if chain:
        return np.tile(np.arange(T) - 1, (B, 1)).astype(np.int32)
    return np.stack([[max(-1, i - 1 - int(rng.integers(0, 5))) if rng.random() > 0.15 else -1 for i in range(T)]
                     for _ in range(B)]).astype(np.int32)


def _cache_inputs(dims, L, seed):
    B, G, T, k, d = dims.B, dims.G, dims.T, dims.k, dims.d
    x = _prefill_inputs(dims, seed)
    x.update(Kc=gi.normal_bf16(seed, "Kc", (B, G, L, d)), Vc=gi.normal_bf16(seed, "Vc", (B, G, L, d)))
    return x


def _poison(t, rows):
    """NaN and infinities in the K or V rows (b, slice) of a [B, G, L, d] tensor."""
    for b, sl in rows:
        t[b, :, sl, 0::2] = NAN
        t[b, :, sl, 1::2] = float("inf")


def _run_tree(dims, L, lens, tlens, parent, x, window, sinks, poison=True, stream=None):
    dc = gq.make_dims(dims)
    dev = {n: None if v is None else bf16_dev(v) for n, v in x.items()}
    tl = [dims.T] * dims.B if tlens is None else tlens
    if poison:
        for n in ("Kc", "Vc"):
            _poison(dev[n], [(b, slice(int(lens[b]), L)) for b in range(dims.B)])
            if window:       # between the sinks and the first drafted token's window
                _poison(dev[n], [(b, slice(sinks, max(sinks, int(lens[b]) - window + 1))) for b in range(dims.B)])
        for n in ("K", "V"):
            _poison(dev[n], [(b, slice(int(tl[b]), dims.T)) for b in range(dims.B)])
        for b in range(dims.B):
            dev["q"][b, :, int(tl[b]):] = NAN
    o = full(*dev["q"].shape)
    os_ = full(*dev["qs"].shape) if dims.n_shared else None
    n = gq.gqe_window_workspace_size(dc, gq.GQE_OP_ATTN_TREE, L, window, sinks)
    ws = full(max(n, 256) // 4, dtype=torch.float32)
    gq.gqe_attn_tree(dc, dev["q"], dev["qs"], dev["K"], dev["V"], i32(parent), None if tlens is None else i32(tlens),
                     dev["Kc"], dev["Vc"], L, i32(lens), window, sinks, o, os_, ws, stream)
    return dev, o, os_


# dims, L_max, cache lengths, tree lengths (None: all), window, sinks, chain
TREE = {
    "one_token": (D(T=1, B=2), 300, [300, 1], None, 0, 0, False),
    "empty_cache": (D(T=9, B=2), 200, [0, 0], None, 0, 0, False),
    "no_live_token": (D(T=5, B=3), 200, [0, 100, 200], [0, 0, 5], 0, 0, False),
    "rep4": (D(T=8, B=3, G=3, sg=2), 700, [700, 129, 0], [8, 3, 1], 0, 0, False),
    "rep2": (D(T=40, B=2), 900, [900, 513], [40, 33], 0, 0, False),
    "rep1": (D(T=100, B=2, n_shared=0), 600, [600, 255], [100, 65], 0, 0, False),
    "tree_128": (D(T=128, B=2, G=1, k=1), 400, [400, 128], [128, 127], 0, 0, False),
    "k8_two_tiles": (D(T=63, G=1, E=8, k=8), 500, [499], None, 0, 0, False),
    "k3_odd": (D(T=37, B=2, G=3, E=3, k=3, sg=1), 777, [777, 650], [37, 2], 0, 0, False),
    "chain": (D(T=20, B=2), 300, [257, 128], [20, 11], 0, 0, True),
    "many_shares": (D(T=4, G=1), 9000, [8999], None, 0, 0, False),
    "window": (D(T=24, B=3, E=4, k=2), 1500, [1500, 640, 7], [24, 24, 20], 300, 4, False),
    "window_no_sink": (D(T=24, B=2, k=1), 1500, [1500, 1301], None, 129, 0, False),
    "window_in_tree": (D(T=60, B=2, k=1), 400, [300, 2], [60, 59], 5, 3, True),
    "window_one": (D(T=30, B=2, k=1), 400, [300, 0], None, 1, 0, False),
    "window_one_sinks_in_tree": (D(T=40, B=2, k=1), 400, [3, 200], None, 1, 6, True),
    "sinks_over_tile": (D(T=24, B=2, k=1), 1500, [1500, 200], None, 100, 260, False),
    "d128_rep4": (D(T=5, B=2, d=128), 700, [700, 65], [5, 4], 0, 0, False),
    "d128_rep2": (D(T=20, B=2, E=3, k=2, d=128), 700, [699, 0], [20, 19], 0, 0, False),
    "d128_rep1": (D(T=100, B=2, d=128, n_shared=0), 300, [300, 63], [100, 64], 0, 0, False),
    "d128_k4_window": (D(T=63, B=2, E=4, k=4, d=128, sg=1), 1200, [1200, 801], [63, 50], 257, 2, False),
    "d128_window_in_tree": (D(T=128, B=1, G=1, d=128), 300, [200], None, 7, 1, True),
}


@pytest.mark.parametrize("case", list(TREE))
def test_tree(case):
    dims, L, lens, tlens, window, sinks, chain = TREE[case]
    x = _cache_inputs(dims, L, 17)
    parent = random_parents(dims.B, dims.T, 17, chain)
    tl = [dims.T] * dims.B if tlens is None else tlens
    _, o, os_ = _run_tree(dims, L, lens, tlens, parent, x, window, sinks)
    (ro, rs), (bo, bs) = ow.attn_tree(x["q"], x["qs"], x["K"], x["V"], parent, tl, x["Kc"], x["Vc"], lens, dims, window,
                                      sinks)
    close(o, ro, bo, "o_routed")
    if dims.n_shared:
        close(os_, rs, bs, "o_sh")
    for b in range(dims.B):
        assert not o[b, :, tl[b]:].any()


def test_tree_sharp_scores():
    """Scores that grow along the cache (every tile rescales) and scores in the hundreds."""
    dims, L = D(T=12, B=2), 1000
    x = _cache_inputs(dims, L, 18)
    K = gi.bf16_bits_to_f32(x["Kc"]) * np.linspace(0.1, 30, L, dtype=np.float32)[None, None, :, None]
    x["Kc"] = gi.f32_to_bf16_bits(K)
    parent = random_parents(2, 12, 18)
    _, o, os_ = _run_tree(dims, L, [1000, 990], None, parent, x, 0, 0)
    (ro, rs), (bo, bs) = ow.attn_tree(x["q"], x["qs"], x["K"], x["V"], parent, [12, 12], x["Kc"], x["Vc"], [1000, 990],
                                      dims, 0, 0)
    close(o, ro, bo, "o_routed")
    close(os_, rs, bs, "o_sh")


def test_tree_a_nan_query_stays_in_its_row():
    """A NaN in one live token's query makes that row NaN and leaves the others alone."""
    for shape in (D(T=6, B=2), D(T=100, B=1, n_shared=0), D(T=5, B=1, d=128)):
        L, B = 700, shape.B
        x = _cache_inputs(shape, L, 20)
        parent = random_parents(B, shape.T, 20)
        (ro, _), (bo, _) = ow.attn_tree(x["q"], x["qs"], x["K"], x["V"], parent, [shape.T] * B, x["Kc"], x["Vc"], [600] * B,
                                        shape, 0, 0)
        x["q"][0, 1, 3, 0, 7] = 0x7FC0
        _, o, _ = _run_tree(shape, L, [600] * B, None, parent, x, 0, 0, poison=False)
        assert torch.isnan(o[0, 1, 3]).all()
        o[0, 1, 3], ro[0, 1, 3], bo[0, 1, 3] = 0, 0, 0
        close(o, ro, bo, "the other rows")


def test_tree_bad_values_are_flagged_and_contained():
    dims, L = D(T=6, B=3), 200
    x = _cache_inputs(dims, L, 19)
    parent = random_parents(3, 6, 19)
    good = parent.copy()
    parent[0, 2], good[0, 2] = 2, -1           # itself
    parent[1, 4], good[1, 4] = 77, -1          # past the tree
    parent[2, 1], good[2, 1] = -9, -1
    (ro, rs), (bo, bs) = ow.attn_tree(x["q"], x["qs"], x["K"], x["V"], good, [6] * 3, x["Kc"], x["Vc"], [150] * 3, dims,
                                      0, 0)
    _, o, os_ = _run_tree(dims, L, [150] * 3, None, parent, x, 0, 0, poison=False)
    torch.cuda.synchronize()
    assert gq.gqe_device_error() == 0x304
    close(o, ro, bo, "o_routed")
    _, o, os_ = _run_tree(dims, L, [150] * 3, [6, 9, -2], good, x, 0, 0, poison=False)
    torch.cuda.synchronize()
    assert gq.gqe_device_error() == 0x304
    close(o[:2], ro[:2], bo[:2], "tree_len past T is T")
    assert not o[2].any() and not os_[2].any()
    _, o, os_ = _run_tree(dims, L, [150, L + 3, -1], None, good, x, 0, 0, poison=False)
    torch.cuda.synchronize()
    assert gq.gqe_device_error() == 0x302
    (ro, rs), (bo, bs) = ow.attn_tree(x["q"], x["qs"], x["K"], x["V"], good, [6] * 3, x["Kc"], x["Vc"], [150, L, 0], dims,
                                      0, 0)
    close(o, ro, bo, "clamped lengths")


# dims (T = 1), L_max, cache lengths, window, sinks
DECODE = {
    "one_row": (D(T=1, B=2), 64, [1, 64], 5, 0),
    "window_one": (D(T=1, B=3), 300, [1, 128, 300], 1, 0),
    "sinks_behind": (D(T=1, B=3, G=3, E=4, k=3, sg=1), 2000, [2000, 1025, 3], 200, 5),
    "sinks_meet_window": (D(T=1, B=2), 700, [700, 260], 250, 300),
    "window_over_cache": (D(T=1, B=2, n_shared=0), 700, [700, 1], 5000, 2),
    "no_window": (D(T=1, B=2, k=2), 700, [700, 90], 0, 0),
    "k8": (D(T=1, B=2, G=1, E=8, k=8), 900, [900, 513], 333, 1),
    "d128_odd": (D(T=1, B=3, E=4, k=4, d=128, sg=1), 1191, [1191, 640, 64], 500, 0),
    "d128_sinks": (D(T=1, B=2, d=128), 1191, [1191, 100], 65, 70),
}


@pytest.mark.parametrize("case", list(DECODE))
def test_decode_window(case):
    dims, L, lens, window, sinks = DECODE[case]
    x = _cache_inputs(dims, L, 23)
    dc = gq.make_dims(dims)
    dev = {n: None if v is None else bf16_dev(v) for n, v in x.items()}
    for n in ("Kc", "Vc"):
        _poison(dev[n], [(b, slice(int(lens[b]), L)) for b in range(dims.B)])
        if window:
            _poison(dev[n], [(b, slice(sinks, max(sinks, int(lens[b]) - window))) for b in range(dims.B)])
    o = full(*dev["q"].shape)
    os_ = full(*dev["qs"].shape) if dims.n_shared else None
    ws = full(max(256, gq.gqe_window_workspace_size(dc, gq.GQE_OP_ATTN_DECODE_WINDOW, L, window, sinks)) // 4,
              dtype=torch.float32)
    gq.gqe_attn_decode_window(dc, dev["q"], dev["qs"], dev["Kc"], dev["Vc"], L, i32(lens), window, sinks, o, os_, ws)
    (ro, rs), (bo, bs) = ow.attn_decode_window(x["q"], x["qs"], x["Kc"], x["Vc"], lens, dims, window, sinks)
    close(o, ro, bo, "o_routed")
    if dims.n_shared:
        close(os_, rs, bs, "o_sh")


def test_decode_window_lengths_out_of_range():
    dims, L = D(T=1, B=3), 200
    x = _cache_inputs(dims, L, 24)
    dc = gq.make_dims(dims)
    dev = {n: bf16_dev(v) for n, v in x.items()}
    o, os_ = full(*dev["q"].shape), full(*dev["qs"].shape)
    ws = full(max(256, gq.gqe_window_workspace_size(dc, gq.GQE_OP_ATTN_DECODE_WINDOW, L, 50, 2)) // 4,
              dtype=torch.float32)
    gq.gqe_attn_decode_window(dc, dev["q"], dev["qs"], dev["Kc"], dev["Vc"], L, i32([0, L + 9, 70]), 50, 2, o, os_, ws)
    torch.cuda.synchronize()
    assert gq.gqe_device_error() == 0x302
    assert not o[0].any() and not os_[0].any()
    (ro, rs), (bo, bs) = ow.attn_decode_window(x["q"], x["qs"], x["Kc"], x["Vc"], [1, L, 70], dims, 50, 2)
    close(o[1:], ro[1:], bo[1:], "o_routed")
    close(os_[1:], rs[1:], bs[1:], "o_sh")


# ----------------------------------------------------------------------------
# commit

def _commit_case(B, G, T, L, d, seed):
    rng = np.random.default_rng(seed)
    Kt, Vt = rng.integers(0, 1 << 16, (2, B, G, T, d)).astype(np.uint16)
    Kc, Vc = rng.integers(0, 1 << 16, (2, B, G, L, d)).astype(np.uint16)
    return rng, Kt, Vt, Kc, Vc


def _bits(t):
    return t.view(torch.int16).cpu().numpy().view(np.uint16)


@pytest.mark.parametrize("B,G,T,L,d,in_place", [(1, 1, 1, 1, 64, True), (3, 2, 8, 50, 64, False), (5, 3, 128, 300, 128, True),
                                                (70, 8, 5, 33, 64, True)])
def test_commit(B, G, T, L, d, in_place):
    rng, Kt, Vt, Kc, Vc = _commit_case(B, G, T, L, d, 29)
    acc = rng.integers(0, min(T, L) + 1, B)
    acc[0] = min(T, L)
    lens = np.array([int(rng.integers(0, L - a + 1)) for a in acc])
    path = np.full((B, T), 1 << 30, dtype=np.int32)      # past n_accept: not used
    for b in range(B):
        path[b, :acc[b]] = rng.integers(0, T, acc[b])    # the same token may come twice
    dims = gq.make_dims(D(B=B, T=T, G=G, d=d))
    dKc, dVc, dl = bf16_dev(Kc), bf16_dev(Vc), i32(lens)
    nl = dl if in_place else i32(np.full(B, -7))
    gq.gqe_cache_commit(dims, bf16_dev(Kt), bf16_dev(Vt), i32(path), i32(acc), dKc, dVc, L, dl, nl)
    rK, rV, rn = ow.cache_commit(Kt, Vt, path, acc, Kc, Vc, lens)
    np.testing.assert_array_equal(nl.cpu().numpy(), rn)
    np.testing.assert_array_equal(_bits(dKc), rK)
    np.testing.assert_array_equal(_bits(dVc), rV)
    if not in_place:
        np.testing.assert_array_equal(dl.cpu().numpy(), lens)


def test_commit_out_of_range_is_flagged_and_contained():
    B, G, T, L, d = 5, 2, 6, 20, 64
    _, Kt, Vt, Kc, Vc = _commit_case(B, G, T, L, d, 31)
    path = np.tile(np.arange(T, dtype=np.int32), (B, 1))
    path[2, 1], path[2, 3] = -1, T
    lens, acc = [L - 2, L + 5, 3, -4, 7], [5, 1, 5, 2, 99]
    dKc, dVc, dl = bf16_dev(Kc), bf16_dev(Vc), i32(lens)
    gq.gqe_cache_commit(gq.make_dims(D(B=B, T=T, G=G)), bf16_dev(Kt), bf16_dev(Vt), i32(path), i32(acc), dKc, dVc, L, dl, dl)
    torch.cuda.synchronize()
    assert gq.gqe_device_error() == 0x305
    assert dl.tolist() == [L, L, 8, 2, 7 + T]
    rK, rV, _ = ow.cache_commit(Kt, Vt, np.where((path >= 0) & (path < T), path, 0), [2, 0, 5, 2, T], Kc, Vc,
                                np.array([L - 2, L, 3, 0, 7]))
    for r, c in ((rK, Kc), (rV, Vc)):
        r[2][:, [4, 6]] = c[2][:, [4, 6]]
    np.testing.assert_array_equal(_bits(dKc), rK)
    np.testing.assert_array_equal(_bits(dVc), rV)


# ----------------------------------------------------------------------------
# streams, graphs, workspaces

def test_index_tensors_of_the_wrong_size_are_refused():
    """Lengths, parents and paths of another size than the call reads raise
    before anything is launched."""
    B, G, T, L, d = 2, 1, 4, 32, 64
    dims = gq.make_dims(D(B=B, T=T, G=G))
    rows = torch.zeros(B, G, T, d, dtype=torch.bfloat16, device="cuda")
    cache = torch.zeros(B, G, L, d, dtype=torch.bfloat16, device="cuda")
    n = lambda *shape: torch.zeros(*shape, dtype=torch.int32, device="cuda")  # noqa: E731
    commit = lambda path=n(B, T), acc=n(B), ln=n(B), new=n(B): gq.gqe_cache_commit(  # noqa: E731
        dims, rows, rows, path, acc, cache, cache, L, ln, new)
    commit()
    for bad in (dict(path=n(B, T - 1)), dict(acc=n(B - 1)), dict(ln=n(B + 1)), dict(new=n(1))):
        with pytest.raises(ValueError, match="entries"):
            commit(**bad)
    o, os_ = torch.empty_like(rows), torch.empty(B, T, d, dtype=torch.bfloat16, device="cuda")
    tree = lambda par=n(B, T) - 1, tl=None, ln=n(B): gq.gqe_attn_tree(  # noqa: E731
        dims, rows, rows.view(B, T, d), rows, rows, par, tl, cache, cache, L, ln, 0, 0, o, os_)
    tree()
    for bad in (dict(par=n(B, T + 1)), dict(tl=n(1)), dict(ln=n(B, 2))):
        with pytest.raises(ValueError, match="entries"):
            tree(**bad)
    assert gq.gqe_device_error() == 0


def test_calls_run_on_the_stream_they_are_given():
    dims, L, lens, tlens, window, sinks, chain = TREE["window"]
    x = _cache_inputs(dims, L, 37)
    parent = random_parents(dims.B, dims.T, 37)
    _, o, os_ = _run_tree(dims, L, lens, tlens, parent, x, window, sinks)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        _, o2, os2 = _run_tree(dims, L, lens, tlens, parent, x, window, sinks)
    s.synchronize()
    assert torch.equal(o, o2) and torch.equal(os_, os2)


def test_tree_and_commit_replayed_from_one_graph():
    """Lengths, trees and paths are read on the device: a captured step follows them."""
    dims, L = D(T=8, B=2), 400
    x = _cache_inputs(dims, L, 41)
    dc = gq.make_dims(dims)
    dev = {n: bf16_dev(v) for n, v in x.items()}
    o, os_ = full(*dev["q"].shape), full(*dev["qs"].shape)
    ws = full(max(256, gq.gqe_window_workspace_size(dc, gq.GQE_OP_ATTN_TREE, L, 64, 2)) // 4, dtype=torch.float32)
    par, tl, ln = i32(random_parents(2, 8, 1)), i32([8, 8]), i32([100, 0])
    path, acc = i32(np.tile(np.arange(8), (2, 1))), i32([0, 0])

    def step():
        gq.gqe_attn_tree(dc, dev["q"], dev["qs"], dev["K"], dev["V"], par, tl, dev["Kc"], dev["Vc"], L, ln, 64, 2, o, os_,
                         ws)
        gq.gqe_cache_commit(dc, dev["K"], dev["V"], path, acc, dev["Kc"], dev["Vc"], L, ln, ln)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    Kc, Vc, lens = x["Kc"], x["Vc"], np.array([100, 0])
    for it in range(3):
        parent = random_parents(2, 8, 50 + it)
        par.copy_(i32(parent)), tl.copy_(i32([8, 6 - it])), acc.copy_(i32([3, it]))
        g.replay()
        (ro, rs), (bo, bs) = ow.attn_tree(x["q"], x["qs"], x["K"], x["V"], parent, [8, 6 - it], Kc, Vc, lens, dims, 64, 2)
        close(o, ro, bo, f"replay {it}")
        close(os_, rs, bs, f"replay {it}")
        Kc, Vc, lens = ow.cache_commit(x["K"], x["V"], np.tile(np.arange(8), (2, 1)), [3, it], Kc, Vc, lens)
        assert ln.tolist() == list(lens)
    np.testing.assert_array_equal(_bits(dev["Kc"]), Kc)


def test_a_long_cache_past_two_to_the_31_elements():
    """Cache offsets past 2^31 elements: the last sequence of a 4.5 GB cache."""
    B, G, L, d = 1, 34, 1 << 20, 64
    dims = D(B=B, T=2, G=G, E=1, k=1, n_shared=0)
    gen = torch.Generator(device="cuda").manual_seed(3)
    Kc = torch.empty((B, G, L, d), dtype=BF16, device="cuda").normal_(generator=gen)
    Vc = torch.empty_like(Kc).normal_(generator=gen)
    x = _prefill_inputs(dims, 43)
    dev = {n: None if v is None else bf16_dev(v) for n, v in x.items()}
    dc = gq.make_dims(dims)
    o = full(*dev["q"].shape)
    lens, win = [L - 5], 400
    ws = full(max(256, gq.gqe_window_workspace_size(dc, gq.GQE_OP_ATTN_TREE, L, win, 3)) // 4, dtype=torch.float32)
    par = np.array([[-1, 0]], dtype=np.int32)
    gq.gqe_attn_tree(dc, dev["q"], None, dev["K"], dev["V"], i32(par), None, Kc, Vc, L, i32(lens), win, 3, o, None, ws)
    gq.gqe_cache_commit(dc, dev["K"], dev["V"], i32(par * 0 + [[1, 0]]), i32([2]), Kc, Vc, L, i32(lens), i32([0]))
    torch.cuda.synchronize()
    keep = torch.cat([torch.arange(3), torch.arange(L - 5 - win, L - 5)]).cuda()      # what the first token sees, moved
    sub = dims.replace(G=1)
    lo = Kc[:, -1:, keep].double().cpu().numpy(), Vc[:, -1:, keep].double().cpu().numpy()
    n = keep.numel()
    (ro, _), (bo, _) = ow.attn_tree(x["q"][:, -1:], None, x["K"][:, -1:], x["V"][:, -1:], par, [2], lo[0], lo[1], [n], sub,
                                    win, 3)
    close(o[:, -1:], ro, bo, "last group")
    assert torch.equal(Kc[0, -1, L - 5], dev["K"][0, -1, 1]) and torch.equal(Vc[0, -1, L - 4], dev["V"][0, -1, 0])
