"""The windowed GQE layer and its serving path end to end (GPU): prefill,
training step, decode steps, drafted trees and commits on one cache, against
the fp64 oracle chain with the window's attention in it."""
from unittest import mock

import numpy as np
import pytest
import torch

import gqe_inputs as gi
import oracle as orc
from oracle import gqe_backward as ob
from oracle import gqe_oracle as oo
from oracle import gqe_window as ow
from helpers import bf16_dev, to_f64

pytestmark = pytest.mark.gpu

gq = pytest.importorskip("moe_gqa_query_b200")

# Norm-wise relative error of a layer's outputs through every bf16 intermediate
# (q, K, V, o, h, y: six roundings of 2^-8 relative at most, each norm-wise at
# most that): 6 * 2^-8 = 2.4e-2; and of its gradients, as for the layer without
# a window (2e-2, 5e-2 for the router's).
Y_REL = 2.4e-2
GRAD_REL, ROUTER_REL = 2e-2, 5e-2


@pytest.fixture(autouse=True)
def _cuda_and_error_word():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    yield
    torch.cuda.synchronize()
    assert gq.gqe_device_error() == 0


def cfg(dims, window, sinks):
    return gq.GQEConfig(B=dims.B, T=dims.T, D=dims.D, G=dims.G, E=dims.E, k=dims.k, d=dims.d, n_shared=dims.n_shared,
                        sg=dims.sg, window=window, sinks=sinks)


def weights(dims, seed):
    """Layer weights with K projections scaled up, so that attention is not close to uniform."""
    Wt = gi.layer_weights(dims, seed)
    Wt["Wk"] = gi.f32_to_bf16_bits(gi.bf16_bits_to_f32(Wt["Wk"]) * 8)
    return Wt


def dev_weights(Wt):
    return {k: torch.from_numpy(v.view(np.int16)) for k, v in Wt.items()}


def windowed(window, sinks):
    """The oracle's layer functions with the window's attention in place of the causal one."""
    def fwd(q, qs, K, V, dims, chunk=2048):
        (o, os_, lse), _ = ow.attn_prefill_window(q, qs, K, V, dims, window, sinks)
        return o, os_, None, None

    def bwd(q, qs, K, V, do, dos, dims, *a):
        (o, os_, lse), _ = ow.attn_prefill_window(q, qs, K, V, dims, window, sinks)
        return ow.attn_prefill_window_bwd(q, qs, K, V, window, sinks, lse, do, dos, dims)[0]
    stack = mock.patch.multiple(ob, attn_prefill=fwd, attn_prefill_bwd=bwd)
    stack2 = mock.patch.object(oo, "attn_prefill", fwd)
    return stack, stack2


def rel(got, ref):
    return np.linalg.norm(got - ref) / np.linalg.norm(ref)


LAYERS = {
    "k2_sinks": (gi.GQEDims(B=2, T=300, D=256, G=3, E=4, k=2, d=64, sg=1), 70, 3),
    "k1_no_shared": (gi.GQEDims(B=1, T=257, D=128, G=2, E=2, k=1, d=64, n_shared=0), 128, 0),
    "d128": (gi.GQEDims(B=1, T=300, D=256, G=2, E=4, k=4, d=128), 33, 40),
}


@pytest.mark.parametrize("case", list(LAYERS))
def test_windowed_layer_forward_and_training_step(case):
    dims, window, sinks = LAYERS[case]
    x, Wt = gi.layer_input(dims, 4), weights(dims, 4)
    dy = gi.normal_bf16(4, "dy", (dims.B, dims.T, dims.D))
    layer = gq.GQELayer(cfg(dims, window, sinks), dev_weights(Wt))
    tx = bf16_dev(x)
    y, saved = layer.forward(tx, keep=True)
    y = to_f64(y).reshape(dims.N, -1)
    g = layer.backward(tx, bf16_dev(dy), saved)
    torch.cuda.synchronize()
    a, b = windowed(window, sinks)
    with a, b:
        ref = orc.gqe_forward(x, Wt, dims)
        gref = ob.gqe_backward(x, Wt, dims, dy)
    assert np.array_equal(saved["idx"].cpu().numpy(), ref["router"]["idx"])
    assert rel(y, ref["y"]) <= Y_REL
    assert rel(y, orc.gqe_forward(x, Wt, dims)["y"]) > 4 * Y_REL        # the window matters here
    for name in ("dx", "dWr", "dWq", "dWk", "dWv", "dWo") + (("dWsh",) if dims.n_shared else ()):
        err = rel(to_f64(g[name]).reshape(gref[name].shape), gref[name])
        assert err <= (ROUTER_REL if name == "dWr" else GRAD_REL), (name, err)


def test_windowed_forward_entry_points_agree():
    dims, window, sinks = LAYERS["k2_sinks"]
    layer = gq.GQELayer(cfg(dims, window, sinks), dev_weights(weights(dims, 5)))
    xs = gi.layer_input(dims, 5)
    x = bf16_dev(xs)
    y = layer.forward(x).clone()
    assert torch.equal(layer.forward_graph(x), y)
    xh = bf16_dev(xs, "cpu").pin_memory()
    yh = torch.empty_like(xh).pin_memory()
    layer.forward_host(xh, yh)
    torch.cuda.synchronize()
    assert torch.equal(yh, y.cpu())
    with pytest.raises(ValueError, match="windowed"):
        layer.forward_host_c(xh, yh)
    with pytest.raises(ValueError):
        gq.GQEConfig(B=1, T=1, D=64, G=1, E=1, k=1, d=64, window=-1)


@pytest.mark.parametrize("window,sinks", [(0, 0), (60, 2)])
def test_prefill_drafts_commits_and_decode_on_one_cache(window, sinks):
    """A serving run.  Each sequence's prompt goes into the cache; a tree drafts
    its true continuation among wrong branches; the true path is committed, then
    a second tree and single decode steps go on.  Every true token's output must
    be the row that one forward over the whole text gives."""
    dims = gi.GQEDims(B=3, T=200, D=256, G=2, E=4, k=2, d=64, sg=1)
    Wt = weights(dims, 6)
    layer = gq.GQELayer(cfg(dims, window, sinks), dev_weights(Wt))
    text = bf16_dev(gi.layer_input(dims, 6))                          # [B, 200, D]
    noise = bf16_dev(gi.normal_bf16(7, "x", (dims.B, 200, dims.D)))
    y, saved = layer.forward(text, keep=True)
    y, K, V = to_f64(y), saved["K"].clone(), saved["V"].clone()
    L_max = 256
    prompt = [150, 97, 0]
    Kc = torch.full((dims.B, dims.G, L_max, dims.d), float("nan"), dtype=torch.bfloat16, device="cuda")
    Vc = Kc.clone()
    for b, n in enumerate(prompt):
        Kc[b, :, :n], Vc[b, :, :n] = K[b, :, :n], V[b, :, :n]
    lens = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    at = np.array(prompt)
    rng = np.random.default_rng(3)

    def check(got, b, pos, what):
        err = rel(got, y[b, pos])
        assert err <= Y_REL, (what, b, pos, err)

    for T, tlen in ((24, [24, 20, 7]), (9, [9, 1, 9])):
        parent = np.full((dims.B, T), -1, dtype=np.int32)
        path = np.full((dims.B, T), -1, dtype=np.int32)
        acc = np.zeros(dims.B, dtype=np.int32)
        xd = noise[:, :T].clone()
        true = {}
        for b in range(dims.B):
            line = []                              # drafted tokens that carry the true text
            for i in range(T):
                if rng.random() < 0.5 and i < tlen[b]:
                    parent[b, i] = line[-1] if line else -1
                    xd[b, i] = text[b, at[b] + len(line)]
                    line.append(i)
                elif i:
                    parent[b, i] = rng.integers(-1, i)
            true[b] = line
            acc[b] = len(line)
            path[b, :len(line)] = line
        yd, draft = layer.decode_tree(xd, torch.from_numpy(parent).cuda(), Kc, Vc, lens,
                                      torch.tensor(tlen, dtype=torch.int32, device="cuda"))
        yd = to_f64(yd)
        for b, line in true.items():
            for depth, i in enumerate(line):
                check(yd[b, i], b, at[b] + depth, "drafted token")
        out = layer.commit(draft, torch.from_numpy(path).cuda(), torch.from_numpy(acc).cuda(), Kc, Vc, lens)
        at = at + acc
        assert out is lens and lens.tolist() == list(at)
    for _ in range(3):
        lens += 1
        yn = to_f64(layer.decode_step(text[torch.arange(dims.B), torch.from_numpy(at)].contiguous(), Kc, Vc, lens))
        for b in range(dims.B):
            check(yn[b], b, at[b], "decode step")
        at = at + 1
    # the committed and appended rows are the prefill's, the rows behind the last sequence untouched
    for b in range(dims.B):
        assert rel(to_f64(Kc[b, :, :at[b]]), to_f64(K[b, :, :at[b]])) <= 2 ** -8
        assert torch.isnan(Kc[b, :, at[b]:]).all() and torch.isnan(Vc[b, :, at[b]:]).all()


def test_two_layers_calls_on_two_streams():
    """Two windowed layers trained and decoded at once on streams of their own
    give what each gives alone."""
    dims, window, sinks = LAYERS["k2_sinks"]
    runs = []
    for seed in (8, 9):
        layer = gq.GQELayer(cfg(dims, window, sinks), dev_weights(weights(dims, seed)))
        x = bf16_dev(gi.layer_input(dims, seed))
        dy = bf16_dev(gi.normal_bf16(seed, "dy", (dims.B, dims.T, dims.D)))

        def step(layer=layer, x=x, dy=dy):
            y, saved = layer.forward(x, stream=torch.cuda.current_stream(), keep=True)
            g = layer.backward(x, dy, saved)
            return y, g["dK"], g["dV"]
        runs.append((step, [t.clone() for t in step()]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in runs]
    outs = []
    for _ in range(3):
        for s, (step, _) in zip(streams, runs):
            with torch.cuda.stream(s):
                outs.append([t.clone() for t in step()])
    torch.cuda.synchronize()
    for i, out in enumerate(outs):
        for got, want in zip(out, runs[i % 2][1]):
            assert torch.equal(got, want)
