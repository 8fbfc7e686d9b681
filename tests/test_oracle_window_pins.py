"""Pins of the windowed, tree and cache oracle (CPU)."""
import math

import numpy as np
import pytest
import torch

import gqe_inputs as gi
import oracle as orc
from oracle import gqe_window as ow


def D(**kw):
    base = dict(B=1, T=20, D=64, G=2, E=2, k=1, d=64)
    base.update(kw)
    return gi.GQEDims(**base)


def _inputs(dims, seed=3, T=None):
    T = dims.T if T is None else T
    return (gi.normal_bf16(seed, "q", (dims.B, dims.G, T, dims.k, dims.d)), gi.normal_bf16(seed, "qsh", (dims.B, T, dims.d)),
            gi.normal_bf16(seed, "K", (dims.B, dims.G, T, dims.d)), gi.normal_bf16(seed, "V", (dims.B, dims.G, T, dims.d)))


@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 0), (3, 2), (5, 9), (19, 1), (20, 0), (100, 0), (0, 4)])
def test_window_matches_scalar_loops(window, sinks):
    dims = D(G=1, k=2, d=64, n_shared=0)
    q, _, K, V = _inputs(dims)
    (o, _, lse), _ = ow.attn_prefill_window(q, None, K, V, dims, window, sinks)
    qf, Kf, Vf = orc.f64(q), orc.f64(K), orc.f64(V)
    for t in range(dims.T):
        keys = [p for p in range(t + 1) if window == 0 or t - p < window or p < sinks]
        for j in range(2):
            s = [sum(qf[0, 0, t, j, c] * Kf[0, 0, p, c] for c in range(64)) / 8.0 for p in keys]
            z = [math.exp(x) for x in s]
            ref = sum(w * Vf[0, 0, p] for w, p in zip(z, keys)) / sum(z)
            np.testing.assert_allclose(o[0, 0, t, j], ref, rtol=1e-11, atol=1e-12)
            np.testing.assert_allclose(lse[t * 2 + j], math.log(sum(z)), rtol=1e-11)


@pytest.mark.parametrize("window", [0, 20, 64])
def test_no_window_is_the_causal_oracle(window):
    dims = D(B=2, k=2, sg=1)
    q, qs, K, V = _inputs(dims)
    (o, os_, lse), _ = ow.attn_prefill_window(q, qs, K, V, dims, window, 3)
    ro, rs, rl, rls = orc.attn_prefill(q, qs, K, V, dims)
    np.testing.assert_allclose(o, ro, rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(os_, rs, rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(lse, np.concatenate([rl.reshape(-1), rls.reshape(-1)]), rtol=1e-12)


def test_window_of_one_token_returns_its_value_row():
    dims = D(k=1)
    q, qs, K, V = _inputs(dims)
    (o, os_, _), _ = ow.attn_prefill_window(q, qs, K, V, dims, 1, 0)
    np.testing.assert_allclose(o[:, :, :, 0], orc.f64(V), rtol=1e-13)
    np.testing.assert_allclose(os_, orc.f64(V)[:, 0], rtol=1e-13)


@pytest.mark.parametrize("window,sinks", [(1, 0), (4, 0), (4, 3), (7, 1), (0, 0)])
def test_backward_matches_autograd(window, sinks):
    dims = D(B=2, T=17, G=2, k=2, sg=1)
    q, qs, K, V = _inputs(dims)
    do = gi.normal_bf16(3, "do", q.shape)
    dos = gi.normal_bf16(3, "dosh", qs.shape)
    (o, os_, lse), _ = ow.attn_prefill_window(q, qs, K, V, dims, window, sinks)
    (dq, dqs, dK, dV), _ = ow.attn_prefill_window_bwd(q, qs, K, V, window, sinks, lse, do, dos, dims)
    tq, tqs, tK, tV = (torch.tensor(orc.f64(x), requires_grad=True) for x in (q, qs, K, V))
    t = torch.arange(17)
    hide = t[None] > t[:, None]
    if window:
        hide = hide | ((t[:, None] - t[None] >= window) & (t[None] >= sinks))
    x = torch.einsum("bgtkd,bgpd->bgktp", tq, tK) / 8.0
    y = torch.einsum("bgktp,bgpd->bgtkd", x.masked_fill(hide, -math.inf).softmax(-1), tV)
    xs = torch.einsum("btd,bpd->btp", tqs, tK[:, 1]) / 8.0
    ys = xs.masked_fill(hide, -math.inf).softmax(-1) @ tV[:, 1]
    ((y * torch.tensor(orc.f64(do))).sum() + (ys * torch.tensor(orc.f64(dos))).sum()).backward()
    for got, ref in ((dq, tq), (dqs, tqs), (dK, tK), (dV, tV)):
        np.testing.assert_allclose(got, ref.grad.numpy(), rtol=1e-10, atol=1e-12)


def test_backward_matches_finite_differences():
    """Along random directions of q, K and V, in fp64."""
    dims = D(T=15, G=1, k=1, n_shared=0)
    rng = np.random.default_rng(5)
    q, K, V, dO = (rng.standard_normal((15, 64)) for _ in range(4))
    vis = ow.sees(np.arange(15)[:, None], np.arange(15)[None], 4, 2)
    f = lambda a, b, c: float((ow.masked_attention(a, vis, b, c, 0.125)[0] * dO).sum())
    o, lse = ow.masked_attention(q, vis, K, V, 0.125)
    grads, _ = ow.masked_attention_bwd(q, vis, K, V, dO, 0.125, lse)
    h = 1e-5
    for i, g in enumerate(grads):
        u = rng.standard_normal((15, 64))
        hi, lo = [q, K, V], [q, K, V]
        hi[i], lo[i] = hi[i] + h * u, lo[i] - h * u
        np.testing.assert_allclose((f(*hi) - f(*lo)) / (2 * h), (g * u).sum(), rtol=1e-7, atol=1e-8)


@pytest.mark.parametrize("window,sinks", [(0, 0), (4, 0), (4, 3), (11, 1), (2, 0)])
def test_a_chain_of_drafted_tokens_equals_the_prefill_rows(window, sinks):
    dims = D(B=2, T=20, G=2, k=2, sg=1)
    q, qs, K, V = _inputs(dims)
    (ro, rs, _), _ = ow.attn_prefill_window(q, qs, K, V, dims, window, sinks)
    n = 13
    sub = dims.replace(T=20 - n)
    par = np.tile(np.arange(20 - n) - 1, (2, 1))
    (o, os_), _ = ow.attn_tree(q[:, :, n:], qs[:, n:], K[:, :, n:], V[:, :, n:], par, [20 - n] * 2, K, V, [n] * 2,
                               sub, window, sinks)
    np.testing.assert_allclose(o, ro[:, :, n:], rtol=1e-11, atol=1e-12)
    np.testing.assert_allclose(os_, rs[:, n:], rtol=1e-11, atol=1e-12)
    one = dims.replace(T=1)
    (o1, os1), _ = ow.attn_decode_window(q[:, :, n:n + 1], qs[:, n:n + 1], K, V, [n + 1] * 2, one, window, sinks)
    np.testing.assert_allclose(o1, ro[:, :, n:n + 1], rtol=1e-11, atol=1e-12)
    np.testing.assert_allclose(os1, rs[:, n:n + 1], rtol=1e-11, atol=1e-12)


def test_siblings_do_not_see_each_other():
    """Each leaf of a two-branch tree equals the chain that leads to it; dead rows are 0."""
    dims = D(B=1, T=6, G=1, k=1, n_shared=0)
    q, _, Kt, Vt = _inputs(dims, 4)
    Kc, Vc = gi.normal_bf16(4, "Kc", (1, 1, 9, 64)), gi.normal_bf16(4, "Vc", (1, 1, 9, 64))
    parent = np.array([[-1, 0, 0, 2, -1, 4]])
    (o, _), _ = ow.attn_tree(q, None, Kt, Vt, parent, [5], Kc, Vc, [9], dims, 0, 0)
    assert not o[0, 0, 5].any()
    for leaf, line in ((1, [0, 1]), (3, [0, 2, 3]), (4, [4])):
        sub = dims.replace(T=len(line))
        (c, _), _ = ow.attn_tree(q[:, :, line], None, Kt[:, :, line], Vt[:, :, line],
                                 np.arange(len(line))[None] - 1, [len(line)], Kc, Vc, [9], sub, 0, 0)
        np.testing.assert_allclose(o[0, 0, leaf], c[0, 0, -1], rtol=1e-12)


def test_commit_moves_the_path_and_nothing_else():
    rng = np.random.default_rng(0)
    Kt, Vt = rng.integers(0, 1 << 16, (2, 2, 3, 5, 8)).astype(np.uint16)
    Kc, Vc = rng.integers(0, 1 << 16, (2, 2, 3, 9, 8)).astype(np.uint16)
    path = np.array([[0, 2, 4, -1, -1], [3, -1, -1, -1, -1]])
    K2, V2, n = ow.cache_commit(Kt, Vt, path, [3, 0], Kc, Vc, np.array([4, 9]))
    assert list(n) == [7, 9]
    np.testing.assert_array_equal(K2[0][:, 4:7], Kt[0][:, [0, 2, 4]])
    np.testing.assert_array_equal(np.delete(V2[0], [4, 5, 6], 1), np.delete(Vc[0], [4, 5, 6], 1))
    np.testing.assert_array_equal(K2[1], Kc[1])
