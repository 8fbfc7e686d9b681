"""Plain fp64 CPU oracle of the windowed, tree and cache operators.

TEST INFRASTRUCTURE ONLY, like the layer oracle beside it, and it shares no
code with the CUDA library.  GQE's pages describe full causal attention; these
operators run the same attention over a smaller set of keys:

  a query at position t sees key p when p <= t and
  (p > t - window or p < sinks)                      (window 0: p <= t),

and a drafted token sits at the cache's length plus its depth in its tree and
sees of the drafted tokens its ancestors and itself.  Every function takes an
explicit visibility matrix [rows, keys] and is the attention equation ("GQE"
study note §1-1) over the keys that are True; a row that sees nothing is 0.

Pinned by tests/test_oracle_window_pins.py: scalar loops, the causal oracle
(window 0), torch autograd in fp64, central finite differences, and a chain of
drafted tokens against the prefill's rows.
"""
from __future__ import annotations

import numpy as np

from .gqe_oracle import f64, attention_scale

U_BF16 = 2.0 ** -8      # half a step of bf16, relative
U_FP32 = 2.0 ** -24


def sees(t, p, window, sinks):
    """Visibility of positions p [..] to query positions t (broadcast)."""
    t, p = np.asarray(t), np.asarray(p)
    ok = p <= t
    if window:
        ok = ok & ((p > t - window) | (p < sinks))
    return ok


def masked_attention(q, vis, K, V, scale):
    """o_r = sum_{j: vis_rj} softmax_j(q_r . K_j * scale) V_j, and the natural
    log-sum-exp of the visible scaled scores (-inf and o = 0 for an empty row)."""
    q, K, V = f64(q), f64(K), f64(V)
    o, lse = np.zeros((q.shape[0], V.shape[1])), np.full(q.shape[0], -np.inf)
    used = vis.any(0)                      # keys nobody sees may hold anything
    K, V, vis = K[used], V[used], vis[:, used]
    s = np.where(vis, q @ K.T * scale, -np.inf)
    rows = vis.any(1)
    m = s[rows].max(1, keepdims=True)
    z = np.exp(s[rows] - m)
    den = z.sum(1, keepdims=True)
    o[rows] = z @ V / den
    lse[rows] = (m + np.log(den))[:, 0]
    return o, lse


def masked_attention_error_bound(q, vis, K, V, scale):
    """Worst-case error of masked_attention's o computed with bf16 operands P
    and V, fp32 sums and approximate exponentials, before the final rounding.

    The exponent errs by e_rj = scale d 2^-24 sum|q||K| (a sum of d products
    in fp32) and the exponential by 1e-4 relative (the kernels' polynomial
    2^x is within 7.5e-5, the hardware's and the rescalings' a few 2^-22).
    P is rounded to bf16 for the numerator alone, so with w the softmax and
    g = L 2^-24 (fp32 sums over L keys):
      err o <= sum_j w_j (u + e_j + 1e-4 + g) |V_j| + |o| (sum_j w_j (e_j + 1e-4) + g).
    """
    q, K, V = f64(q), f64(K), f64(V)
    used = vis.any(0)
    K, V, vis = K[used], V[used], vis[:, used]
    out = np.zeros((q.shape[0], V.shape[1]))
    if not used.any():
        return out
    s = np.where(vis, q @ K.T * scale, -np.inf)
    rows = vis.any(1)
    z = np.exp(s[rows] - s[rows].max(1, keepdims=True))
    w = z / z.sum(1, keepdims=True)
    e = scale * q.shape[1] * U_FP32 * (np.abs(q[rows]) @ np.abs(K).T) + 1e-4
    g = K.shape[0] * U_FP32
    out[rows] = (w * (U_BF16 + e + g)) @ np.abs(V) + np.abs(w @ V) * ((w * e).sum(1, keepdims=True) + g)
    return out


FEW_KEYS = 8        # rows that see at most this many keys have their Delta from P and dP (see below)


def masked_attention_bwd(q, vis, K, V, dO, scale, lse):
    """Gradients of masked_attention: with P = exp(S - lse) on visible keys,
    dP = dO V^T, Delta = sum_j P_j dP_j, dS = P (dP - Delta): dV = P^T dO,
    dq = scale dS K, dK = scale dS^T q.

    And the worst-case errors of the three computed as the tensor cores do it
    (P and dS rounded to bf16, fp32 sums; see causal_attention_bwd_error_bound,
    plus 1e-4 for the exponential).  Delta may come from dO . O with O rounded
    to bf16, 2^-8 sum|dO||O| off, for rows that see more than FEW_KEYS keys.
    Returns (dq, dK, dV), (bound_dq, bound_dK, bound_dV)."""
    q, K, V, dO = f64(q), f64(K), f64(V), f64(dO)
    P = np.where(vis, np.exp(np.where(vis, q @ K.T * scale, -np.inf) - np.asarray(lse)[:, None]), 0.0)
    dP = dO @ V.T
    delta = (P * dP).sum(1, keepdims=True)
    dS = P * (dP - delta)
    d, L, R = q.shape[1], K.shape[0], q.shape[0]
    gd, gL, gR = d * U_FP32, L * U_FP32, R * U_FP32
    aq, aK, aV, aO = np.abs(q), np.abs(K), np.abs(V), np.abs(dO)
    eE = scale * gd * (aq @ aK.T) + 1e-4
    eP = P * eE
    adOO = (aO * np.abs(P @ V)).sum(1, keepdims=True)
    few = vis.sum(1, keepdims=True) <= FEW_KEYS
    e_delta = np.where(few, (P * eE * np.abs(dP)).sum(1, keepdims=True), U_BF16 * adOO)
    edS = scale * (np.abs(dP - delta) * eP + P * (e_delta + gd * (aO @ aV.T + adOO)))
    aS = np.abs(scale * dS)
    bounds = (((U_BF16 + gL) * aS + edS) @ aK, ((U_BF16 + gR) * aS + edS).T @ aq,
              ((U_BF16 + gR) * P + eP).T @ aO)
    return (scale * (dS @ K), scale * (dS.T @ q), P.T @ dO), bounds


# ----------------------------------------------------------------------------
# the calls

def _row_sets(dims, T, q_routed, q_sh):
    """(b, g, tokens of the rows, rows) of every routed group and shared head."""
    for b in range(dims.B):
        for g in range(dims.G):
            yield b, g, False, np.repeat(np.arange(T), dims.k), np.asarray(q_routed[b, g]).reshape(T * dims.k, dims.d)
        if dims.n_shared:
            yield b, dims.sg, True, np.arange(T), np.asarray(q_sh[b])


def attn_prefill_window(q_routed, q_sh, K, V, dims, window, sinks):
    """(o_routed, o_sh, lse), (bound_routed, bound_sh); lse in the library's
    layout: routed rows, then shared rows."""
    B, T, G, k, d = dims.B, dims.T, dims.G, dims.k, dims.d
    sc = attention_scale(dims)
    o, e = np.empty((2, B, G, T, k, d))
    os_, es = np.empty((2, B, T, d))
    lse, lse_s = np.empty((B, G, T * k)), np.empty((B, T))
    for b, g, sh, tok, rows in _row_sets(dims, T, q_routed, q_sh):
        vis = sees(tok[:, None], np.arange(T)[None], window, sinks)
        a, l = masked_attention(rows, vis, K[b, g], V[b, g], sc)
        bd = masked_attention_error_bound(rows, vis, K[b, g], V[b, g], sc)
        if sh:
            os_[b], es[b], lse_s[b] = a, bd, l
        else:
            o[b, g], e[b, g], lse[b, g] = a.reshape(T, k, d), bd.reshape(T, k, d), l
    flat = np.concatenate([lse.reshape(-1)] + ([lse_s.reshape(-1)] if dims.n_shared else []))
    return (o, os_ if dims.n_shared else None, flat), (e, es if dims.n_shared else None)


def attn_prefill_window_bwd(q_routed, q_sh, K, V, window, sinks, lse, do_routed, do_sh, dims):
    """(dq_routed, dq_sh, dK, dV) and their error bounds, from the forward's lse
    (library layout)."""
    B, T, G, k, d = dims.B, dims.T, dims.G, dims.k, dims.d
    sc = attention_scale(dims)
    out = [np.zeros((B, G, T, k, d)), np.zeros((B, T, d)), np.zeros((B, G, T, d)), np.zeros((B, G, T, d))]
    bnd = [np.zeros_like(x) for x in out]
    for b, g, sh, tok, rows in _row_sets(dims, T, q_routed, q_sh):
        vis = sees(tok[:, None], np.arange(T)[None], window, sinks)
        dO = do_sh[b] if sh else np.asarray(do_routed[b, g]).reshape(T * k, d)
        l0 = B * G * T * k + b * T if sh else (b * G + g) * T * k
        grads, bounds = masked_attention_bwd(rows, vis, K[b, g], V[b, g], dO, sc, lse[l0:l0 + len(tok)])
        for dst, (dq, dK, dV) in ((out, grads), (bnd, bounds)):
            if sh:
                dst[1][b] = dq
            else:
                dst[0][b, g] = dq.reshape(T, k, d)
            dst[2][b, g] += dK
            dst[3][b, g] += dV
    if not dims.n_shared:
        out[1] = bnd[1] = None
    return out, bnd


def tree_lines(parent):
    """For each drafted token the list of the tokens above it and itself, root first."""
    lines = []
    for i, p in enumerate(parent):
        lines.append((list(lines[p]) if p >= 0 else []) + [i])
    return lines


def attn_tree(q_routed, q_sh, Kt, Vt, parent, tree_len, Kc, Vc, cache_len, dims, window, sinks):
    """(o_routed, o_sh), (bounds): drafted tokens over the cache and their tree;
    rows past tree_len are 0."""
    B, T, G, k, d = dims.B, dims.T, dims.G, dims.k, dims.d
    sc = attention_scale(dims)
    o, e = np.zeros((2, B, G, T, k, d))
    os_, es = np.zeros((2, B, T, d))
    for b, g, sh, tok, rows in _row_sets(dims, T, q_routed, q_sh):
        n, m = int(cache_len[b]), int(tree_len[b])
        lines = tree_lines(parent[b][:m])
        pos = np.array([n + len(x) - 1 for x in lines], dtype=np.int64)
        up = np.zeros((m, m), dtype=bool)
        for i, x in enumerate(lines):
            up[i, x] = True
        vis = np.concatenate([sees(pos[:, None], np.arange(n)[None], window, sinks),
                              up & sees(pos[:, None], pos[None], window, sinks)], 1)
        live = tok < m
        Kb = np.concatenate([f64(Kc[b, g][:n]), f64(Kt[b, g][:m])])
        Vb = np.concatenate([f64(Vc[b, g][:n]), f64(Vt[b, g][:m])])
        for dst_r, dst_s, fn in ((o, os_, lambda *a: masked_attention(*a)[0]), (e, es, masked_attention_error_bound)):
            full = np.zeros((len(tok), d))
            if m:
                full[live] = fn(rows[live], vis[tok[live]], Kb, Vb, sc)
            if sh:
                dst_s[b] = full
            else:
                dst_r[b, g] = full.reshape(T, k, d)
    return (o, os_ if dims.n_shared else None), (e, es if dims.n_shared else None)


def attn_decode_window(q_routed, q_sh, Kc, Vc, cache_len, dims, window, sinks):
    """(o_routed, o_sh), (bounds) of one new token at position cache_len - 1;
    q_routed [B, G, 1, k, d], q_sh [B, 1, d]."""
    B, G, k, d = dims.B, dims.G, dims.k, dims.d
    sc = attention_scale(dims)
    o, e = np.zeros((2, B, G, 1, k, d))
    os_, es = np.zeros((2, B, 1, d))
    for b, g, sh, tok, rows in _row_sets(dims, 1, q_routed, q_sh):
        n = int(cache_len[b])
        vis = np.broadcast_to(sees(n - 1, np.arange(n), window, sinks)[None], (len(tok), n))
        a = masked_attention(rows, vis, Kc[b, g][:n], Vc[b, g][:n], sc)[0]
        bd = masked_attention_error_bound(rows, vis, Kc[b, g][:n], Vc[b, g][:n], sc)
        if sh:
            os_[b], es[b] = a, bd
        else:
            o[b, g, 0], e[b, g, 0] = a, bd
    return (o, os_ if dims.n_shared else None), (e, es if dims.n_shared else None)


def cache_commit(Kt, Vt, path, n_accept, Kc, Vc, cache_len):
    """The caches after the accepted rows moved in, and the new lengths (any dtype; nothing is computed)."""
    Kc, Vc = Kc.copy(), Vc.copy()
    new_len = np.array(cache_len).copy()
    for b in range(Kc.shape[0]):
        for i in range(int(n_accept[b])):
            Kc[b, :, cache_len[b] + i] = Kt[b, :, path[b][i]]
            Vc[b, :, cache_len[b] + i] = Vt[b, :, path[b][i]]
        new_len[b] += n_accept[b]
    return Kc, Vc, new_len
