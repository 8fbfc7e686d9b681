"""What is measured of the windowed, tree and cache operators: cases, inputs, one pass, work.

Five operators of a GQE attention layer whose context is a sliding window with
a few first tokens that stay visible (sinks), or whose decoding drafts a tree
of tokens:

  prefill  attention of a whole prompt under the window (forward)
  train    the same forward with its backward pass: o and dq, dK, dV
  decode   one new token per sequence over a dense [B, G, L, d] cache, under the window
  tree     a tree of T drafted tokens per sequence over the cache and over itself
  commit   the accepted drafted tokens' K/V rows moved to the end of the cache

Visibility.  A query at position t sees key p when p <= t and (p > t - W or
p < S), W the window (0: unlimited) and S the sinks.  Drafted token i of a
sequence sits at position cache_len + depth(i), sees the cache rows its
position sees, and of the drafted tokens its ancestors and itself under the
same window.  Query rows: k routed rows per token and KV group, and one shared
head per token that reads group sg.
"""
import math

import torch

own = False

BF16 = torch.bfloat16
INF = float("inf")


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # the tiny prefill shape under a window of half its length: a call that is all latency
        dict(name="prefill_tiny", op="prefill", B=1, T=128, G=2, k=1, d=64, sh=1, sg=0, W=64, S=4),
        # one long document through the main layer's heads, 1024-token window
        dict(name="prefill_long", op="prefill", B=1, T=32768, G=8, k=1, d=64, sh=1, sg=0, W=1024, S=4),
        # a training step's attention at the main layer, window a quarter of the context
        dict(name="train_main", op="train", B=8, T=2048, G=8, k=1, d=64, sh=1, sg=0, W=512, S=4),
        # wide groups (4 of 8 experts, d = 128) trained at 8192 tokens
        dict(name="train_wide", op="train", B=2, T=8192, G=4, k=4, d=128, sh=1, sg=0, W=1024, S=16),
        # nothing a multiple of a tile: 1001 tokens, 3 rows a token, window 200, one sink, shared head elsewhere
        dict(name="train_odd", op="train", B=3, T=1001, G=3, k=3, d=64, sh=1, sg=2, W=200, S=1),
        # serving batch of the main layer over 32768-row caches, 4096-token window
        dict(name="decode_main", op="decode", B=64, L=32768, G=8, k=1, d=64, sh=1, sg=0, W=4096, S=4, ragged=False),
        # a small batch of wide groups: five rows share each key, odd lengths, no sinks
        dict(name="decode_wide", op="decode", B=5, L=8191, G=4, k=4, d=128, sh=1, sg=1, W=1000, S=0, ragged=True),
        # one chat being drafted for: 8 drafted tokens over a 4096-row cache
        dict(name="tree_one", op="tree", B=1, T=8, L=4096, G=8, k=1, d=64, sh=1, sg=0, W=0, S=0, ragged=False),
        # a full serving batch with 32-token trees over 32768-row caches
        dict(name="tree_batch", op="tree", B=64, T=32, L=32768, G=8, k=1, d=64, sh=1, sg=0, W=0, S=0, ragged=False),
        # wide groups, 63-token trees (315 rows in one group), window and sinks, ragged lengths
        dict(name="tree_wide", op="tree", B=8, T=63, L=8192, G=4, k=4, d=128, sh=1, sg=0, W=2048, S=4, ragged=True),
        # a step of one chat: up to 5 of 8 drafted tokens kept
        dict(name="commit_one", op="commit", B=1, T=8, A=5, L=4096, G=8, d=64),
        # a full batch after 64-token trees, up to 17 tokens kept, some sequences none
        dict(name="commit_batch", op="commit", B=64, T=64, A=17, L=2048, G=8, d=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _within(case):
    """Fewer tokens where the heads and the lengths drawn would cost more than the listed cases."""
    while work(case)["flops"] > 300e9 and case.get("T", 1) > 1:
        case["T"] = case["T"] * 2 // 3
    return case


def draw(rng):
    op = rng.choice(["prefill", "train", "decode", "tree", "commit"])
    d = rng.choice([64, 64, 128])
    G = rng.choice([1, 2, 3, 4, 8])
    k = rng.choice([1, 1, 2, 3, 4])
    sh = rng.choice([0, 1, 1])
    sg = rng.randrange(G)
    S = rng.choice([0, 1, 4, _log(rng, 1, 300)])
    if op in ("prefill", "train"):
        T = _log(rng, 1, 16384)
        B = max(1, min(8, 16384 // T, _log(rng, 1, 16)))
        W = rng.choice([_log(rng, 1, 2048), _log(rng, 32, 1024), 0 if T <= 2048 else 512])
        return _within(dict(op=op, B=B, T=T, G=G, k=k, d=d, sh=sh, sg=sg, W=W, S=S))
    if op == "commit":
        T = _log(rng, 1, 128)
        return dict(op=op, B=_log(rng, 1, 48), T=T, A=rng.randrange(0, T + 1), L=_log(rng, T + 200, 2048), G=G, d=d)
    B = _log(rng, 1, 64)
    L = _log(rng, 1, min(32768, (1 << 30) // (B * G * d)))
    W = rng.choice([0, _log(rng, 1, 4096), _log(rng, 64, 2048)]) if op == "tree" else _log(rng, 1, 4096)
    case = dict(op=op, B=B, L=L, G=G, k=k, d=d, sh=sh, sg=sg, W=W, S=S, ragged=rng.random() < 0.7)
    if op == "tree":
        case["T"] = _log(rng, 1, 128)
    return _within(case)


# Lengths that differ between the sequences of a batch, fixed by the case.

def _cache_lens(c):
    L = c["L"]
    if not c.get("ragged"):
        return [L] * c["B"]
    return [max(0 if c["op"] == "tree" else 1, L - (b * 37 + 11) * max(1, L // 97) % (L // 2 + 1))
            if not (c["op"] == "tree" and b == 2) else 0 for b in range(c["B"])]


def _tree_lens(c):
    T = c["T"]
    return [T if not c.get("ragged") else max(1, T - (b * 5) % (T // 2 + 1)) for b in range(c["B"])]


def _accepts(c):
    return [0 if (b % 7 == 3 or c["A"] == 0) else 1 + (c["A"] - 1 + b * 5) % c["A"] for b in range(c["B"])]


def _commit_lens(c):
    return [max(0, (c["L"] - c["T"]) - (b * 53) % (c["L"] // 2)) for b in range(c["B"])]


# --------------------------------------------------------------------------- inputs

def _normal(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=BF16)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    cpu = torch.Generator()
    cpu.manual_seed(seed)
    s = {"case": c}
    op, B, G, d = c["op"], c["B"], c["G"], c["d"]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")
    if op in ("prefill", "train", "tree", "decode"):
        T, k, sh = (1 if op == "decode" else c["T"]), c["k"], c["sh"]
        s["q"] = _normal(gen, B, G, T, k, d)
        s["qs"] = _normal(gen, B, T, d) if sh else None
    if op in ("prefill", "train"):
        s["K"], s["V"] = _normal(gen, B, G, T, d), _normal(gen, B, G, T, d)
        if op == "train":
            s["do"] = _normal(gen, B, G, T, k, d)
            s["dos"] = _normal(gen, B, T, d) if sh else None
    if op in ("decode", "tree"):
        s["Kc"], s["Vc"] = _normal(gen, B, G, c["L"], d), _normal(gen, B, G, c["L"], d)
        s["len"] = i32(_cache_lens(c))
    if op in ("tree", "commit"):
        T = c["T"]
        s["Kt"], s["Vt"] = _normal(gen, B, G, T, d), _normal(gen, B, G, T, d)
    if op == "tree":
        # a drafted token hangs under one of the few tokens before it; about one in eight starts a branch at the root
        u = torch.rand(B, T, generator=cpu)
        back = (torch.rand(B, T, generator=cpu) * 4).floor().long() + 1
        idx = torch.arange(T)
        par = torch.where(u < 0.125, torch.full((B, T), -1), (idx - back).clamp(min=-1))
        s["parent"] = par.to(torch.int32).cuda()
        s["tlen"] = i32(_tree_lens(c))
    if op == "commit":
        s["Kc"], s["Vc"] = _normal(gen, B, G, c["L"], d), _normal(gen, B, G, c["L"], d)
        s["len"], s["acc"] = i32(_commit_lens(c)), i32(_accepts(c))
        path = torch.full((B, T), -1, dtype=torch.int32)
        for b, n in enumerate(_accepts(c)):
            path[b, :n] = torch.randperm(T, generator=cpu)[:n].sort().values.to(torch.int32)
        s["path"] = path.cuda()
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """Shape struct, outputs and scratch, which a user's program keeps from call to call."""
    import moe_gqa_query_b200 as gq
    c = s["case"]
    op, B, G, d = c["op"], c["B"], c["G"], c["d"]
    T, k, sh = (1 if op == "decode" else c["T"]), c.get("k", 1), c.get("sh", 0)
    s["dims"] = gq.gqe_dims(B=B, T=T, d_model=64, G=G, E=max(k, 1), k=k, d_head=d, n_shared=sh,
                            shared_kv_group=c.get("sg", 0), renorm_scope=0, scale=0.0, output_mode=0)
    new = lambda *shape, dtype=BF16: torch.empty(*shape, dtype=dtype, device="cuda")
    ws = None
    if op == "commit":
        s["new_len"] = new(B, dtype=torch.int32)
        return
    s["o"] = new(B, G, T, k, d)
    s["os"] = new(B, T, d) if sh else None
    if op == "train":
        s["lse"] = new(B * G * T * k + B * T * sh, dtype=torch.float32)
        s["dq"], s["dqs"] = new(B, G, T, k, d), (new(B, T, d) if sh else None)
        s["dK"], s["dV"] = new(B, G, T, d), new(B, G, T, d)
        ws = gq.gqe_window_workspace_size(s["dims"], gq.GQE_OP_ATTN_WINDOW_BWD, 0, c["W"], c["S"])
    if op == "decode":
        ws = gq.gqe_window_workspace_size(s["dims"], gq.GQE_OP_ATTN_DECODE_WINDOW, c["L"], c["W"], c["S"])
    if op == "tree":
        ws = gq.gqe_window_workspace_size(s["dims"], gq.GQE_OP_ATTN_TREE, c["L"], c["W"], c["S"])
    if ws is not None:
        s["ws"] = new(max(ws, 256), dtype=torch.uint8)


# --------------------------------------------------------------------------- one pass

def run(state):
    return (_run_own if own else _run_plain)(state)


def _out(*parts):
    return [p for p in parts if p is not None]


def _run_own(s):
    import moe_gqa_query_b200 as gq
    c = s["case"]
    op = c["op"]
    if op == "prefill":
        gq.gqe_attn_prefill_window(s["dims"], s["q"], s["qs"], s["K"], s["V"], c["W"], c["S"], s["o"], s["os"])
        return _out(s["o"], s["os"])
    if op == "train":
        gq.gqe_attn_prefill_window(s["dims"], s["q"], s["qs"], s["K"], s["V"], c["W"], c["S"], s["o"], s["os"],
                                   s["lse"])
        gq.gqe_attn_prefill_window_bwd(s["dims"], s["q"], s["qs"], s["K"], s["V"], c["W"], c["S"], s["o"], s["os"],
                                       s["lse"], s["do"], s["dos"], s["dq"], s["dqs"], s["dK"], s["dV"], s["ws"])
        return _out(s["o"], s["os"], s["dq"], s["dqs"], s["dK"], s["dV"])
    if op == "decode":
        gq.gqe_attn_decode_window(s["dims"], s["q"], s["qs"], s["Kc"], s["Vc"], c["L"], s["len"], c["W"], c["S"],
                                  s["o"], s["os"], s["ws"])
        return _out(s["o"], s["os"])
    if op == "tree":
        gq.gqe_attn_tree(s["dims"], s["q"], s["qs"], s["Kt"], s["Vt"], s["parent"], s["tlen"], s["Kc"], s["Vc"],
                         c["L"], s["len"], c["W"], c["S"], s["o"], s["os"], s["ws"])
        return _out(s["o"], s["os"])
    gq.gqe_cache_commit(s["dims"], s["Kt"], s["Vt"], s["path"], s["acc"], s["Kc"], s["Vc"], c["L"], s["len"],
                        s["new_len"])
    return [s["Kc"], s["Vc"], s["new_len"]]


# Plain forms: products, exp and sums in 32 bits, rounded once at the end.

def _run_plain(s):
    return {"prefill": _plain_prefill, "train": _plain_train, "decode": _plain_decode, "tree": _plain_tree,
            "commit": _plain_commit}[s["case"]["op"]](s)


def _blocks(T, W, S):
    """Query blocks with the key positions any of their tokens sees."""
    step = min(T, max(64, min(512, W if W else 512)))
    for a in range(0, T, step):
        e = min(T, a + step)
        lo = max(0, a - W + 1) if W else 0
        yield a, e, min(S, lo), lo


def _keys(X, ns, lo, e):
    return X[:, :, lo:e] if ns == 0 else torch.cat((X[:, :, :ns], X[:, :, lo:e]), 2)


def _block_mask(a, e, ns, lo, W, S, dev):
    t = torch.arange(a, e, device=dev)[:, None]
    p = torch.cat((torch.arange(ns, device=dev), torch.arange(lo, e, device=dev)))[None, :]
    ok = p <= t
    return ok & ((p > t - W) | (p < S)) if W else ok


def _softmax(x):
    x = (x - x.amax(-1, keepdim=True)).exp()
    return x / x.sum(-1, keepdim=True)


def _plain_prefill(s):
    c = s["case"]
    T, W, S, sg = c["T"], c["W"], c["S"], c["sg"]
    sc = c["d"] ** -0.5
    o = torch.empty_like(s["q"])
    os_ = torch.empty_like(s["qs"]) if c["sh"] else None
    for a, e, ns, lo in _blocks(T, W, S):
        K, V = _keys(s["K"], ns, lo, e).float(), _keys(s["V"], ns, lo, e).float()
        ok = _block_mask(a, e, ns, lo, W, S, K.device)
        x = torch.einsum("bgtkd,bgpd->bgtkp", s["q"][:, :, a:e].float(), K) * sc
        pr = _softmax(x.masked_fill(~ok[None, None, :, None, :], -INF))
        o[:, :, a:e] = torch.einsum("bgtkp,bgpd->bgtkd", pr, V).to(BF16)
        if c["sh"]:
            x = torch.einsum("btd,bpd->btp", s["qs"][:, a:e].float(), K[:, sg]) * sc
            os_[:, a:e] = torch.einsum("btp,bpd->btd", _softmax(x.masked_fill(~ok, -INF)), V[:, sg]).to(BF16)
    return _out(o, os_)


def _plain_train(s):
    c = s["case"]
    T, W, S, sg = c["T"], c["W"], c["S"], c["sg"]
    sc = c["d"] ** -0.5
    o, dq = torch.empty_like(s["q"]), torch.empty_like(s["q"])
    os_, dqs = (torch.empty_like(s["qs"]), torch.empty_like(s["qs"])) if c["sh"] else (None, None)
    dK = torch.zeros(s["K"].shape, device="cuda")
    dV = torch.zeros(s["V"].shape, device="cuda")
    for a, e, ns, lo in _blocks(T, W, S):
        K, V = _keys(s["K"], ns, lo, e).float(), _keys(s["V"], ns, lo, e).float()
        ok = _block_mask(a, e, ns, lo, W, S, K.device)
        q, do = s["q"][:, :, a:e].float(), s["do"][:, :, a:e].float()
        x = torch.einsum("bgtkd,bgpd->bgtkp", q, K) * sc
        pr = _softmax(x.masked_fill(~ok[None, None, :, None, :], -INF))
        o[:, :, a:e] = torch.einsum("bgtkp,bgpd->bgtkd", pr, V).to(BF16)
        dp = torch.einsum("bgtkd,bgpd->bgtkp", do, V)
        ds = sc * pr * (dp - (pr * dp).sum(-1, keepdim=True))
        dq[:, :, a:e] = torch.einsum("bgtkp,bgpd->bgtkd", ds, K).to(BF16)
        gK = torch.einsum("bgtkp,bgtkd->bgpd", ds, q)
        gV = torch.einsum("bgtkp,bgtkd->bgpd", pr, do)
        if c["sh"]:
            q, do = s["qs"][:, a:e].float(), s["dos"][:, a:e].float()
            x = torch.einsum("btd,bpd->btp", q, K[:, sg]) * sc
            pr = _softmax(x.masked_fill(~ok, -INF))
            os_[:, a:e] = torch.einsum("btp,bpd->btd", pr, V[:, sg]).to(BF16)
            dp = torch.einsum("btd,bpd->btp", do, V[:, sg])
            ds = sc * pr * (dp - (pr * dp).sum(-1, keepdim=True))
            dqs[:, a:e] = torch.einsum("btp,bpd->btd", ds, K[:, sg]).to(BF16)
            gK[:, sg] += torch.einsum("btp,btd->bpd", ds, q)
            gV[:, sg] += torch.einsum("btp,btd->bpd", pr, do)
        for acc, g in ((dK, gK), (dV, gV)):
            acc[:, :, :ns] += g[:, :, :ns]
            acc[:, :, lo:e] += g[:, :, ns:]
    return _out(o, os_, dq, dqs, dK.to(BF16), dV.to(BF16))


def _pack_rows(q, qs, sg):
    """Routed and shared rows of every group as [B, G, T, k (+1), d]; the shared head's row only counts in group sg."""
    if qs is None:
        return q
    B, G, T, _, d = q.shape
    return torch.cat((q, qs[:, None, :, None].expand(B, G, T, 1, d)), 3)


def _unpack_rows(o, k, sh, sg):
    return _out(o[..., :k, :].contiguous().to(BF16), o[:, sg, :, k].contiguous().to(BF16) if sh else None)


def _batches(B, per_seq):
    n = max(1, min(B, (1 << 28) // max(1, per_seq)))
    return [(a, min(B, a + n)) for a in range(0, B, n)]


def _plain_decode(s):
    c = s["case"]
    B, G, k, L, W, S = c["B"], c["G"], c["k"], c["L"], c["W"], c["S"]
    q = _pack_rows(s["q"], s["qs"], c["sg"])[:, :, 0].float()
    out = torch.empty_like(q)
    p = torch.arange(L, device="cuda")[None, :]
    n = s["len"][:, None].long()
    ok = p < n
    if W:
        ok &= (p >= n - W) | (p < S)
    for a, e in _batches(B, G * L * max(c["d"], q.shape[2])):
        x = torch.einsum("bgrd,bgpd->bgrp", q[a:e], s["Kc"][a:e].float()) * c["d"] ** -0.5
        pr = _softmax(x.masked_fill(~ok[a:e, None, None], -INF))
        out[a:e] = torch.einsum("bgrp,bgpd->bgrd", pr, s["Vc"][a:e].float())
    return _unpack_rows(out[:, :, None], k, c["sh"], c["sg"])


def _ancestors(parent):
    """anc[b, i, j]: j is i or above it; by repeated squaring of the parent relation."""
    B, T = parent.shape
    j = torch.arange(T, device=parent.device)
    anc = ((parent[:, :, None].long() == j) | (j[:, None] == j)).float()
    for _ in range(max(1, (T - 1).bit_length())):
        anc = (torch.bmm(anc, anc) > 0).float()
    return anc > 0


def _plain_tree(s):
    c = s["case"]
    B, T, G, k, L, W, S = c["B"], c["T"], c["G"], c["k"], c["L"], c["W"], c["S"]
    q = _pack_rows(s["q"], s["qs"], c["sg"]).float()
    out = torch.empty_like(q)
    anc = _ancestors(s["parent"])
    depth = anc.sum(-1) - 1
    n = s["len"][:, None].long()
    pos = n + depth                                                   # [B, T]
    p = torch.arange(L, device="cuda")
    ok_c = (p < n[:, :, None]).expand(B, T, L)
    ok_t = anc
    if W:
        ok_c = ok_c & ((p > pos[:, :, None] - W) | (p < S))
        ok_t = anc & ((pos[:, None, :] > pos[:, :, None] - W) | (pos[:, None, :] < S))
    ok = torch.cat((ok_c, ok_t), 2)
    live = (torch.arange(T, device="cuda") < s["tlen"][:, None])[:, None, :, None, None]
    for a, e in _batches(B, G * (L + T) * max(c["d"], T * q.shape[3])):
        K = torch.cat((s["Kc"][a:e], s["Kt"][a:e]), 2).float()
        x = torch.einsum("bgtrd,bgpd->bgtrp", q[a:e], K) * c["d"] ** -0.5
        del K
        pr = _softmax(x.masked_fill(~ok[a:e, None, :, None], -INF))
        V = torch.cat((s["Vc"][a:e], s["Vt"][a:e]), 2).float()
        out[a:e] = torch.einsum("bgtrp,bgpd->bgtrd", pr, V)
    return _unpack_rows(out.masked_fill(~live, 0.0), k, c["sh"], c["sg"])


def _plain_commit(s):
    c = s["case"]
    b = torch.arange(c["B"], device="cuda")[:, None]
    i = torch.arange(c["T"], device="cuda")[None, :]
    take = (i < s["acc"][:, None])[:, :, None, None]
    src = s["path"].long().clamp(min=0)
    dst = s["len"][:, None].long() + i                    # every case leaves room for T rows
    for cache, rows in ((s["Kc"], s["Kt"]), (s["Vc"], s["Vt"])):
        cache[b, :, dst] = torch.where(take, rows[b, :, src], cache[b, :, dst])
    return [s["Kc"], s["Vc"], s["len"] + s["acc"]]


# --------------------------------------------------------------------------- work

def _pairs(T, W, S):
    """Visible (query, key) pairs of one head over T tokens."""
    if not W or W >= T:
        return T * (T + 1) // 2
    n = W * (W + 1) // 2 + (T - W) * W
    for t in range(W, T):                      # sinks that the window has left behind
        hid = t + 1 - W
        if hid >= S:
            return n + (T - t) * S
        n += hid
    return n


def work(case):
    c = case
    op, B, G, d = c["op"], c["B"], c["G"], c["d"]
    if op == "commit":
        return {"bytes": sum(_accepts(c)) * (G * d * 2 * 2 * 2 + 4) + 12 * B, "flops": 0}
    k, sh, W, S = c["k"], c["sh"], c["W"], c["S"]
    heads = G * k + sh
    if op in ("prefill", "train"):
        T = c["T"]
        row, kv = B * heads * T * d * 2, B * G * T * d * 2 * 2
        pairs = B * heads * _pairs(T, W, S)
        if op == "prefill":
            return {"bytes": 2 * row + kv, "flops": 4 * d * pairs}
        return {"bytes": 4 * row + 2 * kv, "flops": 14 * d * pairs}
    nbytes = flops = 0
    tl = _tree_lens(c) if op == "tree" else [1] * B
    for n, m in zip(_cache_lens(c), tl):
        # the lowest position of the call sees the most of the cache: the first drafted tokens', or the new token's
        first = n if op == "tree" else n - 1
        lo = max(0, first - W + 1) if W else 0
        rows = n - lo + min(S, lo)
        nbytes += rows * G * d * 2 * 2 + m * heads * d * 2 * 2 + (m * G * d * 2 * 2 + 4 * m if op == "tree" else 0) + 4
        flops += 4 * d * heads * m * (rows + (1 if op == "tree" else 0))     # and at least itself of the tree
    return {"bytes": nbytes, "flops": flops}


# --------------------------------------------------------------------------- exact values

def exact(case, seed):
    """The definition in 64 bits, one sequence and group after the other, every key with a mask of its own."""
    global own
    keep, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = keep
    c = s["case"]
    return {"prefill": _exact_prefill, "train": _exact_prefill, "decode": _exact_cache, "tree": _exact_cache,
            "commit": _exact_commit}[c["op"]](c, s)


def _sees(t, p, W, S):
    return (p <= t) & ((p < S) | (t - p < W)) if W else p <= t


def _exact_prefill(c, s):
    B, T, G, k, d, W, S = (c[x] for x in ("B", "T", "G", "k", "d", "W", "S"))
    train = c["op"] == "train"
    f64 = dict(dtype=torch.float64, device="cuda")
    o, os_ = torch.zeros(B, G, T, k, d, **f64), torch.zeros(B, T, d, **f64)
    dq, dqs = torch.zeros_like(o), torch.zeros_like(os_)
    dK, dV = torch.zeros(B, G, T, d, **f64), torch.zeros(B, G, T, d, **f64)
    p = torch.arange(T, device="cuda")
    step = max(1, min(T, (1 << 25) // T))
    for b in range(B):
        for g in range(G):
            heads = [(s["q"][b, g, :, j], o[b, g, :, j], dq[b, g, :, j], s["do"][b, g, :, j] if train else None)
                     for j in range(k)]
            if c["sh"] and g == c["sg"]:
                heads.append((s["qs"][b], os_[b], dqs[b], s["dos"][b] if train else None))
            K, V = s["K"][b, g].double(), s["V"][b, g].double()
            K.requires_grad_(train)
            V.requires_grad_(train)
            for q, out, gq, do in heads:
                for a in range(0, T, step):
                    e = min(T, a + step)
                    qa = q[a:e].double().requires_grad_(train)
                    hide = ~_sees(p[a:e, None], p[None, :e], W, S)
                    y = torch.softmax((qa @ K[:e].T / math.sqrt(d)).masked_fill(hide, -INF), 1) @ V[:e]
                    out[a:e] = y.detach()
                    if train:
                        y.backward(do[a:e].double())
                        gq[a:e] = qa.grad
            if train:
                dK[b, g], dV[b, g] = K.grad, V.grad
    if not train:
        return _out(o, os_ if c["sh"] else None)
    return _out(o, os_ if c["sh"] else None, dq, dqs if c["sh"] else None, dK, dV)


def _exact_cache(c, s):
    B, G, k, d, W, S, tree = c["B"], c["G"], c["k"], c["d"], c["W"], c["S"], c["op"] == "tree"
    T = c["T"] if tree else 1
    o = torch.zeros(B, G, T, k, d, dtype=torch.float64, device="cuda")
    os_ = torch.zeros(B, T, d, dtype=torch.float64, device="cuda")
    for b, n in enumerate(_cache_lens(c)):
        m, pos, sees = 1, [n - 1], None
        if tree:
            m, par = _tree_lens(c)[b], s["parent"][b].tolist()
            lines = []                                   # each token's ancestors and itself
            for i in range(m):
                lines.append((lines[par[i]] if par[i] >= 0 else []) + [i])
            pos = [n + len(line) - 1 for line in lines]
            sees = torch.zeros(m, m, dtype=torch.bool)
            for i, line in enumerate(lines):
                sees[i, line] = True
        t = torch.tensor(pos, device="cuda")[:, None]
        hide = ~_sees(t, torch.arange(n, device="cuda")[None], W, S)
        K, V = s["Kc"][b, :, :n].double(), s["Vc"][b, :, :n].double()
        if tree:
            hide = torch.cat((hide, ~(sees.cuda() & _sees(t, t.T, W, S))), 1)
            K = torch.cat((K, s["Kt"][b, :, :m].double()), 1)
            V = torch.cat((V, s["Vt"][b, :, :m].double()), 1)
        for j in range(k):
            x = s["q"][b, :, :m, j].double() @ K.transpose(1, 2) / math.sqrt(d)
            o[b, :, :m, j] = torch.softmax(x.masked_fill(hide, -INF), 2) @ V
        if c["sh"]:
            x = s["qs"][b, :m].double() @ K[c["sg"]].T / math.sqrt(d)
            os_[b, :m] = torch.softmax(x.masked_fill(hide, -INF), 1) @ V[c["sg"]]
    return _out(o, os_ if c["sh"] else None)


def _exact_commit(c, s):
    Kc, Vc = s["Kc"].clone(), s["Vc"].clone()
    lens, acc, path = s["len"].tolist(), s["acc"].tolist(), s["path"].tolist()
    for b in range(c["B"]):
        for i in range(acc[b]):
            Kc[b, :, lens[b] + i] = s["Kt"][b, :, path[b][i]]
            Vc[b, :, lens[b] + i] = s["Vt"][b, :, path[b][i]]
    return [Kc.double(), Vc.double(), torch.tensor([n + m for n, m in zip(lens, acc)], device="cuda")]
