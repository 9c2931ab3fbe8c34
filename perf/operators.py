"""Measured work of the operators of a tree-drafted decoding step.

A hybrid model (KDA layers with softmax-attention layers between them) that
decodes with drafts runs, per step and sequence, M drafted tokens that form a
tree: node m hangs below node parent[m] < m (-1: directly below the tokens that
came before; -2: no node, padding).  Node 0 is the last token that is certain.

    decode_tree     a KDA layer over the tree: every node's output
    tree_attention  a softmax layer over the tree and a paged cache
    verify_drafts   which nodes the target's probabilities accept, and the token after them
    decode_commit   a KDA layer's state after the accepted path
    cache_append    the accepted path's keys and values into the pages

``run`` computes the plain form with elementary torch operations in fp32 where
``own`` is false, and calls the library's entry points where it is true.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ESZ = {"bf16": 2, "f32": 4}
ONE = 1 << 38            # fixed-point one of the drafts' probability masses


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # one KDA layer at the decode workload of this repository's benchmark (256 sequences,
        # 96 heads of 128), 16 drafted nodes each
        dict(name="decode_tree_256x16", op="decode_tree", N=256, M=16, H=96, d=128, dt="bf16", shape="tree"),
        # fp32 inputs, a small batch, odd counts, some trees shorter than the row
        dict(name="decode_tree_f32_odd", op="decode_tree", N=3, M=13, H=12, d=64, dt="f32", shape="padded"),
        # the accepted paths (one to six tokens) into the same 256 x 96 states
        dict(name="decode_commit_256", op="decode_commit", N=256, M=16, H=96, d=128, dt="bf16", depth=6),
        # a single user's step: latency
        dict(name="decode_commit_one", op="decode_commit", N=1, M=8, H=24, d=128, dt="f32", depth=4),
        # a single user's step over a short cache: latency
        dict(name="attention_one_short", op="tree_attention", N=1, M=8, Hq=32, Hkv=8, d=128, dt="bf16",
             lo=501, hi=501, page=16, shape="tree"),
        # a serving batch, lengths as ragged as the packed documents of the benchmark, 12 query
        # heads to a cache head
        dict(name="attention_batch_ragged", op="tree_attention", N=64, M=16, Hq=96, Hkv=8, d=128, dt="bf16",
             lo=512, hi=8192, page=64, shape="tree"),
        # few sequences over a very long cache (the benchmark's long context)
        dict(name="attention_long", op="tree_attention", N=4, M=7, Hq=32, Hkv=4, d=128, dt="bf16",
             lo=250001, hi=262144, page=64, shape="chain"),
        # fp32, head size 64, a page size that divides no tile, trees shorter than the row
        dict(name="attention_f32_odd", op="tree_attention", N=5, M=11, Hq=12, Hkv=4, d=64, dt="f32",
             lo=1, hi=3001, page=24, shape="padded"),
        # a tree of the draft's likeliest tokens, no draft probabilities; an odd vocabulary
        dict(name="verify_tree_small", op="verify_drafts", N=3, M=16, V=50257, dt="f32", shape="tree", q=False),
        # chains sampled from the draft's distribution over the whole decode batch
        dict(name="verify_chain_256", op="verify_drafts", N=256, M=8, V=131072, dt="f32", shape="chain", q=True),
        # the accepted tokens of a small batch
        dict(name="append_step", op="cache_append", N=16, M=8, Hkv=8, d=128, dt="bf16", lo=100, hi=4096, page=64,
             path=True),
        # the keys and values of eight prompts going into their pages
        dict(name="append_prompts", op="cache_append", N=8, M=4096, Hkv=8, d=128, dt="bf16", lo=0, hi=100, page=64,
             path=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["decode_tree", "decode_commit", "tree_attention", "tree_attention", "verify_drafts",
                     "cache_append"])
    dt = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op in ("decode_tree", "decode_commit"):
        while True:
            c = dict(op=op, N=_log(rng, 1, 256), M=_log(rng, 1, 48), H=_log(rng, 1, 96),
                     d=rng.choice([16, 32, 64, 128, 128, 128, 128]), dt=dt)
            # the node states of the plain form bound the cost
            if c["N"] * c["M"] * c["H"] * c["d"] ** 2 <= 256 * 16 * 96 * 128 ** 2:
                break
        if op == "decode_tree":
            c["shape"] = rng.choice(["tree", "chain", "padded"])
        else:
            c["depth"] = rng.randint(1, min(c["M"], 8))
        return c
    if op == "tree_attention":
        while True:
            Hkv = rng.choice([1, 2, 4, 8, 16])
            hi = _log(rng, 1, 262144)
            c = dict(op=op, N=_log(rng, 1, 128), M=_log(rng, 1, 64), Hq=Hkv * rng.choice([1, 2, 3, 4, 8, 12, 16]),
                     Hkv=Hkv, d=rng.choice([64, 128, 128, 128]), dt=dt, lo=rng.choice([0, hi // 2, hi]), hi=hi,
                     page=rng.choice([16, 32, 64, 64, 128, 24, 256]), shape=rng.choice(["tree", "chain", "padded"]))
            tokens = c["N"] * c["hi"]
            if tokens * c["M"] * c["Hq"] * c["d"] <= (6e10 if dt == "bf16" else 6e9) \
                    and tokens * c["Hkv"] * c["d"] <= 4 * 262144 * 4 * 128:
                return c
    if op == "verify_drafts":
        while True:
            q = rng.random() < 0.5
            c = dict(op=op, N=_log(rng, 1, 256), M=rng.randint(1, 32), V=_log(rng, 1000, 200000), dt=dt,
                     shape="chain" if q else rng.choice(["tree", "chain", "padded"]), q=q)
            if c["N"] * c["M"] * c["V"] <= 256 * 8 * 131072:
                return c
    while True:
        path = rng.random() < 0.6
        lo = _log(rng, 1, 4096) - 1
        c = dict(op=op, N=_log(rng, 1, 64), M=rng.randint(1, 32) if path else _log(rng, 1, 8192),
                 Hkv=rng.choice([1, 2, 4, 8, 16]), d=rng.choice([16, 32, 64, 128, 128]), dt=dt, lo=lo,
                 hi=lo + rng.randint(0, 2000), page=rng.choice([16, 32, 64, 128, 24]), path=path)
        if c["N"] * (c["M"] + c["hi"]) * c["Hkv"] * c["d"] <= 8 * 4196 * 8 * 128:
            return c


# ---------------------------------------------------------------------------- inputs

def _parents(case, rs):
    """[N, M] int32: trees whose nodes branch often near the root, chains, or trees of 1..M nodes."""
    N, M = case["N"], case["M"]
    m = np.arange(M)
    if case.get("shape") == "chain":
        par = np.broadcast_to(m - 1, (N, M)).copy()
    else:
        par = np.floor(rs.random_sample((N, M)) ** 0.7 * m).astype(np.int64)
        par[:, 0] = -1
    if case.get("shape") == "padded":
        par[m[None, :] >= rs.randint(1, M + 1, (N, 1))] = -2
    return par.astype(np.int32)


def _lengths(case, rs):
    return rs.randint(case["lo"], case["hi"] + 1, case["N"]).astype(np.int32)


def _pages(case, need, most, rs):
    """A page table [N, pages of `most` tokens] over a pool with some spare pages, in random order."""
    page = case["page"]
    per = np.maximum(1, -(-need.astype(np.int64) // page))
    width = max(1, -(-most // page))
    pool = len(need) * width + 3
    order = rs.permutation(pool).astype(np.int32)
    table, at = np.zeros((len(need), width), np.int32), 0
    for n, c in enumerate(per):
        table[n, :c] = order[at:at + c]
        at += int(c)
    return pool, table


def prepare(case, seed):
    rs = np.random.RandomState(seed % (1 << 32))
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[case["dt"]]
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda")
    rand = lambda *s: torch.rand(s, generator=gen, device="cuda")
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    op = case["op"]
    st = {"case": case}
    if op in ("decode_tree", "decode_commit"):
        N, M, H, d = (case[x] for x in ("N", "M", "H", "d"))
        unit = lambda x: x / x.norm(dim=-1, keepdim=True)
        st["k"] = unit(randn(N * M, H, d)).to(dt)
        st["v"] = randn(N * M, H, d).to(dt)
        st["g"] = -5 * torch.sigmoid(randn(N * M, H, d))
        st["beta"] = torch.sigmoid(randn(N * M, H))
        # the state that a long prefix leaves: of the values' size
        st["state"] = randn(N, H, d, d) * 0.3
        if op == "decode_tree":
            st["q"] = unit(randn(N * M, H, d)).to(dt)
            st["parent"] = dev(_parents(case, rs))
        else:
            depth = rs.randint(1, case["depth"] + 1, N)
            # an accepted path skips the siblings that were not taken
            path = np.sort(np.stack([rs.permutation(M)[:case["depth"]] for _ in range(N)]), axis=1).astype(np.int32)
            st["path"], st["accept"] = dev(path), dev(depth.astype(np.int32))
            st["state_out"] = torch.empty_like(st["state"])
        return st
    if op == "tree_attention":
        N, M, Hq, Hkv, d = (case[x] for x in ("N", "M", "Hq", "Hkv", "d"))
        lens = _lengths(case, rs)
        pool, table = _pages(case, lens, case["hi"], rs)
        st["q"] = (randn(N * M, Hq, d) * 1.5).to(dt)
        st["k_new"], st["v_new"] = randn(N * M, Hkv, d).to(dt), randn(N * M, Hkv, d).to(dt)
        cache = []
        for _ in range(2):
            x = torch.empty((pool, Hkv, case["page"], d), dtype=dt, device="cuda")
            x.normal_(generator=gen)
            cache.append(x)
        st["k_cache"], st["v_cache"] = cache
        st["table"], st["lens"] = dev(table), dev(lens)
        st["parent"] = dev(_parents(case, rs))
        return st
    if op == "verify_drafts":
        N, M, V = (case[x] for x in ("N", "M", "V"))
        par = _parents(case, rs)
        st["parent"] = dev(par)
        tokens = torch.zeros((N, M), dtype=torch.int32, device="cuda")
        draft = torch.empty((N, M, V), dtype=dt, device="cuda")
        target = torch.empty((N, M, V), dtype=dt, device="cuda")
        for n in range(N):
            logits = randn(M, V) * 3.0
            target[n] = torch.softmax(logits, -1).to(dt)
            dlog = logits + randn(M, V) * 0.6       # the draft model's, near the target's
            draft[n] = torch.softmax(dlog, -1).to(dt)
            if case["q"]:                           # sampled from the draft
                pick = (dlog - torch.log(-torch.log(rand(M, V).clamp_min(1e-20)))).argmax(-1)
                tokens[n, 1:] = pick[:-1].int()
            else:                                   # the draft's likeliest, in order, per parent
                rank, seen = np.zeros(M, np.int64), {}
                for m in range(1, M):
                    rank[m] = seen.get(int(par[n, m]), 0)
                    seen[int(par[n, m])] = rank[m] + 1
                k = min(int(rank.max()) + 1, V)
                top = dlog.topk(k, dim=-1).indices
                rows = dev(np.maximum(par[n], 0).astype(np.int64))
                tokens[n] = top[rows, dev(rank)].int()
        tokens[:, 0] = (rand(N) * V).int().clamp_max(V - 1)
        st["tokens"], st["target"] = tokens, target
        st["draft"] = draft if case["q"] else None
        st["u"] = rand(N, M + 1)
        return st
    N, M, Hkv, d = (case[x] for x in ("N", "M", "Hkv", "d"))
    lens = _lengths(case, rs)
    if case["path"]:
        count = rs.randint(1, M + 1, N).astype(np.int32)
        path = np.full((N, M), -1, np.int32)
        for n in range(N):
            path[n, :count[n]] = np.sort(rs.permutation(M)[:count[n]])
        st["path"] = dev(path)
    else:
        count = rs.randint(max(1, M // 2), M + 1, N).astype(np.int32)
        st["path"] = None
    pool, table = _pages(case, lens + M, case["hi"] + M, rs)
    st["k_new"], st["v_new"] = randn(N * M, Hkv, d).to(dt), randn(N * M, Hkv, d).to(dt)
    st["k_cache"] = torch.zeros((pool, Hkv, case["page"], d), dtype=dt, device="cuda")
    st["v_cache"] = torch.zeros((pool, Hkv, case["page"], d), dtype=dt, device="cuda")
    st["table"], st["lens"], st["accept"] = dev(table), dev(lens), dev(count)
    return st


# ---------------------------------------------------------------------------- one pass

def run(st):
    c = st["case"]
    if own:
        return _run_own(st, c["op"])
    return {"decode_tree": _plain_decode_tree, "decode_commit": _plain_decode_commit,
            "tree_attention": _plain_attention, "verify_drafts": _plain_verify,
            "cache_append": _plain_append}[c["op"]](st)


def _run_own(st, op):
    from linear_attention_03_gb300 import kda
    if op == "decode_tree":
        return kda.kda_decode_tree(st["q"], st["k"], st["v"], st["g"], st["beta"], st["state"], st["parent"])
    if op == "decode_commit":
        return kda.kda_decode_commit(st["k"], st["v"], st["g"], st["beta"], st["state"], st["path"], st["accept"],
                                     state_out=st["state_out"])
    if op == "tree_attention":
        out, lse = kda.kda_tree_attention(st["q"], st["k_new"], st["v_new"], st["k_cache"], st["v_cache"],
                                          st["table"], st["lens"], st["parent"], want_lse=True)
        return {"out": out, "lse": lse}
    if op == "verify_drafts":
        accept, path, token = kda.kda_verify_drafts(st["target"], st["tokens"], st["parent"], st["u"],
                                                    draft_probs=st["draft"])
        return {"accept": accept, "path": path, "next": token}
    lens = kda.kda_cache_append(st["k_new"], st["v_new"], st["k_cache"], st["v_cache"], st["table"], st["lens"],
                                path=st["path"], accept=st["accept"])
    return {"k": st["k_cache"], "v": st["v_cache"], "lens": lens}


def _plain_decode_tree(st):
    """o_m = S_m^T q_m with S_m = Diag(a) S_p + k (beta (v - (Diag(a) S_p)^T k))^T, p = parent[m]."""
    c = st["case"]
    N, M, H, d = (c[x] for x in ("N", "M", "H", "d"))
    q, k, v = (st[x].float().view(N, M, H, d) for x in ("q", "k", "v"))
    a, beta = torch.exp(st["g"]).view(N, M, H, d), st["beta"].view(N, M, H)
    par = st["parent"].long()
    # all states in one tensor: slot 0 is the prefix's, slot m + 1 node m's
    S = torch.empty((M + 1, N, H, d, d), device="cuda")
    S[0] = st["state"]
    out = torch.zeros((N, M, H, d), device="cuda")
    rows = torch.arange(N, device="cuda")
    live = torch.zeros((N, M + 1), dtype=torch.bool, device="cuda")
    live[:, 0] = True
    for m in range(M):
        ok = (par[:, m] >= -1) & (par[:, m] < m)
        slot = torch.where(ok, par[:, m] + 1, torch.zeros_like(par[:, m]))
        ok = ok & live[rows, slot]
        live[:, m + 1] = ok
        s = S[slot, rows] * a[:, m, :, :, None]
        u = beta[:, m, :, None] * (v[:, m] - torch.matmul(k[:, m, :, None, :], s)[:, :, 0])
        s += k[:, m, :, :, None] * u[:, :, None, :]
        S[m + 1] = s
        o = torch.matmul(q[:, m, :, None, :], s)[:, :, 0]
        out[:, m] = torch.where(ok[:, None, None], o, torch.zeros_like(o))
    return out.view(N * M, H, d).to(st["q"].dtype)


def _plain_decode_commit(st):
    c = st["case"]
    N, M, H, d = (c[x] for x in ("N", "M", "H", "d"))
    k, v = (st[x].view(N, M, H, d) for x in ("k", "v"))
    g, beta = st["g"].view(N, M, H, d), st["beta"].view(N, M, H)
    path, accept = st["path"].long(), st["accept"]
    rows = torch.arange(N, device="cuda")
    s = st["state"].clone()
    for t in range(path.shape[1]):
        at, on = path[:, t].clamp_min(0), t < accept
        kt, vt = k[rows, at].float(), v[rows, at].float()
        new = s * torch.exp(g[rows, at])[..., None]
        u = beta[rows, at][..., None] * (vt - torch.matmul(kt[:, :, None, :], new)[:, :, 0])
        new += kt[..., None] * u[:, :, None, :]
        s = torch.where(on[:, None, None, None], new, s)
    return s


def _ancestors(par):
    """[N, M, M] truth values: j is m or above it; no entry in the rows of padding."""
    N, M = par.shape
    anc = torch.zeros((N, M, M), dtype=torch.bool, device=par.device)
    rows = torch.arange(N, device=par.device)
    for m in range(M):
        p = par[:, m].long()
        up = anc[rows, p.clamp(0, M - 1)]
        ok = (p == -1) | ((p >= 0) & (p < m) & up.any(-1))
        anc[:, m] = up & (p >= 0)[:, None]
        anc[:, m, m] = True
        anc[:, m] &= ok[:, None]
    return anc


def _plain_attention(st):
    c = st["case"]
    N, M, Hq, Hkv, d = (c[x] for x in ("N", "M", "Hq", "Hkv", "d"))
    G, page = Hq // Hkv, c["page"]
    anc = _ancestors(st["parent"])
    lens = st["lens"].tolist()
    out = torch.zeros((N, M, Hq, d), device="cuda")
    lse = torch.full((N, M, Hq), -math.inf, device="cuda")
    q = st["q"].float().view(N, M, Hkv, G, d)
    kn, vn = st["k_new"].float().view(N, M, Hkv, d), st["v_new"].float().view(N, M, Hkv, d)
    for n in range(N):
        L = lens[n]
        idx = st["table"][n, :max(1, -(-L // page))].long()
        gather = lambda x: x[idx].transpose(0, 1).reshape(Hkv, -1, d)[:, :L].float()   # [Hkv, L, d]
        qn = q[n].permute(1, 0, 2, 3).reshape(Hkv, M * G, d)
        s_old = torch.matmul(qn, gather(st["k_cache"]).transpose(1, 2)) / math.sqrt(d)
        s_new = torch.matmul(qn, kn[n].permute(1, 2, 0)) / math.sqrt(d)
        vis = anc[n][:, None, :].expand(M, G, M).reshape(M * G, M)
        s_new = s_new.masked_fill(~vis, -math.inf)
        s = torch.cat([s_old, s_new], -1)
        top = s.amax(-1, keepdim=True)
        top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
        if L == 0:
            top = torch.where(vis.any(-1)[None, :, None], top, torch.zeros_like(top))
        e = torch.exp(s - top)
        z = e.sum(-1, keepdim=True)
        o = torch.matmul(e[..., :L], gather(st["v_cache"])) + torch.matmul(e[..., L:], vn[n].transpose(0, 1))
        o = o / z
        l = (top + torch.log(z))[..., 0]
        on = vis.any(-1)
        o = torch.where(on[None, :, None], o, torch.zeros_like(o))
        l = torch.where(on[None, :], l, torch.full_like(l, -math.inf))
        out[n] = o.view(Hkv, M, G, d).permute(1, 0, 2, 3).reshape(M, Hq, d)
        lse[n] = l.view(Hkv, M, G).permute(1, 0, 2).reshape(M, Hq)
    return {"out": out.view(N * M, Hq, d).to(st["q"].dtype), "lse": lse.view(N * M, Hq)}


def _fixed(p):
    """A probability as a whole number of 2^-38: the sums are exact in any order."""
    return (p.nan_to_num(0.0).clamp(0.0, 1.0).double() * ONE).long()


def _ticks(u):
    return (u.clamp(0.0, 1.0) * (1 << 24)).long().clamp_max((1 << 24) - 1)


def _plain_verify(st):
    c = st["case"]
    N, M, V = (c[x] for x in ("N", "M", "V"))
    p, q, tok, par, u = st["target"], st["draft"], st["tokens"].long(), st["parent"].long(), st["u"]
    rows = torch.arange(N, device="cuda")
    cur = torch.zeros(N, dtype=torch.long, device="cuda")
    on = par[:, 0] == -1
    accept, path = on.int(), torch.full((N, M), -1, dtype=torch.int32, device="cuda")
    path[:, 0] = torch.where(on, 0, -1).int()
    spent = torch.zeros(N, dtype=torch.long, device="cuda")
    out_of = torch.zeros((N, M), dtype=torch.bool, device="cuda")     # the current node's refused children
    tick = _ticks(u)
    for m in range(1, M):
        child = on & (par[:, m] == cur)
        t = tok[:, m]
        good = (t >= 0) & (t < V)
        px = p[rows, cur, t.clamp(0, V - 1)].float()
        if q is not None:
            take = u[rows, cur] * q[rows, cur, t.clamp(0, V - 1)].float() < px
            # one child can be tested against a distribution it was sampled from: the first
            take = child & good & take & ~out_of.any(-1)
        else:
            twice = (out_of & (tok == t[:, None])).any(-1)
            mass = torch.where(good & ~twice, _fixed(px), torch.zeros_like(spent))
            take = child & ((tick[rows, cur] << 14) < spent + mass)
            spent = torch.where(take, 0, torch.where(child, spent + mass, spent))
        out_of[:, m] = child & ~take
        out_of &= ~take[:, None]
        cur = torch.where(take, m, cur)
        path[rows, torch.where(take, accept.long(), 0)] = torch.where(take, torch.full_like(path[:, 0], m), path[:, 0])
        accept = accept + take.int()
    pr = p[rows, cur].float()
    full = _fixed(pr)
    refused = out_of.any(-1)
    if q is not None:
        w = _fixed(pr - q[rows, cur].float())
        w = torch.where(refused[:, None], w, full)
    else:
        w = full.clone()
        for m in range(1, M):
            t = tok[:, m]
            gone = out_of[:, m] & (t >= 0) & (t < V)
            at = t.clamp(0, V - 1)
            w[rows, at] = torch.where(gone, torch.zeros_like(cur), w[rows, at])
    w = torch.where((w.sum(-1) == 0)[:, None], full, w)
    cum = w.cumsum(-1)
    total = cum[:, -1]
    need = (tick[:, M] * total) >> 24
    token = (cum <= need[:, None]).sum(-1)
    token = torch.where(on & (total > 0), token, torch.full_like(token, -1))
    return {"accept": accept, "path": path, "next": token.int()}


def _plain_append(st):
    c = st["case"]
    N, M, Hkv, d, page = (c[x] for x in ("N", "M", "Hkv", "d", "page"))
    t = torch.arange(M, device="cuda")
    n_idx, t_idx = torch.nonzero(t[None, :] < st["accept"][:, None], as_tuple=True)
    src = t_idx if st["path"] is None else st["path"][n_idx, t_idx].long()
    pos = st["lens"][n_idx].long() + t_idx
    pg = st["table"][n_idx, pos // page].long()
    for new, cache in ((st["k_new"], st["k_cache"]), (st["v_new"], st["v_cache"])):
        cache[pg, :, pos % page] = new.view(N, M, Hkv, d)[n_idx, src]
    return {"k": st["k_cache"], "v": st["v_cache"], "lens": st["lens"] + st["accept"]}


# ---------------------------------------------------------------------------- floors

def work(case):
    op, e = case["op"], ESZ[case["dt"]]
    if op == "decode_tree":
        N, M, H, d = (case[x] for x in ("N", "M", "H", "d"))
        node = H * (d * (4 * e + 4) + 4)                        # q, k, v, out; g; beta
        # reads of the state for k and q (2 d^2 multiply-adds each); pairs are far fewer
        return {"bytes": N * (H * d * d * 4 + M * (node + 4)), "flops": N * M * H * 4 * d * d}
    if op == "decode_commit":
        N, H, d = (case[x] for x in ("N", "H", "d"))
        mean = (1 + case["depth"]) / 2
        return {"bytes": int(N * H * (2 * d * d * 4 + mean * (d * (2 * e + 4) + 4))),
                "flops": int(N * H * mean * 5 * d * d)}
    if op == "tree_attention":
        N, M, Hq, Hkv, d = (case[x] for x in ("N", "M", "Hq", "Hkv", "d"))
        keys = N * (case["lo"] + case["hi"]) / 2
        return {"bytes": int(keys * Hkv * d * 2 * e + N * M * ((2 * Hq + 2 * Hkv) * d * e + Hq * 4)),
                "flops": int(4 * (keys + N) * M * Hq * d)}
    if op == "verify_drafts":
        N, M, V = (case[x] for x in ("N", "M", "V"))
        # the last accepted node's row; with draft probabilities about three rows in four are
        # read beside it (a chain that was not accepted whole)
        rows = 1.75 if case["q"] and M > 1 else 1.0
        return {"bytes": int(N * V * e * rows + N * M * 16), "flops": int(N * V * 2 * rows)}
    N, M, Hkv, d = (case[x] for x in ("N", "M", "Hkv", "d"))
    mean = (1 + M) / 2 if case["path"] else (max(1, M // 2) + M) / 2
    return {"bytes": int(N * mean * Hkv * d * e * 4), "flops": 0}


# ---------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """The definition in fp64; None where a case has whole numbers alone."""
    op = case["op"]
    if op == "verify_drafts":
        return None                 # whole numbers alone
    st = prepare(case, seed)
    if op == "cache_append":
        return _exact_append(st, case)
    if op == "decode_tree":
        return _exact_tree(st, case)
    if op == "decode_commit":
        return _exact_commit(st, case)
    return _exact_attention(st, case)


def _step64(S, k, v, g, beta):
    """(I - beta k k^T) Diag(e^g) S + beta k v^T, one state [..., d, d]."""
    D = g.double().exp().unsqueeze(-1) * S
    kk = k.double()
    read = (kk.unsqueeze(-1) * D).sum(-2)
    return D - (beta.double().unsqueeze(-1) * kk).unsqueeze(-1) * (read - v.double()).unsqueeze(-2)


def _exact_tree(st, c):
    N, M, H, d = (c[x] for x in ("N", "M", "H", "d"))
    par = st["parent"].tolist()
    out = torch.zeros((N, M, H, d), dtype=torch.float64, device="cuda")
    sh = lambda x: x.view(N, M, *x.shape[1:])
    q, k, v, g, beta = (sh(st[x]) for x in ("q", "k", "v", "g", "beta"))
    for n in range(N):
        states = {-1: st["state"][n].double()}
        for m in range(M):
            if par[n][m] in states and par[n][m] < m:
                states[m] = _step64(states[par[n][m]], k[n, m], v[n, m], g[n, m], beta[n, m])
                out[n, m] = (q[n, m].double().unsqueeze(-1) * states[m]).sum(-2)
    return out.view(N * M, H, d)


def _exact_commit(st, c):
    N, M = c["N"], c["M"]
    sh = lambda x: x.view(N, M, *x.shape[1:])
    k, v, g, beta = (sh(st[x]) for x in ("k", "v", "g", "beta"))
    path, count = st["path"].tolist(), st["accept"].tolist()
    out = torch.empty(st["state"].shape, dtype=torch.float64, device="cuda")
    for n in range(N):
        S = st["state"][n].double()
        for m in path[n][:count[n]]:
            S = _step64(S, k[n, m], v[n, m], g[n, m], beta[n, m])
        out[n] = S
    return out


def _exact_attention(st, c):
    N, M, Hq, Hkv, d = (c[x] for x in ("N", "M", "Hq", "Hkv", "d"))
    G, page = Hq // Hkv, c["page"]
    par, lens = st["parent"].tolist(), st["lens"].tolist()
    out = torch.zeros((N, M, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((N, M, Hq), -math.inf, dtype=torch.float64, device="cuda")
    q = st["q"].view(N, M, Hq, d).double()
    kn, vn = (st[x].view(N, M, Hkv, d).double() for x in ("k_new", "v_new"))
    for n in range(N):
        L = lens[n]
        idx = st["table"][n, :-(-L // page)].long()
        up = [set() for _ in range(M)]
        for m in range(M):
            p = par[n][m]
            if p == -1 or (0 <= p < m and up[p]):
                up[m] = (up[p] if p >= 0 else set()) | {m}
        seen = torch.tensor([[j in up[m] for j in range(M)] for m in range(M)], device="cuda")
        live = torch.tensor([bool(s) for s in up], device="cuda")
        for h in range(Hkv):
            K = torch.cat([st["k_cache"][idx, h].reshape(-1, d)[:L].double(), kn[n, :, h]])
            W = torch.cat([st["v_cache"][idx, h].reshape(-1, d)[:L].double(), vn[n, :, h]])
            qh = q[n, :, h * G:(h + 1) * G]                      # [M, G, d]
            s = (qh.reshape(M * G, d) @ K.T).view(M, G, L + M) * d ** -0.5
            s[..., L:].masked_fill_(~seen[:, None, :], -math.inf)
            l = torch.logsumexp(s, -1)
            w = torch.exp(s - torch.where(live[:, None], l, torch.zeros_like(l))[..., None])
            o = (w.view(M * G, -1) @ W).view(M, G, d)
            out[n, :, h * G:(h + 1) * G] = o * live[:, None, None]
            lse[n, :, h * G:(h + 1) * G] = l
    return {"out": out.view(N * M, Hq, d), "lse": lse.view(N * M, Hq)}


def _exact_append(st, c):
    N, M, page = c["N"], c["M"], c["page"]
    lens, count, table = st["lens"].tolist(), st["accept"].tolist(), st["table"].tolist()
    res = {}
    for name, new, cache in (("k", st["k_new"], st["k_cache"]), ("v", st["v_new"], st["v_cache"])):
        full = cache.double()
        for n in range(N):
            rows = new[n * M:(n + 1) * M].double()
            rows = rows[:count[n]] if st["path"] is None else rows[st["path"][n, :count[n]].long()]
            done = 0
            while done < count[n]:                                # page by page
                at = lens[n] + done
                slot = at % page
                take = min(page - slot, count[n] - done)
                full[table[n][at // page], :, slot:slot + take] = rows[done:done + take].transpose(0, 1)
                done += take
        res[name] = full
    return {"k": res["k"], "v": res["v"], "lens": None}
