"""Measured work of the operators around the softmax layers of a serving step.

A hybrid model (KDA layers with softmax-attention layers between them) that
serves a batch normalises and rotates the queries and keys of its softmax
layers, attends over a paged cache whose sequences often begin alike (a system
prompt, a document that many requests ask about), and draws the next tokens
from the last layer's logits.

    head_norm_rope    RMS norm of every query and key head and the rotation by its position
    prefix_attention  a softmax layer over shared prefixes, each sequence's own pages and its drafted nodes
    sample            temperature, top-k, top-p, min-p: the filtered distribution and a token drawn from it

``run`` computes the plain form with elementary torch operations where ``own``
is false, and calls the library's entry points where it is true.
"""
import math

import numpy as np
import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ESZ = {"bf16": 2, "f32": 4}


# ---------------------------------------------------------------------------- cases

def listed():
    return [
        # the token of a single user's step: latency
        dict(name="rope_one", op="head_norm_rope", T=1, Hq=32, Hkv=8, d=128, rot=128, pairs=False, fused=False,
             dt="bf16"),
        # prompts as long as the benchmark's packed documents together, 96 query heads, read out of
        # the projection that holds queries, keys and values side by side
        dict(name="rope_prompts", op="head_norm_rope", T=32388, Hq=96, Hkv=8, d=128, rot=128, pairs=False, fused=True,
             dt="bf16"),
        # fp32, half of each small head rotated, neighbouring channels as pairs, an odd count
        dict(name="rope_f32_odd", op="head_norm_rope", T=1777, Hq=12, Hkv=4, d=64, rot=32, pairs=True, fused=True,
             dt="f32"),
        # four users behind one short system prompt: latency
        dict(name="prefix_few_short", op="prefix_attention", N=4, M=1, Hq=32, Hkv=8, d=128, dt="bf16", P=1, plo=1000,
             phi=1000, lo=1, hi=60, page=16, shape="chain"),
        # a serving batch that asks about one long document
        dict(name="prefix_batch_long", op="prefix_attention", N=64, M=1, Hq=32, Hkv=8, d=128, dt="bf16", P=1, plo=65001,
             phi=65001, lo=1, hi=1024, page=64, shape="chain"),
        # drafted trees of a batch behind three system prompts, 12 query heads to a cache head
        dict(name="prefix_trees_three", op="prefix_attention", N=40, M=16, Hq=96, Hkv=8, d=128, dt="bf16", P=3, plo=5000,
             phi=9000, lo=0, hi=600, page=64, shape="tree"),
        # fp32, head size 64, a page size that divides no tile, trees shorter than the row
        dict(name="prefix_f32_odd", op="prefix_attention", N=9, M=5, Hq=12, Hkv=4, d=64, dt="f32", P=2, plo=700,
             phi=2100, lo=0, hi=300, page=24, shape="padded"),
        # one user's next token: latency
        dict(name="sample_one", op="sample", N=1, V=50257, dt="f32", k=True, p=True, m=False, mask=False, probs=False),
        # the decode batch of the benchmark, every user with settings of their own, an even vocabulary
        dict(name="sample_batch", op="sample", N=256, V=131072, dt="bf16", k=True, p=True, m=True, mask=False,
             probs=False),
        # nucleus alone, where nothing bounds the count of tokens that stay
        dict(name="sample_nucleus", op="sample", N=96, V=131072, dt="f32", k=False, p=True, m=False, mask=True,
             probs=False),
        # the target's distributions after every drafted node of a batch, as the verification takes them
        dict(name="sample_probs", op="sample", N=384, V=50257, dt="f32", k=True, p=True, m=False, mask=False, probs=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["head_norm_rope", "prefix_attention", "prefix_attention", "sample", "sample"])
    dt = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if op == "head_norm_rope":
        while True:
            Hkv = rng.choice([1, 2, 4, 8, 16])
            d = rng.choice([16, 32, 64, 128, 128, 128])
            c = dict(op=op, T=_log(rng, 1, 32388), Hq=Hkv * rng.choice([1, 2, 3, 4, 8, 12]), Hkv=Hkv, d=d,
                     rot=rng.choice([d, d, d // 2, d // 4 + 2]), pairs=rng.random() < 0.4, fused=rng.random() < 0.5,
                     dt=dt)
            if c["T"] * (c["Hq"] + 2 * Hkv) * d * ESZ[dt] <= 32388 * 112 * 128 * 2:
                return c
    if op == "prefix_attention":
        while True:
            Hkv = rng.choice([1, 2, 4, 8, 16])
            phi, N = _log(rng, 1, 131072), _log(rng, 1, 128)
            c = dict(op=op, N=N, M=_log(rng, 1, 32), Hq=Hkv * rng.choice([1, 2, 3, 4, 8, 12, 16]), Hkv=Hkv,
                     d=rng.choice([64, 128, 128, 128]), dt=dt, P=rng.randint(1, min(N, 4)), plo=rng.choice([0, phi // 2, phi]),
                     phi=phi, lo=0, hi=_log(rng, 1, 4096), page=rng.choice([16, 32, 64, 64, 128, 24, 256]),
                     shape=rng.choice(["tree", "chain", "padded"]))
            tokens = c["P"] * phi + N * c["hi"]
            if N * c["M"] * c["Hq"] * c["d"] * (phi + c["hi"]) <= (5.5e10 if dt == "bf16" else 5e9) \
                    and tokens * Hkv * c["d"] <= 131072 * 8 * 128:
                return c
    while True:
        c = dict(op=op, N=_log(rng, 1, 256), V=_log(rng, 1000, 200000), dt=rng.choice(["bf16", "f32"]),
                 k=rng.random() < 0.5, p=rng.random() < 0.6, m=rng.random() < 0.3, mask=rng.random() < 0.3,
                 probs=rng.random() < 0.4)
        if c["N"] * c["V"] <= 384 * 50257:
            return c


# ---------------------------------------------------------------------------- inputs

def _parents(case, rs):
    """[N, M] int32: trees whose nodes branch often near the root, chains, or trees of 1..M nodes."""
    N, M = case["N"], case["M"]
    m = np.arange(M)
    if case["shape"] == "chain":
        par = np.broadcast_to(m - 1, (N, M)).copy()
    else:
        par = np.floor(rs.random_sample((N, M)) ** 0.7 * m).astype(np.int64)
        par[:, 0] = -1
    if case["shape"] == "padded":
        par[m[None, :] >= rs.randint(1, M + 1, (N, 1))] = -2
    return par.astype(np.int32)


def prepare(case, seed):
    rs = np.random.RandomState(seed % (1 << 32))
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dt = DT[case["dt"]]
    randn = lambda *s: torch.randn(s, generator=gen, device="cuda")
    rand = lambda *s: torch.rand(s, generator=gen, device="cuda")
    dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).cuda()
    st = {"case": case}
    if case["op"] == "head_norm_rope":
        T, Hq, Hkv, d, rot = (case[x] for x in ("T", "Hq", "Hkv", "d", "rot"))
        if case["fused"]:
            qkv = (randn(T, Hq + 2 * Hkv, d) * 2.0).to(dt)
            st["q"], st["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
        else:
            st["q"], st["k"] = (randn(T, Hq, d) * 2.0).to(dt), (randn(T, Hkv, d) * 2.0).to(dt)
        st["q_weight"], st["k_weight"] = 1.0 + 0.2 * randn(d), 1.0 + 0.2 * randn(d)
        st["inv_freq"] = dev((500000.0 ** (-np.arange(rot // 2) / (rot / 2.0))).astype(np.float32))
        # documents (or sequences of one token) anywhere in a context of 262,144
        pos, at = np.empty(T, np.int32), 0
        while at < T:
            n = min(T - at, int(rs.randint(1, 8193)) if T > 64 else 1)
            pos[at:at + n] = int(rs.randint(0, 262144 - n)) + np.arange(n)
            at += n
        st["positions"] = dev(pos)
        return st
    if case["op"] == "prefix_attention":
        N, M, Hq, Hkv, d, P, page = (case[x] for x in ("N", "M", "Hq", "Hkv", "d", "P", "page"))
        lens = rs.randint(case["lo"], case["hi"] + 1, N).astype(np.int32)
        plens = rs.randint(case["plo"], case["phi"] + 1, P).astype(np.int32)
        cut = np.sort(rs.permutation(N - 1)[:P - 1] + 1) if P > 1 else np.zeros(0, np.int64)
        st["prefix_seqs"] = dev(np.concatenate([[0], cut, [N]]).astype(np.int32))
        own_w, pre_w = max(1, -(-case["hi"] // page)), max(1, -(-case["phi"] // page))
        need = int(sum(-(-int(x) // page) for x in lens) + sum(-(-int(x) // page) for x in plens))
        order, at = rs.permutation(need + 3).astype(np.int32), 0
        tables = [np.zeros((N, own_w), np.int32), np.zeros((P, pre_w), np.int32)]
        for table, ls in zip(tables, (lens, plens)):
            for i, x in enumerate(ls):
                c = -(-int(x) // page)
                table[i, :c] = order[at:at + c]
                at += c
        st["table"], st["prefix_table"] = dev(tables[0]), dev(tables[1])
        st["lens"], st["prefix_lens"], st["parent"] = dev(lens), dev(plens), dev(_parents(case, rs))
        st["q"] = (randn(N * M, Hq, d) * 1.5).to(dt)
        st["k_new"], st["v_new"] = randn(N * M, Hkv, d).to(dt), randn(N * M, Hkv, d).to(dt)
        for name in ("k_cache", "v_cache"):
            x = torch.empty((need + 3, Hkv, page, d), dtype=dt, device="cuda")
            x.normal_(generator=gen)
            st[name] = x
        return st
    N, V = case["N"], case["V"]
    # some rows are nearly certain, some nearly flat
    logits = randn(N, V) * (1.0 + 2.5 * rand(N, 1))
    if case["mask"]:
        # a grammar that allows two tokens in three, in half of the rows
        off = (rand(N, V) < 1 / 3) & (rand(N, 1) < 0.5)
        logits.masked_fill_(off, -math.inf)
    st["logits"] = logits.to(dt)
    st["u"] = rand(N)
    temp = 0.5 + rand(N)
    st["temperature"] = torch.where(rand(N) < 0.05, torch.zeros_like(temp), temp)      # some decode greedily
    pick = lambda vals: dev(np.asarray(vals, np.int32)[rs.randint(0, len(vals), N)])
    st["top_k"] = pick([0, 1, 20, 40, 50, 100, 1000]) if case["k"] else None
    st["top_p"] = 0.5 + 0.5 * rand(N) if case["p"] else None
    st["min_p"] = rand(N) * 0.1 if case["m"] else None
    return st


# ---------------------------------------------------------------------------- one pass

def run(st):
    op = st["case"]["op"]
    if own:
        return _run_own(st, op)
    return {"head_norm_rope": _plain_rope, "prefix_attention": _plain_attention, "sample": _plain_sample}[op](st)


def _run_own(st, op):
    from linear_attention_03_gb300 import kda
    if op == "head_norm_rope":
        q, k = kda.kda_head_norm_rope(st["q"], st["k"], st["positions"], st["inv_freq"], q_weight=st["q_weight"],
                                      k_weight=st["k_weight"], interleaved=st["case"]["pairs"])
        return {"q": q, "k": k}
    if op == "prefix_attention":
        out, lse = kda.kda_prefix_attention(st["q"], st["k_new"], st["v_new"], st["k_cache"], st["v_cache"],
                                            st["prefix_table"], st["prefix_lens"], st["prefix_seqs"], st["table"],
                                            st["lens"], st["parent"], want_lse=True)
        return {"out": out, "lse": lse}
    token, probs = kda.kda_sample(st["logits"], st["u"], temperature=st["temperature"], top_k=st["top_k"],
                                  top_p=st["top_p"], min_p=st["min_p"], want_probs=st["case"]["probs"])
    return {"token": token, "probs": probs} if st["case"]["probs"] else {"token": token}


def _plain_rope(st):
    c = st["case"]
    half = c["rot"] // 2
    angle = st["positions"].double()[:, None] * st["inv_freq"].double()      # far positions: 32 bits are too few
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]
    res = {}
    for name in ("q", "k"):
        x = st[name].float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * st[name + "_weight"]
        if c["pairs"]:
            a, b = x[..., 0:c["rot"]:2], x[..., 1:c["rot"]:2]
        else:
            a, b = x[..., :half], x[..., half:c["rot"]]
        y = x.clone()
        ra, rb = a * cos - b * sin, b * cos + a * sin
        if c["pairs"]:
            y[..., 0:c["rot"]:2], y[..., 1:c["rot"]:2] = ra, rb
        else:
            y[..., :half], y[..., half:c["rot"]] = ra, rb
        res[name] = y.to(st[name].dtype)
    return res


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
    """Each prefix once for all its sequences, then what each sequence has of its own, joined by their sums."""
    c = st["case"]
    N, M, Hq, Hkv, d, page = (c[x] for x in ("N", "M", "Hq", "Hkv", "d", "page"))
    G = Hq // Hkv
    lens, plens, seqs = st["lens"].tolist(), st["prefix_lens"].tolist(), st["prefix_seqs"].tolist()
    anc = _ancestors(st["parent"])
    q = st["q"].float().view(N, M, Hkv, G, d)
    kn, vn = st["k_new"].float().view(N, M, Hkv, d), st["v_new"].float().view(N, M, Hkv, d)

    def gather(cache, pages, L, h):                                       # [L, d] of one head
        idx = pages[:max(1, -(-L // page))].long()
        return cache[idx, h].reshape(-1, d)[:L].float()

    def part(s, v):                                                       # maximum, sum and weighted values
        top = s.amax(-1, keepdim=True)
        top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
        e = torch.exp(s - top)
        return top, e.sum(-1, keepdim=True), torch.matmul(e, v)

    pre_o = torch.zeros((N, M, Hkv, G, d), device="cuda")
    pre_z = torch.zeros((N, M, Hkv, G, 1), device="cuda")
    pre_t = torch.full((N, M, Hkv, G, 1), -math.inf, device="cuda")
    for p, L in enumerate(plens):
        a, b = seqs[p], seqs[p + 1]
        if L == 0 or a == b:
            continue
        for h in range(Hkv):
            K = gather(st["k_cache"], st["prefix_table"][p], L, h)
            s = torch.matmul(q[a:b, :, h].reshape(-1, d), K.t()) / math.sqrt(d)
            t, z, o = part(s, gather(st["v_cache"], st["prefix_table"][p], L, h))
            pre_t[a:b, :, h], pre_z[a:b, :, h] = t.view(b - a, M, G, 1), z.view(b - a, M, G, 1)
            pre_o[a:b, :, h] = o.view(b - a, M, G, d)
    out = torch.empty((N, M, Hkv, G, d), device="cuda")
    lse = torch.empty((N, M, Hkv, G), device="cuda")
    for n in range(N):
        L = lens[n]
        idx = st["table"][n, :max(1, -(-L // page))].long()
        mine = lambda x: x[idx].transpose(0, 1).reshape(Hkv, -1, d)[:, :L].float()
        K = torch.cat([mine(st["k_cache"]), kn[n].transpose(0, 1)], 1)
        W = torch.cat([mine(st["v_cache"]), vn[n].transpose(0, 1)], 1)
        qn = q[n].permute(1, 0, 2, 3).reshape(Hkv, M * G, d)
        s = torch.matmul(qn, K.transpose(1, 2)) / math.sqrt(d)
        vis = anc[n][:, None, :].expand(M, G, M).reshape(M * G, M)
        s[..., L:] = s[..., L:].masked_fill(~vis, -math.inf)
        t, z, o = (x.view(Hkv, M, G, -1).permute(1, 0, 2, 3) for x in part(s, W))
        top = torch.maximum(t, pre_t[n])
        e1, e2 = torch.exp(t - top), torch.exp(pre_t[n] - top)
        z = e1 * z + e2 * pre_z[n]
        on = anc[n].any(-1)[:, None, None, None]
        out[n] = torch.where(on, (e1 * o + e2 * pre_o[n]) / z, torch.zeros_like(o))
        lse[n] = torch.where(on, top + torch.log(z), torch.full_like(z, -math.inf))[..., 0]
    return {"out": out.view(N * M, Hq, d).to(st["q"].dtype), "lse": lse.view(N * M, Hq)}


def _plain_sample(st):
    """Weights exp((x - max) / T) in 64 bits: a 32-bit sum of a vocabulary moves what stays and what is drawn."""
    x, V = st["logits"].double(), st["case"]["V"]
    N = x.shape[0]
    T = st["temperature"].double()[:, None]
    greedy = T <= 0
    order = torch.sort(x, dim=-1, descending=True, stable=True)           # ties: the lowest index first
    xs = order.values
    d = xs - xs[:, :1]
    w = torch.where(greedy, (torch.arange(V, device="cuda") == 0)[None].double(),
                    torch.exp(d / torch.where(greedy, torch.ones_like(T), T)))
    rank = torch.arange(V, device="cuda")[None]
    keep = torch.ones((N, V), dtype=torch.bool, device="cuda")
    if st["top_k"] is not None:
        k = st["top_k"].long()[:, None]
        keep = (rank < k) | (k <= 0)
    if st["top_p"] is not None:
        wk = w * keep
        before = wk.cumsum(-1) - wk
        keep = keep & ((before < st["top_p"].double()[:, None] * wk.sum(-1, keepdim=True)) | (rank == 0))
    if st["min_p"] is not None:
        keep = keep & (w >= st["min_p"].double()[:, None])
    w = torch.zeros_like(w).scatter_(1, order.indices, w * keep)          # back in the vocabulary's order
    cum = w.cumsum(-1)
    total = cum[:, -1:]
    token = (cum <= st["u"].double()[:, None] * total).sum(-1).int()
    if st["case"]["probs"]:
        return {"token": token, "probs": (w / total).float()}
    return {"token": token}


# ---------------------------------------------------------------------------- floors

def work(case):
    op, e = case["op"], ESZ[case["dt"]]
    if op == "head_norm_rope":
        n = case["T"] * (case["Hq"] + case["Hkv"]) * case["d"]
        return {"bytes": 2 * n * e + case["T"] * 4, "flops": 8 * n}
    if op == "prefix_attention":
        N, M, Hq, Hkv, d = (case[x] for x in ("N", "M", "Hq", "Hkv", "d"))
        pre, mine = (case["plo"] + case["phi"]) / 2, (case["lo"] + case["hi"]) / 2
        return {"bytes": int((case["P"] * pre + N * mine) * Hkv * d * 2 * e
                             + N * M * ((2 * Hq + 2 * Hkv) * d * e + Hq * 4)),
                "flops": int(4 * (pre + mine + 1) * N * M * Hq * d)}
    return {"bytes": case["N"] * case["V"] * (e + (4 if case["probs"] else 0)), "flops": 4 * case["N"] * case["V"]}


# ---------------------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """The definition in fp64; tokens are whole numbers and have no such value."""
    op = case["op"]
    if op == "sample" and not case["probs"]:
        return None
    st = prepare(case, seed)
    return {"head_norm_rope": _exact_rope, "prefix_attention": _exact_attention, "sample": _exact_sample}[op](st, case)


def _exact_rope(st, c):
    rot = c["rot"]
    # each pair as a complex number, turned by e^(i angle)
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda").expand(c["T"], rot // 2).contiguous(),
                       torch.outer(st["positions"].double(), st["inv_freq"].double()))
    res = {}
    for name in ("q", "k"):
        x = st[name].double()
        y = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / c["d"] + 1e-6) * st[name + "_weight"].double()
        head = y[..., :rot]
        if c["pairs"]:
            z = torch.view_as_complex(head.unflatten(-1, (rot // 2, 2)).contiguous()) * turn[:, None]
            head = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(*head.unflatten(-1, (2, rot // 2)).unbind(-2)) * turn[:, None]
            head = torch.cat([z.real, z.imag], -1)
        res[name] = torch.cat([head, y[..., rot:]], -1)
    return res


def _exact_attention(st, c):
    """Every sequence by itself over the whole line of its tokens."""
    N, M, Hq, Hkv, d, page = (c[x] for x in ("N", "M", "Hq", "Hkv", "d", "page"))
    if N * M * Hq * d * (c["phi"] + c["hi"]) > 2e11:
        return None
    G = Hq // Hkv
    par, lens, plens, seqs = (st[x].tolist() for x in ("parent", "lens", "prefix_lens", "prefix_seqs"))
    out = torch.zeros((N, M, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((N, M, Hq), -math.inf, dtype=torch.float64, device="cuda")
    q = st["q"].view(N, M, Hq, d).double()
    kn, vn = (st[x].view(N, M, Hkv, d).double() for x in ("k_new", "v_new"))
    for p in range(c["P"]):
        pages = st["prefix_table"][p, :-(-plens[p] // page)].long()
        for h in range(Hkv):
            pk, pv = (st[x][pages, h].reshape(-1, d)[:plens[p]].double() for x in ("k_cache", "v_cache"))
            for n in range(seqs[p], seqs[p + 1]):
                idx = st["table"][n, :-(-lens[n] // page)].long()
                line = lambda pre, cache, new: torch.cat([pre, cache[idx, h].reshape(-1, d)[:lens[n]].double(), new[n, :, h]])
                K, W = line(pk, st["k_cache"], kn), line(pv, st["v_cache"], vn)
                for m in range(M):
                    up, at = [], m                               # the node and those above it
                    while at >= 0:
                        up.append(at)
                        nxt = par[n][at]
                        if nxt != -1 and not 0 <= nxt < at:
                            up = []
                            break
                        at = nxt
                    if not up:
                        continue
                    s = (q[n, m, h * G:(h + 1) * G] @ K.T) * d ** -0.5
                    hidden = torch.ones(M, dtype=torch.bool)
                    hidden[up] = False
                    s[:, len(K) - M:].masked_fill_(hidden.cuda(), -math.inf)
                    l = torch.logsumexp(s, -1)
                    out[n, m, h * G:(h + 1) * G] = torch.exp(s - l[:, None]) @ W
                    lse[n, m, h * G:(h + 1) * G] = l
    return {"out": out.view(N * M, Hq, d), "lse": lse.view(N * M, Hq)}


def _exact_sample(st, c):
    """Row by row on the host."""
    probs = np.zeros((c["N"], c["V"]))
    rows = st["logits"].float().cpu().numpy().astype(np.float64)
    T = st["temperature"].cpu().numpy().astype(np.float64)
    par = {x: None if st[x] is None else st[x].cpu().numpy() for x in ("top_k", "top_p", "min_p")}
    for n, x in enumerate(rows):
        best = np.lexsort((np.arange(c["V"]), -x))                # by value, then by index
        if T[n] <= 0:
            probs[n, best[0]] = 1.0
            continue
        if par["top_k"] is not None and par["top_k"][n] > 0:
            best = best[:par["top_k"][n]]
        w = np.exp((x[best] - x[best[0]]) / T[n])
        if par["top_p"] is not None:
            ends = np.add.accumulate(w) >= float(par["top_p"][n]) * w.sum()
            count = int(np.argmax(ends)) + 1 if ends.any() else len(w)
            best, w = best[:count], w[:count]
        if par["min_p"] is not None:
            stay = w >= float(par["min_p"][n])
            best, w = best[stay], w[stay]
        probs[n, best] = w / w.sum()
    return {"token": None, "probs": torch.from_numpy(probs).cuda()}
