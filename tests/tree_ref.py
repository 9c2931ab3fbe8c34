"""Plain fp64 / whole-number implementations of the tree-drafted decoding
operators, written from their definitions (numpy, loops), and the inputs of
their tests."""
import numpy as np
import torch

ONE = 1 << 38


def lines(parent):
    """For each node of one sequence the list of nodes on its line (root first), [] for no node."""
    out = []
    for m, p in enumerate(parent):
        if p == -1:
            out.append([m])
        elif 0 <= p < m and out[p]:
            out.append(out[p] + [m])
        else:
            out.append([])
    return out


def kda_step(S, k, v, g, beta):
    """S [H, dk, dv]; k, g [H, dk]; v [H, dv]; beta [H]."""
    S = np.exp(g)[:, :, None] * S
    u = beta[:, None] * (v - np.einsum("hk,hkv->hv", k, S))
    return S + k[:, :, None] * u[:, None, :]


def decode_tree(q, k, v, g, beta, state, parent):
    N, M = parent.shape
    H, d = q.shape[1:]
    sh = lambda x: x.reshape(N, M, *x.shape[1:])
    q, k, v, g, beta = map(sh, (q, k, v, g, beta))
    out = np.zeros((N, M, H, d))
    for n in range(N):
        S = {-1: state[n]}
        for m, line in enumerate(lines(parent[n])):
            if line:
                S[m] = kda_step(S[parent[n, m]], k[n, m], v[n, m], g[n, m], beta[n, m])
                out[n, m] = np.einsum("hk,hkv->hv", q[n, m], S[m])
    return out.reshape(N * M, H, d)


def decode_commit(k, v, g, beta, state, path, accept):
    N, P = path.shape
    M = k.shape[0] // N
    out = state.copy()
    for n in range(N):
        for t in range(min(max(accept[n], 0), P)):
            m = path[n, t]
            if not 0 <= m < M:
                break
            r = n * M + m
            out[n] = kda_step(out[n], k[r], v[r], g[r], beta[r])
    return out


def attention(q, k_new, v_new, k_cache, v_cache, table, lens, parent, scale):
    """(out, lse, weight) with weight = sum_j p_j |v_j|, the scale of rounding errors in out."""
    N, M = parent.shape
    H, d = q.shape[1:]
    Hkv, page = k_cache.shape[1:3]
    G = H // Hkv
    out, wt = np.zeros((N * M, H, d)), np.zeros((N * M, H, d))
    lse = np.full((N * M, H), -np.inf)
    for n in range(N):
        pos = np.arange(lens[n])
        K0, V0 = (c[table[n][pos // page], :, pos % page] for c in (k_cache, v_cache))   # [L, Hkv, d]
        for m, line in enumerate(lines(parent[n])):
            if not line:
                continue
            rows = [n * M + j for j in line]
            K, V = np.concatenate([K0, k_new[rows]]), np.concatenate([V0, v_new[rows]])
            for h in range(H):
                s = scale * (K[:, h // G] @ q[n * M + m, h])
                top = s.max()
                e = np.exp(s - top)
                lse[n * M + m, h] = top + np.log(e.sum())
                out[n * M + m, h] = e @ V[:, h // G] / e.sum()
                wt[n * M + m, h] = e @ np.abs(V[:, h // G]) / e.sum()
    return out, lse, wt


def fixed(p):
    """Probabilities (float32 values) as whole multiples of 2^-38, toward zero."""
    p = np.asarray(p, np.float32)
    return (np.clip(np.nan_to_num(p, nan=0.0), 0, 1).astype(np.float64) * ONE).astype(np.int64)


def tick(u):
    return min(int(max(float(u), 0.0) * (1 << 24)), (1 << 24) - 1)


def verify(target, tokens, parent, uniforms, draft=None):
    """Float32 arrays; Python integers throughout the draws."""
    N, M, V = target.shape
    accept, path, nxt = np.zeros(N, np.int64), np.full((N, M), -1), np.full(N, -1)
    for n in range(N):
        if parent[n, 0] != -1:
            continue
        kept, cur = [0], 0
        while True:
            refused, spent, into = [], 0, None
            for m in [m for m in range(1, M) if parent[n, m] == cur and m > cur]:
                t = int(tokens[n, m])
                ok = 0 <= t < V
                if draft is not None:
                    take = ok and not refused and \
                        np.float32(uniforms[n, cur]) * draft[n, cur, t] < target[n, cur, t]
                else:
                    mass = int(fixed(target[n, cur, t])) if ok and t not in refused else 0
                    take = (tick(uniforms[n, cur]) << 14) < spent + mass
                    spent += 0 if take else mass
                if take:
                    into = m
                    break
                refused.append(t)
            if into is None:
                break
            kept.append(into)
            cur = into
        row = fixed(target[n, cur])
        w = row.copy()
        if refused and draft is not None:
            w = fixed(target[n, cur] - draft[n, cur])
        elif refused:
            w[[t for t in refused if 0 <= t < V]] = 0
        if not w.any():
            w = row
        total = int(w.sum())
        if total:
            need = (tick(uniforms[n, M]) * total) >> 24
            nxt[n] = int(np.searchsorted(np.cumsum(w), need, side="right"))
        accept[n] = len(kept)
        path[n, :len(kept)] = kept
    return accept, path, nxt


def append(k_new, v_new, k_cache, v_cache, table, lens, path, accept):
    k_cache, v_cache = k_cache.clone(), v_cache.clone()
    N, M, page = len(lens), k_new.shape[0] // len(lens), k_cache.shape[2]
    P = M if path is None else path.shape[1]
    out = lens.copy()
    for n in range(N):
        a = P if accept is None else min(max(int(accept[n]), 0), P)
        out[n] += a
        for t in range(a):
            m = t if path is None else int(path[n, t])
            pos = int(lens[n]) + t
            if not 0 <= m < M or pos // page >= table.shape[1]:
                continue
            pg = int(table[n, pos // page])
            if 0 <= pg < len(k_cache):
                k_cache[pg, :, pos % page] = k_new[n * M + m]
                v_cache[pg, :, pos % page] = v_new[n * M + m]
    return k_cache, v_cache, out


# ------------------------------------------------------------------ inputs

def parents(N, M, kind, rng):
    par = np.floor(rng.random((N, M)) ** 0.7 * np.arange(M)).astype(np.int32)
    par[:, 0] = -1
    if kind == "chain":
        par[:] = np.arange(M) - 1
    elif kind == "star":
        par[:] = 0
        par[:, 0] = -1
    elif kind == "forest":                       # several nodes directly below the prefix
        par[rng.random((N, M)) < 0.3] = -1
    elif kind == "holes":                        # no node in any places, and what hangs below
        par[rng.random((N, M)) < 0.3] = -2
    elif kind == "odd":                          # values that name no node
        par[:, M // 2] = M // 2
        par[:, -1] = 1000
    elif kind == "none":
        par[:] = -2
    return par


def kda_inputs(N, M, H, d, dtype, rng):
    f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32))
    unit = lambda x: x / x.norm(dim=-1, keepdim=True)
    return dict(q=unit(f(N * M, H, d)).to(dtype), k=unit(f(N * M, H, d)).to(dtype),
                v=f(N * M, H, d).to(dtype), g=-5 * torch.sigmoid(f(N * M, H, d)),
                beta=torch.sigmoid(f(N * M, H)), state=f(N, H, d, d) * 0.3)


def cache_inputs(N, M, H, Hkv, d, page, lens, dtype, rng, spare=3):
    """Pages in random order; everything past a length holds NaN."""
    f = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(dtype)
    per = [max(1, -(-int(x) // page)) for x in lens]
    pool = sum(per) + spare
    order = rng.permutation(pool).astype(np.int32)
    table = np.full((N, max(per)), 2 ** 30, np.int32)        # never to be read past a length
    k, v = f(pool, Hkv, page, d), f(pool, Hkv, page, d)
    at = 0
    used = torch.zeros(pool, page, dtype=torch.bool)
    for n, c in enumerate(per):
        table[n, :c] = order[at:at + c]
        at += c
        for t in range(int(lens[n])):
            used[table[n, t // page], t % page] = True
    bad = ~used[:, None, :, None].expand_as(k)
    k[bad] = float("nan")
    v[bad] = float("nan")
    return dict(q=f(N * M, H, d) * 1.5, k_new=f(N * M, Hkv, d), v_new=f(N * M, Hkv, d), k_cache=k, v_cache=v,
                page_table=torch.from_numpy(table), cache_lens=torch.from_numpy(np.asarray(lens, np.int32)))
