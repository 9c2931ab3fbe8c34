"""Plain fp64 implementations of the operators around the softmax layers of a
serving step, written from their definitions (numpy, loops), and the inputs of
their tests."""
import numpy as np

from tests import tree_ref


def norm_rope(x, positions, inv_freq, weight=None, eps=1e-6, interleaved=False):
    """x [T, H, d] -> (y, size): the result and |a| + |b| of each element's pair before the turn."""
    T, H, d = x.shape
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if weight is not None:
        y = y * weight
    out, size = y.copy(), np.abs(y)
    for i, f in enumerate(inv_freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + len(inv_freq))
        for t, p in enumerate(positions):
            # exact: an fp32 frequency times an integer fits 64 bits of significand
            angle = float(np.fmod(np.longdouble(float(f)) * int(p), 2 * PI))
            c, s = np.cos(angle), np.sin(angle)
            out[t, :, a] = y[t, :, a] * c - y[t, :, b] * s
            out[t, :, b] = y[t, :, b] * c + y[t, :, a] * s
            size[t, :, a] = size[t, :, b] = np.abs(y[t, :, a]) + np.abs(y[t, :, b])
    return out, size


# pi to the 64 bits of the extended type (on machines where that is a double, angles are taken there)
PI = np.longdouble("3.14159265358979323846264338327950288")


def prefix_attention(q, k_new, v_new, k_cache, v_cache, ptable, plens, seqs, table, lens, parent, scale):
    """(out, lse, weight) as tree_ref.attention, over each sequence's prefix, own keys and line."""
    N, M = parent.shape
    H, d = q.shape[1:]
    Hkv, page = k_cache.shape[1:3]
    G = H // Hkv
    out, wt = np.zeros((N * M, H, d)), np.zeros((N * M, H, d))
    lse = np.full((N * M, H), -np.inf)

    def keys(pages, count):
        pos = np.arange(count)
        return [c[pages[pos // page], :, pos % page] for c in (k_cache, v_cache)]       # [count, Hkv, d]

    for n in range(N):
        own = keys(table[n], lens[n])
        for p in range(len(plens)):
            if seqs[p] <= n < seqs[p + 1]:
                own = [np.concatenate([a, b]) for a, b in zip(keys(ptable[p], plens[p]), own)]
        for m, line in enumerate(tree_ref.lines(parent[n])):
            if not line:
                continue
            rows = [n * M + j for j in line]
            K, V = np.concatenate([own[0], k_new[rows]]), np.concatenate([own[1], v_new[rows]])
            for h in range(Hkv):
                at = slice(h * G, (h + 1) * G)
                s = scale * (q[n * M + m, at] @ K[:, h].T)
                top = s.max(-1, keepdims=True)
                e = np.exp(s - top)
                z = e.sum(-1, keepdims=True)
                lse[n * M + m, at] = (top + np.log(z))[:, 0]
                out[n * M + m, at] = e @ V[:, h] / z
                wt[n * M + m, at] = e @ np.abs(V[:, h]) / z
    return out, lse, wt


def prefix_inputs(N, M, H, Hkv, d, page, lens, plens, seqs, dtype, rng):
    """Pages of all sequences and prefixes in one pool in random order; what is past a length holds NaN."""
    import torch
    x = tree_ref.cache_inputs(N + len(plens), M, H, Hkv, d, page, list(lens) + list(plens), dtype, rng)
    for name in ("q", "k_new", "v_new"):
        x[name] = x[name][:N * M].contiguous()
    table, all_lens = x.pop("page_table"), x.pop("cache_lens")
    x.update(page_table=table[:N].contiguous(), prefix_table=table[N:].contiguous(), cache_lens=all_lens[:N].contiguous(),
             prefix_lens=all_lens[N:].contiguous(), prefix_seqs=torch.from_numpy(np.asarray(seqs, np.int32)))
    return x


def sample_row(x, u=None, T=1.0, k=0, p=1.0, m=0.0, tol=0.0, first=None):
    """One row (float64 values of the logits): (token, probs), from the definition.  `tol` moves the
    weight that top-p asks for, relative to it; `first` is how many it leaves."""
    V = len(x)
    x = np.where(np.isnan(x), -np.inf, x)
    if np.isposinf(x).any():
        x = np.where(np.isposinf(x), 0.0, -np.inf)
    top = x.max()
    probs = np.zeros(V)
    if np.isneginf(top):
        return -1, probs
    order = np.lexsort((np.arange(V), -x))
    if not T > 0:
        order, T = order[:1], 1.0
    w = np.exp((x - top) / T)
    if 0 < k < V:
        order = order[:k]
    if p < 1:
        mass = w[order]
        before = np.concatenate([[0.0], np.cumsum(mass)[:-1]])
        on = before < max(p, 0.0) * mass.sum() * (1 + tol)
        on[0] = True
        order = order[on] if first is None else order[:first]
    if m > 0:
        order = order[w[order] >= min(m, 1.0)]
    probs[order] = w[order]
    total = probs.sum()
    token = None
    if u is not None:
        token = int(np.searchsorted(np.cumsum(probs), u * total, side="right"))
    return token, probs / total
