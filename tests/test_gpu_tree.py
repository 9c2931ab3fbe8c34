"""The operators of tree-drafted decoding against plain fp64 implementations
(tests/tree_ref.py), and their refusals.

Tolerances, from the roundings that each path makes:
  * decode_tree / decode_commit in fp32: tests/kda_testlib.py (1e-4); bf16
    outputs: half a bf16 ulp of the result (its one rounding, 2^-9 relative)
    plus 2^-10 of the outputs' RMS for the fp32 or split-operand sums.
    States of bf16 inputs are computed and stored in fp32: 1e-4 as well.
  * tree_attention: the output's rounding (bf16: 2^-8 |out|, one ulp; fp32: none)
    plus, against sum_j p_j |v_j|, the rounding of the weights p to bf16
    (2^-9, taken twice) or, in fp32, 2e-5 (scores up to ~30 carry ~30 2^-24
    sqrt(d) of absolute error into the exponent).  lse: 2e-5 + 2e-6 |lse|
    in fp32; bf16 inputs give exact products, so the same.
  * verify_drafts and cache_append: equal.
"""
import math

import numpy as np
import pytest
import torch

from tests import tree_ref as ref
from tests.kda_testlib import compare, f64, half_ulp_bf16, rms

gpu = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]
pytestmark = gpu

BF, F32 = torch.bfloat16, torch.float32
cu = lambda d: {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in d.items()}
i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def check_kda(got, want, dtype, what):
    if dtype == F32 or got.dtype == F32:
        return compare(got, want, F32, what)
    diff = np.abs(f64(got) - want)
    bound = half_ulp_bf16(want) * 1.01 + 2.0 ** -10 * max(rms(want), 1e-30)
    assert np.isfinite(f64(got)).all() and (diff <= bound).all(), (what, float((diff - bound).max()))


# ------------------------------------------------------------------ decode_tree

TREES = [(1, 1, 1, 128, BF, "chain"), (2, 2, 3, 128, BF, "chain"), (3, 16, 5, 128, BF, "tree"),
         (2, 17, 2, 128, BF, "holes"), (1, 64, 2, 128, BF, "chain"), (2, 64, 3, 128, BF, "tree"),
         (2, 33, 2, 128, BF, "star"), (3, 8, 4, 128, BF, "forest"), (2, 7, 2, 128, BF, "odd"),
         (2, 5, 2, 128, BF, "none"), (2, 48, 1, 128, BF, "holes"), (3, 15, 2, 128, F32, "tree"),
         (2, 64, 1, 128, F32, "chain"), (3, 13, 4, 64, F32, "holes"), (2, 9, 3, 64, BF, "tree"),
         (2, 20, 3, 32, F32, "forest"), (2, 6, 5, 16, F32, "tree"), (2, 31, 2, 16, BF, "odd")]


@pytest.mark.parametrize("N,M,H,d,dtype,kind", TREES)
def test_decode_tree(kda, N, M, H, d, dtype, kind):
    rng = np.random.default_rng(N * 1000 + M * 10 + d)
    x, par = ref.kda_inputs(N, M, H, d, dtype, rng), ref.parents(N, M, kind, rng)
    c = cu(x)
    before = c["state"].clone()
    out = kda.kda_decode_tree(c["q"], c["k"], c["v"], c["g"], c["beta"], c["state"], i32(par))
    want = ref.decode_tree(*(f64(x[n]) for n in ("q", "k", "v", "g", "beta", "state")), par)
    check_kda(out, want, dtype, f"tree {N}x{M} {kind}")
    assert torch.equal(before, c["state"])
    empty = np.array([[not l for l in ref.lines(p)] for p in par]).reshape(-1)
    assert (out[torch.from_numpy(empty).cuda()] == 0).all()


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (BF, 32), (BF, 16), (F32, 128), (F32, 64), (F32, 32),
                                     (F32, 16)])
@pytest.mark.parametrize("M", [1, 4, 5, 8, 9, 16, 24, 32, 33, 64])
def test_decode_tree_at_each_size(kda, M, d, dtype):
    """Node counts at and around the row tiles, and units that share a CTA with none left over and some."""
    for N, H, kind in ((3, 7, "holes"), (1, 1, "tree")):
        rng = np.random.default_rng(M * 10 + d + N)
        x, par = ref.kda_inputs(N, M, H, d, dtype, rng), ref.parents(N, M, kind, rng)
        c = cu(x)
        out = kda.kda_decode_tree(c["q"], c["k"], c["v"], c["g"], c["beta"], c["state"], i32(par))
        want = ref.decode_tree(*(f64(x[n]) for n in ("q", "k", "v", "g", "beta", "state")), par)
        check_kda(out, want, dtype, f"tree {N}x{M} {kind}")


def test_decode_tree_chain_is_decode_verify(kda):
    """A chain gives kda_decode_verify's outputs: fp32 inputs, 1e-4."""
    rng = np.random.default_rng(5)
    N, M, H, d = 3, 6, 4, 128
    c = cu(ref.kda_inputs(N, M, H, d, F32, rng))
    par = i32(ref.parents(N, M, "chain", rng))
    out = kda.kda_decode_tree(c["q"], c["k"], c["v"], c["g"], c["beta"], c["state"], par)
    want, state = kda.kda_decode_verify(c["q"], c["k"], c["v"], c["g"], c["beta"], c["state"],
                                        i32([4, 0, 6]), M)
    assert (out - want).abs().max().item() <= 1e-4
    path = i32(np.broadcast_to(np.arange(M), (N, M)))
    got = kda.kda_decode_commit(c["k"], c["v"], c["g"], c["beta"], c["state"], path, i32([4, 0, 6]),
                                state_out=torch.empty_like(c["state"]))
    assert (got - state).abs().max().item() <= 1e-4


@pytest.mark.parametrize("dtype,d", [(BF, 128), (F32, 64)])
def test_decode_tree_ignores_what_no_node_holds(kda, dtype, d):
    """NaN and infinities in the rows of no node, and in siblings, reach no other row."""
    rng = np.random.default_rng(6)
    N, M, H = 2, 12, 2
    x, par = ref.kda_inputs(N, M, H, d, dtype, rng), ref.parents(N, M, "tree", rng)
    par[:, 5] = -2
    clean = cu(x)
    args = lambda c: (c["q"], c["k"], c["v"], c["g"], c["beta"], c["state"], i32(par))
    want = kda.kda_decode_tree(*args(clean))
    lines = [ref.lines(p) for p in par]
    # a leaf that is a node but on nobody else's line
    leaf = [max(m for m in range(M) if lines[n][m] and not any(m in l for i, l in enumerate(lines[n]) if i != m))
            for n in range(N)]
    for name in ("q", "k", "v", "g", "beta"):
        x[name][5] = float("nan")
        x[name][M + 5] = float("inf")
        for n in range(N):
            x[name][n * M + leaf[n]] = float("nan")
    got = kda.kda_decode_tree(*args(cu(x)))
    keep = torch.ones(N * M, dtype=torch.bool)
    keep[[n * M + leaf[n] for n in range(N)]] = False
    assert torch.equal(got[keep.cuda()], want[keep.cuda()])


@pytest.mark.parametrize("dtype,d", [(BF, 64), (BF, 32), (BF, 16), (F32, 128), (F32, 32), (F32, 16)])
def test_decode_tree_ignores_what_no_node_holds_small_heads(kda, dtype, d):
    test_decode_tree_ignores_what_no_node_holds(kda, dtype, d)


def test_decode_tree_deep_decay(kda):
    """A chain of 64 nodes at the gate's bound (e^-5 each): products of decays
    underflow, nothing overflows."""
    rng = np.random.default_rng(7)
    x, par = ref.kda_inputs(1, 64, 2, 128, BF, rng), ref.parents(1, 64, "chain", rng)
    x["g"][:] = -5.0
    c = cu(x)
    out = kda.kda_decode_tree(c["q"], c["k"], c["v"], c["g"], c["beta"], c["state"], i32(par))
    check_kda(out, ref.decode_tree(*(f64(x[n]) for n in ("q", "k", "v", "g", "beta", "state")), par), BF, "deep")


# ------------------------------------------------------------------ decode_commit

@pytest.mark.parametrize("N,M,P,H,d,dtype", [(1, 1, 1, 1, 128, BF), (5, 9, 6, 3, 128, BF), (3, 70, 65, 2, 128, BF),
                                             (4, 8, 5, 2, 128, F32), (3, 6, 4, 5, 64, F32), (3, 6, 3, 3, 32, BF),
                                             (4, 7, 7, 3, 16, F32)])
@pytest.mark.parametrize("in_place", [False, True])
def test_decode_commit(kda, N, M, P, H, d, dtype, in_place):
    rng = np.random.default_rng(N * 100 + M + d)
    x = ref.kda_inputs(N, M, H, d, dtype, rng)
    path = rng.integers(0, M, (N, P)).astype(np.int32)
    accept = rng.integers(0, P + 1, N).astype(np.int32)
    accept[0] = P
    if N > 2:
        accept[1], accept[2] = -3, P + 4          # clamped
        path[2, P // 2] = M                       # outside: the path ends there
    c = cu(x)
    got = kda.kda_decode_commit(c["k"], c["v"], c["g"], c["beta"], c["state"], i32(path), i32(accept),
                                state_out=None if in_place else torch.empty_like(c["state"]))
    want = ref.decode_commit(*(f64(x[n]) for n in ("k", "v", "g", "beta", "state")), path, accept)
    check_kda(got, want, dtype, "commit")
    assert in_place == (got.data_ptr() == c["state"].data_ptr())
    if not in_place:
        assert torch.equal(c["state"].cpu(), x["state"])


# ------------------------------------------------------------------ tree_attention

# N, M, H, H_kv, d, page, lens, dtype, kind
ATT = [(1, 1, 1, 1, 128, 16, [1], BF, "chain"), (1, 1, 4, 2, 128, 16, [0], BF, "chain"),
       (3, 8, 8, 2, 128, 16, [5, 128, 129], BF, "tree"), (4, 16, 12, 1, 128, 64, [0, 63, 64, 700], BF, "holes"),
       (2, 64, 8, 2, 128, 32, [127, 1000], BF, "tree"), (2, 33, 16, 1, 128, 128, [300, 255], BF, "forest"),
       (2, 12, 96, 8, 128, 64, [513, 90], BF, "chain"), (2, 7, 4, 4, 128, 8, [77, 130], BF, "odd"),
       (2, 9, 6, 2, 128, 256, [400, 33], BF, "star"), (3, 5, 4, 2, 128, 16, [40, 0, 9], BF, "none"),
       (1, 7, 8, 1, 128, 64, [9001], BF, "tree"), (2, 11, 12, 4, 64, 16, [200, 1], BF, "tree"),
       (2, 40, 8, 2, 64, 64, [1500, 31], BF, "holes"), (2, 13, 6, 3, 128, 24, [100, 401], BF, "tree"),
       (2, 5, 4, 2, 128, 7, [50, 201], BF, "tree"), (2, 6, 4, 1, 128, 1, [33, 70], BF, "holes"),
       (2, 17, 4, 2, 32, 16, [150, 64], BF, "tree"), (2, 17, 4, 2, 16, 16, [150, 64], BF, "tree"),
       (3, 8, 8, 2, 128, 16, [5, 128, 129], F32, "tree"), (2, 64, 4, 2, 128, 32, [127, 600], F32, "holes"),
       (2, 11, 12, 4, 64, 24, [1, 900], F32, "forest"), (2, 6, 4, 4, 32, 5, [88, 0], F32, "chain"),
       (2, 6, 2, 1, 16, 16, [88, 31], F32, "odd"), (1, 3, 2, 1, 64, 16, [5000], F32, "chain")]


def check_attention(got, want, dtype, what):
    (out, lse), (w_out, w_lse, wt) = got, want
    eps = (2.0 ** -8, 2.0 ** -8) if dtype == BF else (0.0, 2e-5)
    err = np.abs(f64(out) - w_out)
    bound = eps[0] * np.abs(w_out) + eps[1] * wt + 1e-7
    assert np.isfinite(f64(out)).all() and (err <= bound).all(), (what, float((err - bound).max()))
    l, none = f64(lse), np.isinf(w_lse)
    assert (l[none] == -np.inf).all(), what
    dl = np.abs(l[~none] - w_lse[~none])
    assert (dl <= 2e-5 + 2e-6 * np.abs(w_lse[~none])).all(), (what, float(dl.max(initial=0)))


def run_attention(kda, c, par, **kw):
    return kda.kda_tree_attention(c["q"], c["k_new"], c["v_new"], c["k_cache"], c["v_cache"], c["page_table"],
                                  c["cache_lens"], i32(par), want_lse=True, **kw)


def ref_attention(x, par, scale):
    return ref.attention(*(f64(x[n]) for n in ("q", "k_new", "v_new", "k_cache", "v_cache")),
                         x["page_table"].numpy(), x["cache_lens"].numpy(), par, scale)


@pytest.mark.parametrize("N,M,H,Hkv,d,page,lens,dtype,kind", ATT)
def test_tree_attention(kda, N, M, H, Hkv, d, page, lens, dtype, kind):
    """Every entry of the cache past a length is NaN; the page table's unused entries name no page."""
    rng = np.random.default_rng(M * 100 + page + d)
    x, par = ref.cache_inputs(N, M, H, Hkv, d, page, lens, dtype, rng), ref.parents(N, M, kind, rng)
    ws = torch.empty(kda.kda_tree_attention_workspace_size(H, Hkv, d, dtype, N, M, page, x["page_table"].shape[1]),
                     dtype=torch.uint8, device="cuda")
    got = run_attention(kda, cu(x), par, workspace=ws)
    check_attention(got, ref_attention(x, par, d ** -0.5), dtype, f"{lens} page {page} {kind}")
    assert kda.kda_get_device_status(ws) == kda.KDA_DEVICE_OK


@pytest.mark.parametrize("dtype,page", [(BF, 16), (BF, 20), (F32, 16)])
def test_tree_attention_ignores_masked_values(kda, dtype, page):
    """NaN and infinities in no node's rows and in a sibling's reach no other row."""
    rng = np.random.default_rng(11)
    N, M, H, Hkv, d = 2, 10, 8, 2, 128
    x, par = ref.cache_inputs(N, M, H, Hkv, d, page, [200, 17], dtype, rng), ref.parents(N, M, "star", rng)
    par[:, 4] = -2
    want = run_attention(kda, cu(x), par)
    for name in ("k_new", "v_new"):
        x[name][4] = float("nan")
        x[name][M + 4] = float("-inf")
        x[name][7] = float("nan")                 # a leaf: its own row may be NaN
        x[name][M + 8, :, ::3] = float("inf")
    x["q"][4] = float("nan")
    x["q"][M + 4] = float("inf")
    got = run_attention(kda, cu(x), par)
    keep = torch.ones(N * M, dtype=torch.bool)
    keep[[7, M + 8]] = False
    keep = keep.cuda()
    assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[1][keep], want[1][keep])
    # and what a node does see, it sees
    assert torch.isnan(got[0][7]).all()
    assert not torch.isfinite(got[0][M + 8, :, ::3]).any()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_tree_attention_large_scores(kda, dtype):
    """Scores of several hundred: the maximum moves during the pass, weights
    underflow, and the result is the key with the largest score's value."""
    rng = np.random.default_rng(12)
    N, M, H, Hkv, d = 1, 4, 4, 1, 128
    x, par = ref.cache_inputs(N, M, H, Hkv, d, 16, [900], dtype, rng), ref.parents(N, M, "chain", rng)
    x["q"] *= 40
    got = run_attention(kda, cu(x), par)
    w_out, w_lse, wt = ref_attention(x, par, d ** -0.5)
    # scores near 700 hold 700 2^-24 sqrt(d) ~ 5e-4 of absolute error in fp32
    assert (np.abs(f64(got[0]) - w_out) <= 2.0 ** -7 * np.abs(w_out) + 2.0 ** -7 * wt).all()
    assert (np.abs(f64(got[1]) - w_lse) <= 2e-3).all()


@pytest.mark.parametrize("N,dtype,page", [(32, F32, 16), (33, F32, 16), (70, F32, 12), (33, BF, 16), (70, BF, 64),
                                          (70, BF, 12)])
def test_tree_attention_many_sequences(kda, N, dtype, page):
    """More sequences than a warp looks at in one step, ragged, some of them empty."""
    rng = np.random.default_rng(N + page)
    lens = rng.integers(0, 300, N)
    lens[::7] = 0
    x, par = ref.cache_inputs(N, 5, 6, 2, 64, page, lens, dtype, rng), ref.parents(N, 5, "holes", rng)
    check_attention(run_attention(kda, cu(x), par), ref_attention(x, par, 0.125), dtype, f"{N} sequences")


@pytest.mark.parametrize("H", [1, 4, 9])
def test_tree_attention_fp32_sums_of_one_sign(kda, H):
    """Values and weights all positive over a long cache: roundings that all point
    the same way would add up.  Scores err by 3 2^-22 of sum |q k| scale (about 11
    with these queries) and a few 2^-24 per product of their own size, the sums by
    some 2^-21: together below 2^-16 = 1.5e-5 of the sum of weighted values."""
    rng = np.random.default_rng(16 + H)
    x, par = ref.cache_inputs(1, 5, H, 1, 128, 16, [6000], F32, rng), ref.parents(1, 5, "tree", rng)
    for name in ("v_cache", "v_new"):
        x[name] = x[name].abs() + 1
    check_attention(run_attention(kda, cu(x), par), ref_attention(x, par, 128 ** -0.5), F32, "one sign")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_tree_attention_scale(kda, dtype):
    rng = np.random.default_rng(13)
    x, par = ref.cache_inputs(2, 6, 4, 2, 128, 16, [70, 200], dtype, rng), ref.parents(2, 6, "tree", rng)
    got = run_attention(kda, cu(x), par, scale=0.2)
    check_attention(got, ref_attention(x, par, 0.2), dtype, "scale")


@pytest.mark.parametrize("dtype,page", [(BF, 16), (F32, 16), (BF, 5)])
def test_tree_attention_reports_bad_tables(kda, dtype, page):
    """A page outside the cache and a length past the table are reported; no access leaves the buffers."""
    rng = np.random.default_rng(14)
    x, par = ref.cache_inputs(2, 4, 2, 1, 128, page, [40, 40], dtype, rng), ref.parents(2, 4, "chain", rng)
    n_pages = x["k_cache"].shape[0]
    for bad in (-1, n_pages, 2 ** 31 - 1):
        c = cu(x)
        c["page_table"][1, 1] = bad
        ws = torch.empty(kda.kda_tree_attention_workspace_size(2, 1, 128, dtype, 2, 4, page, c["page_table"].shape[1]),
                         dtype=torch.uint8, device="cuda")
        run_attention(kda, c, par, workspace=ws)
        assert kda.kda_get_device_status(ws) == kda.KDA_DEVICE_BAD_PAGE
        assert "page" in kda.kda_last_error()
    for bad in (-1, c["page_table"].shape[1] * page + 1):
        c = cu(x)
        c["page_table"].clamp_(0, n_pages - 1)
        c["cache_lens"][1] = bad
        run_attention(kda, c, par, workspace=ws)
        assert kda.kda_get_device_status(ws) == kda.KDA_DEVICE_BAD_LENGTH
    # the next call clears the word
    run_attention(kda, cu(x), par, workspace=ws)
    assert kda.kda_get_device_status(ws) == kda.KDA_DEVICE_OK


def test_tree_attention_repeats_bit_for_bit_on_another_stream(kda):
    rng = np.random.default_rng(15)
    x, par = ref.cache_inputs(3, 16, 8, 2, 128, 16, [900, 33, 2000], BF, rng), ref.parents(3, 16, "tree", rng)
    c = cu(x)
    want = run_attention(kda, c, par)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(3):
            got = run_attention(kda, c, par)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


# ------------------------------------------------------------------ verify_drafts

def draft_inputs(N, M, V, kind, with_draft, dtype, rng, sharp=2.0):
    logits = rng.standard_normal((N, M, V)) * sharp
    soft = lambda z: np.exp(z - z.max(-1, keepdims=True)) / np.exp(z - z.max(-1, keepdims=True)).sum(-1, keepdims=True)
    p = torch.from_numpy(soft(logits).astype(np.float32)).to(dtype)
    q = torch.from_numpy(soft(logits + rng.standard_normal((N, M, V)) * 0.5).astype(np.float32)).to(dtype)
    par = ref.parents(N, M, kind, rng)
    tokens = rng.integers(0, V, (N, M)).astype(np.int32)
    top = np.argsort(-f64(q), axis=-1)
    for n in range(N):
        rank = {}
        for m in range(1, M):
            p_ = int(par[n, m])
            if 0 <= p_ < m:
                r = rank.get(p_, 0)
                rank[p_] = r + 1
                tokens[n, m] = top[n, p_, min(r, V - 1)]
    u = rng.random((N, M + 1)).astype(np.float32)
    return p, q if with_draft else None, tokens, par, u


VERIFY = [(1, 1, 1, "chain", False, F32), (2, 1, 7, "chain", True, F32), (40, 8, 50, "tree", False, F32),
          (40, 8, 50, "chain", True, F32), (5, 64, 333, "tree", False, F32), (5, 64, 1001, "chain", True, BF),
          (6, 12, 4096, "forest", False, BF), (3, 16, 50257, "star", False, F32), (3, 9, 50257, "holes", True, F32),
          (3, 7, 32001, "odd", False, BF), (4, 5, 100, "none", False, F32), (2, 4, 131072, "chain", True, F32),
          (2, 4, 131075, "chain", False, BF)]


def run_verify(kda, p, q, tokens, par, u):
    return kda.kda_verify_drafts(p.cuda(), i32(tokens), i32(par), torch.from_numpy(u).cuda(),
                                 draft_probs=None if q is None else q.cuda())


def check_verify(kda, p, q, tokens, par, u):
    got = run_verify(kda, p, q, tokens, par, u)
    want = ref.verify(p.float().numpy(), tokens, par, u, None if q is None else q.float().numpy())
    for g, w, name in zip(got, want, ("accept", "path", "next")):
        assert (g.cpu().numpy() == w).all(), (name, g.cpu().numpy(), w)
    return want


@pytest.mark.parametrize("N,M,V,kind,with_draft,dtype", VERIFY)
def test_verify_drafts(kda, N, M, V, kind, with_draft, dtype):
    rng = np.random.default_rng(N * 100 + M + V)
    check_verify(kda, *draft_inputs(N, M, V, kind, with_draft, dtype, rng))


@pytest.mark.parametrize("with_draft", [False, True])
def test_verify_drafts_edges(kda, with_draft):
    """Equal distributions (everything is kept), opposite ones (nothing is),
    tokens outside the vocabulary, twins among the children, uniform numbers
    at and past their ends, rows of zeros, NaN and infinities."""
    rng = np.random.default_rng(21)
    V, M = 37, 6
    p, q, tokens, par, u = draft_inputs(12, M, V, "chain" if with_draft else "tree", with_draft, F32, rng)
    if with_draft:
        q[0] = p[0]
        q[1] = p[1].flip(-1)
        q[5] = 0.0
    p[2] = 0.0
    p[3, 0] = float("nan")
    p[4, :, 3] = float("inf")
    tokens[6, 1:] = V
    tokens[7, 1:] = -1
    tokens[8, 1:] = tokens[8, 1]
    u[9] = 0.0
    u[10] = np.float32(1 - 2.0 ** -24)
    u[11] = 1.0
    check_verify(kda, p, q, tokens, par, u)


def test_verify_drafts_keeps_the_targets_distribution(kda):
    """The first token after node 0 (a kept child's, or the drawn one) is
    distributed as the target's row: chi-square over 8 tokens and 60,000 draws,
    below its 1 - 1e-6 quantile (7 degrees of freedom: 38.3)."""
    rng = np.random.default_rng(22)
    N, V = 60000, 8
    p = np.array([.3, .2, .15, .1, .1, .08, .05, .02], np.float32)
    q = np.array([.1, .3, .05, .2, .1, .05, .1, .1], np.float32)
    for with_draft in (False, True):
        M = 2 if with_draft else 4
        par = np.zeros((N, M), np.int32)
        par[:, 0] = -1
        tokens = np.tile(np.array([0, 1, 4, 6][:M], np.int32), (N, 1))
        if with_draft:
            tokens[:, 1] = rng.choice(V, N, p=q.astype(np.float64) / q.astype(np.float64).sum())
        u = rng.random((N, M + 1)).astype(np.float32)
        P = torch.from_numpy(p).expand(N, M, V).contiguous()
        Q = torch.from_numpy(q).expand(N, M, V).contiguous() if with_draft else None
        accept, path, nxt = (t.cpu().numpy() for t in run_verify(kda, P, Q, tokens, par, u))
        first = np.where(accept > 1, tokens[np.arange(N), np.maximum(path[:, 1], 0)], nxt)
        seen = np.bincount(first, minlength=V)
        expect = N * p.astype(np.float64) / p.sum()
        assert ((seen - expect) ** 2 / expect).sum() < 38.3


# ------------------------------------------------------------------ cache_append

@pytest.mark.parametrize("N,M,Hkv,d,page,dtype,with_path", [
    (1, 1, 1, 16, 1, F32, False), (3, 7, 2, 128, 16, BF, True), (4, 200, 3, 128, 64, BF, False),
    (2, 33, 8, 64, 24, F32, True), (3, 9, 1, 32, 5, BF, True)])
def test_cache_append(kda, N, M, Hkv, d, page, dtype, with_path):
    rng = np.random.default_rng(M + page)
    lens = rng.integers(0, 3 * page, N)
    lens[0] = 0
    x = ref.cache_inputs(N, M, Hkv, Hkv, d, page, lens + M, dtype, rng)
    x["k_cache"].nan_to_num_()
    x["v_cache"].nan_to_num_()
    path = np.stack([rng.permutation(M) for _ in range(N)]).astype(np.int32) if with_path else None
    accept = rng.integers(0, M + 1, N).astype(np.int32)
    accept[-1] = M + 5
    if with_path and N > 1:
        path[1, 0] = M                             # left out
    table = x["page_table"].numpy().copy()
    if N > 2:
        table[2, 0] = -1                           # left out
    lens = lens.astype(np.int32)
    c = cu(x)
    got = kda.kda_cache_append(c["k_new"], c["v_new"], c["k_cache"], c["v_cache"], i32(table), i32(lens),
                               path=None if path is None else i32(path), accept=i32(accept))
    k, v, out = ref.append(x["k_new"], x["v_new"], x["k_cache"], x["v_cache"], table, lens, path, accept)
    assert torch.equal(c["k_cache"].cpu(), k) and torch.equal(c["v_cache"].cpu(), v)
    assert (got.cpu().numpy() == out).all()


# ------------------------------------------------------------------ refusals of the binding

def test_binding_refusals(kda):
    rng = np.random.default_rng(31)
    N, M, H, d = 2, 4, 2, 128
    c, par = cu(ref.kda_inputs(N, M, H, d, BF, rng)), i32(ref.parents(N, M, "tree", rng))
    tree = lambda **o: kda.kda_decode_tree(*(o.get(n, c[n]) for n in ("q", "k", "v", "g", "beta", "state")),
                                           o.get("parent", par))
    with pytest.raises(ValueError):
        tree(parent=par[:1])
    with pytest.raises(TypeError):
        tree(parent=par.long())
    with pytest.raises(TypeError):
        tree(k=c["k"].float())
    with pytest.raises(ValueError):
        tree(state=c["state"].transpose(2, 3))
    with pytest.raises(TypeError):
        tree(q=c["q"].half())
    big = cu(ref.kda_inputs(1, 65, 1, 16, F32, rng))
    with pytest.raises(kda.KDAError) as e:
        kda.kda_decode_tree(big["q"], big["k"], big["v"], big["g"], big["beta"], big["state"],
                            i32(ref.parents(1, 65, "chain", rng)))
    assert e.value.status == kda.KDA_ERR_UNSUPPORTED
    x = cu(ref.cache_inputs(N, M, 4, 2, d, 16, [20, 30], BF, rng))
    with pytest.raises(ValueError):
        run_attention(kda, dict(x, page_table=x["page_table"][:1]), par.cpu().numpy())
    with pytest.raises(ValueError):
        run_attention(kda, dict(x, k_new=x["k_new"][:, :1].contiguous()), par.cpu().numpy())
    with pytest.raises(kda.KDAError):
        run_attention(kda, x, par.cpu().numpy(), scale=math.nan)
    with pytest.raises(kda.KDAError):
        run_attention(kda, x, par.cpu().numpy(), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    p = torch.rand(N, M, 10, device="cuda")
    with pytest.raises(ValueError):
        kda.kda_verify_drafts(p, par, par, torch.rand(N, M, device="cuda"))
    with pytest.raises(ValueError):
        kda.kda_cache_append(x["k_new"][:, :1].contiguous(), x["v_new"], x["k_cache"], x["v_cache"],
                             x["page_table"], x["cache_lens"])
