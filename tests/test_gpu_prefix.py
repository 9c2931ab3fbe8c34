"""kda_prefix_attention against the plain fp64 form (tests/serving_ref.py), with the
tolerances of the tree attention (tests/test_gpu_tree.py): the output's rounding
and that of the weights to bf16; in fp32 2e-5 of sum_j p_j |v_j|; lse 2e-5 + 2e-6 |lse|."""
import numpy as np
import pytest
import torch

from tests import serving_ref as ref
from tests import tree_ref
from tests.kda_testlib import f64
from tests.test_gpu_tree import check_attention, cu, i32

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]
BF, F32 = torch.bfloat16, torch.float32


def run(kda, c, par, **kw):
    return kda.kda_prefix_attention(c["q"], c["k_new"], c["v_new"], c["k_cache"], c["v_cache"], c["prefix_table"],
                                    c["prefix_lens"], c["prefix_seqs"], c["page_table"], c["cache_lens"], i32(par),
                                    want_lse=True, **kw)


def plain(x, par, scale):
    return ref.prefix_attention(*(f64(x[n]) for n in ("q", "k_new", "v_new", "k_cache", "v_cache")),
                                *(x[n].numpy() for n in ("prefix_table", "prefix_lens", "prefix_seqs", "page_table",
                                                         "cache_lens")), par, scale)


def workspace(kda, x, N, M, H, Hkv, d, page, dtype):
    size = kda.kda_prefix_attention_workspace_size(H, Hkv, d, dtype, N, M, len(x["prefix_lens"]), page,
                                                   x["prefix_table"].shape[1], x["page_table"].shape[1])
    return torch.full((size,), 255, dtype=torch.uint8, device="cuda")


# N, M, H, H_kv, d, page, lens, prefix lens, their sequences, dtype, kind
CASES = [
    (1, 1, 1, 1, 128, 16, [0], [1], [0, 1], BF, "chain"),
    (1, 1, 4, 2, 128, 16, [3], [127], [0, 1], BF, "chain"),
    (3, 1, 8, 2, 128, 16, [5, 0, 129], [128], [0, 3], BF, "chain"),
    (4, 4, 32, 8, 128, 64, [5, 0, 200, 9], [129], [0, 4], BF, "tree"),
    (5, 16, 12, 1, 128, 64, [0, 63, 64, 7, 1], [700, 300], [0, 3, 5], BF, "holes"),
    (6, 7, 5, 1, 128, 32, [10, 0, 4, 90, 1, 300], [1000, 65], [1, 3, 5], BF, "tree"),      # two have no prefix
    (9, 16, 96, 8, 128, 64, [20] * 9, [333], [0, 9], BF, "tree"),                          # two row tiles, many units
    (40, 3, 8, 2, 128, 8, [3] * 40, [40] * 40, list(range(41)), BF, "forest"),             # a prefix each
    (8, 2, 6, 3, 128, 24, [100, 3] * 4, [401, 0, 77], [0, 3, 5, 8], BF, "chain"),          # one of no tokens
    (3, 5, 4, 2, 128, 7, [50, 0, 1], [201], [0, 3], BF, "tree"),
    (3, 5, 4, 2, 128, 128, [50, 0, 1], [2049], [0, 2], BF, "odd"),
    (2, 64, 16, 1, 128, 16, [33, 70], [600], [0, 2], BF, "holes"),                         # 2,048 rows
    (3, 9, 128, 1, 128, 16, [33, 70, 0], [250], [0, 3], BF, "tree"),                       # 128 heads to one
    (2, 3, 160, 1, 128, 16, [33, 70], [250], [0, 2], BF, "tree"),                          # more than a tile's rows
    (7, 8, 12, 4, 64, 16, [20, 1, 0, 5, 9, 9, 64], [1500], [0, 7], BF, "tree"),
    (2, 1, 8, 8, 64, 64, [20, 1], [5000], [0, 2], BF, "chain"),
    (2, 17, 4, 2, 32, 16, [15, 64], [150], [0, 2], BF, "tree"),
    (2, 17, 4, 2, 16, 16, [15, 64], [90, 33], [0, 1, 2], BF, "none"),
    (3, 8, 8, 2, 128, 16, [5, 128, 0], [300], [0, 3], F32, "tree"),
    (6, 30, 4, 2, 128, 32, [17] * 6, [600, 41], [0, 4, 6], F32, "holes"),
    (5, 11, 12, 4, 64, 24, [1, 0, 90, 4, 4], [700, 31], [1, 3, 4], F32, "forest"),
    (2, 1, 4, 4, 32, 5, [8, 0], [501], [0, 2], F32, "chain"),
    (40, 2, 2, 1, 16, 16, [8] * 40, [31] * 20, list(range(0, 41, 2)), F32, "odd")]


@pytest.mark.parametrize("N,M,H,Hkv,d,page,lens,plens,seqs,dtype,kind", CASES)
def test_prefix_attention(kda, N, M, H, Hkv, d, page, lens, plens, seqs, dtype, kind):
    """Everything past a length is NaN, unused table entries name no page, the workspace starts as rubbish."""
    rng = np.random.default_rng(M * 100 + page + d)
    x, par = ref.prefix_inputs(N, M, H, Hkv, d, page, lens, plens, seqs, dtype, rng), tree_ref.parents(N, M, kind, rng)
    c, ws = cu(x), workspace(kda, x, N, M, H, Hkv, d, page, dtype)
    got = run(kda, c, par, workspace=ws)
    check_attention(got, plain(x, par, d ** -0.5), dtype, f"{lens} {plens} page {page} {kind}")
    assert kda.kda_get_device_status(ws) == kda.KDA_DEVICE_OK
    for _ in range(3):
        again = run(kda, c, par, workspace=ws)
        assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])


@pytest.mark.parametrize("N,M,H,Hkv,plens,d,dtype,page", [
    (40, 1, 32, 8, [30000, 17001], 128, BF, 64), (70, 16, 96, 8, [2000, 1501], 128, BF, 64),
    (70, 16, 64, 4, [2500], 64, BF, 16), (24, 4, 16, 4, [9000], 128, F32, 16)])
def test_prefix_attention_large(kda, N, M, H, Hkv, plens, d, dtype, page):
    """Several units to a CTA, and units over many CTAs; a sample of the sequences against the plain form."""
    rng = np.random.default_rng(N + M)
    seqs = [0, N] if len(plens) == 1 else [0, N // 3, N]
    lens = rng.integers(0, 300, N)
    x, par = ref.prefix_inputs(N, M, H, Hkv, d, page, lens, plens, seqs, dtype, rng), tree_ref.parents(N, M, "tree", rng)
    c, ws = cu(x), workspace(kda, x, N, M, H, Hkv, d, page, dtype)
    out, lse = run(kda, c, par, workspace=ws)
    assert kda.kda_get_device_status(ws) == kda.KDA_DEVICE_OK
    for n in (0, N // 3 - 1, N // 3, N - 1):
        rows, p = slice(n * M, n * M + M), 0 if len(plens) == 1 or n < N // 3 else 1
        want = ref.prefix_attention(*(f64(x[z][rows]) for z in ("q", "k_new", "v_new")), f64(x["k_cache"]), f64(x["v_cache"]),
                                    x["prefix_table"][p:p + 1].numpy(), [plens[p]], [0, 1],
                                    x["page_table"][n:n + 1].numpy(), [int(lens[n])], par[n:n + 1], d ** -0.5)
        check_attention((out[rows], lse[rows]), want, dtype, f"sequence {n}")
    for _ in range(10):
        again = run(kda, c, par, workspace=ws)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("dtype,page", [(BF, 16), (BF, 20), (F32, 16)])
def test_a_prefix_is_as_good_as_own_keys(kda, dtype, page):
    """The same keys as a prefix and as everyone's own pages give the same attention."""
    rng = np.random.default_rng(5)
    N, M, H, Hkv, d, L = 4, 3, 8, 2, 128, 40 * page
    x, par = ref.prefix_inputs(N, M, H, Hkv, d, page, [0] * N, [L], [0, N], dtype, rng), tree_ref.parents(N, M, "tree", rng)
    c = cu(x)
    out, lse = run(kda, c, par)
    table = c["prefix_table"].expand(N, -1).contiguous()
    out2, lse2 = kda.kda_tree_attention(c["q"], c["k_new"], c["v_new"], c["k_cache"], c["v_cache"], table,
                                        torch.full((N,), L, dtype=torch.int32, device="cuda"), i32(par), want_lse=True)
    tol = 2.0 ** -7 if dtype == BF else 1e-5
    assert ((out - out2).abs().float() <= tol * (out2.abs().float() + 0.2)).all() and torch.allclose(lse, lse2, atol=4e-5, rtol=0)
    # and no prefix at all is the tree attention, bit for bit
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    got = kda.kda_prefix_attention(c["q"], c["k_new"], c["v_new"], c["k_cache"], c["v_cache"], none.view(0, 1), none,
                                   torch.zeros(1, dtype=torch.int32, device="cuda"), table,
                                   torch.full((N,), L, dtype=torch.int32, device="cuda"), i32(par), want_lse=True)
    assert torch.equal(got[0], out2) and torch.equal(got[1], lse2)


@pytest.mark.parametrize("dtype,page", [(BF, 16), (BF, 20), (F32, 16)])
def test_values_that_are_not_finite(kda, dtype, page):
    """What no node's rows hold reaches no one; a NaN in a prefix reaches its sequences alone, one in a
    sequence's own keys that sequence; a node whose own score is -infinity keeps what the prefix gives."""
    rng = np.random.default_rng(6)
    N, M, H, Hkv, d = 5, 4, 4, 2, 128
    lens, plens, seqs = [30, 0, 70, 9, 200], [300, 150], [0, 2, 4]
    x, par = ref.prefix_inputs(N, M, H, Hkv, d, page, lens, plens, seqs, dtype, rng), tree_ref.parents(N, M, "chain", rng)
    par[:, 3] = -2
    want = run(kda, cu(x), par)
    clone = lambda: {n: t.clone() for n, t in x.items()}
    c = clone()
    for name in ("q", "k_new", "v_new"):
        c[name][3], c[name][M + 3] = float("nan"), float("inf")
    got = run(kda, cu(c), par)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert (got[0].view(N, M, H, d)[:, 3] == 0).all() and (got[1].view(N, M, H)[:, 3] == -np.inf).all()
    at = int(x["prefix_table"][1, 100 // page])
    for name, lse_too in (("k_cache", True), ("v_cache", False)):
        c = clone()
        c[name][at, 0, 100 % page] = float("nan")            # prefix 1, cache head 0: heads 0 and 1
        out, lse = (t.view(N, M, H, -1) for t in run(kda, cu(c), par))
        w_out, w_lse = (t.view(N, M, H, -1) for t in want)
        assert torch.isnan(out[2:4, :3, :2]).all() and (out[2:4, 3] == 0).all()
        assert torch.equal(out[2:4, :, 2:], w_out[2:4, :, 2:])
        assert torch.equal(out[[0, 1, 4]], w_out[[0, 1, 4]]) and torch.equal(lse[[0, 1, 4]], w_lse[[0, 1, 4]])
        assert torch.isnan(lse[2:4, :3, :2]).all() if lse_too else torch.equal(lse, w_lse)
    # a lone node without own keys whose score is -infinity
    c = clone()
    c["k_new"][M, :, :] = -2.0 ** 127
    c["q"][M, :, :] = 2.0 ** 60
    c["k_cache"][:] = torch.where(torch.isnan(c["k_cache"]), c["k_cache"], c["k_cache"] * 0)
    out, lse = run(kda, cu(c), par)
    assert torch.isfinite(out[M]).all() and torch.isfinite(lse[M]).all()
    assert torch.allclose(lse[M], torch.full_like(lse[M], float(np.log(300))), atol=1e-4)


@pytest.mark.parametrize("dtype,page", [(BF, 16), (BF, 20), (F32, 16)])
def test_large_scores(kda, dtype, page):
    """Scores of several hundred: the maximum moves within the prefix and between it and the own keys."""
    rng = np.random.default_rng(12)
    N, M, H, Hkv, d = 3, 4, 4, 1, 128
    x, par = ref.prefix_inputs(N, M, H, Hkv, d, page, [40, 0, 300], [900], [0, 3], dtype, rng), tree_ref.parents(N, M, "chain", rng)
    x["q"] *= 40
    out, lse = run(kda, cu(x), par)
    w_out, w_lse, wt = plain(x, par, d ** -0.5)
    # scores near 700 hold 700 2^-24 sqrt(d) ~ 5e-4 of absolute error in fp32
    assert (np.abs(f64(out) - w_out) <= 2.0 ** -7 * np.abs(w_out) + 2.0 ** -7 * wt).all()
    assert (np.abs(f64(lse) - w_lse) <= 2e-3).all()


@pytest.mark.parametrize("dtype,page", [(BF, 16), (BF, 20), (F32, 16)])
def test_status_word(kda, dtype, page):
    """Pages, lengths and offsets out of range are reported, and no access leaves the buffers."""
    rng = np.random.default_rng(9)
    N, M, H, Hkv, d = 4, 2, 4, 2, 64
    x, par = ref.prefix_inputs(N, M, H, Hkv, d, page, [30, 0, 7, 9], [300, 150], [0, 2, 4], dtype, rng), tree_ref.parents(N, M, "chain", rng)
    ws = workspace(kda, x, N, M, H, Hkv, d, page, dtype)

    def status(**changed):
        c = cu({n: t.clone() for n, t in x.items()})
        for n, (at, value) in changed.items():
            c[n][at] = value
        run(kda, c, par, workspace=ws)
        return kda.kda_get_device_status(ws)

    assert status() == kda.KDA_DEVICE_OK
    assert status(prefix_table=((1, 2), len(x["k_cache"]))) == kda.KDA_DEVICE_BAD_PAGE
    assert status(prefix_table=((0, 0), -1)) == kda.KDA_DEVICE_BAD_PAGE
    assert status(page_table=((0, 0), -1)) == kda.KDA_DEVICE_BAD_PAGE
    assert status(prefix_lens=(0, -1)) == kda.KDA_DEVICE_BAD_LENGTH
    assert status(prefix_lens=(0, 2 ** 30), prefix_table=((0, slice(None)), 0)) == kda.KDA_DEVICE_BAD_LENGTH
    assert status(cache_lens=(3, 2 ** 30), page_table=((3, slice(None)), 0)) == kda.KDA_DEVICE_BAD_LENGTH
    assert status(prefix_seqs=(2, 5)) == kda.KDA_DEVICE_BAD_OFFSETS
    assert status(prefix_seqs=(0, -1)) == kda.KDA_DEVICE_BAD_OFFSETS
    assert status(prefix_seqs=(1, 2 ** 31 - 1)) == kda.KDA_DEVICE_BAD_OFFSETS
    assert status() == kda.KDA_DEVICE_OK


def test_refusals(kda):
    rng = np.random.default_rng(9)
    x = cu(ref.prefix_inputs(2, 1, 4, 2, 64, 16, [3, 4], [20], [0, 2], BF, rng))
    par = np.full((2, 1), -1)
    for name, bad, error in (("prefix_lens", x["prefix_lens"].long(), TypeError),
                             ("prefix_seqs", x["prefix_seqs"][:1].contiguous(), ValueError),
                             ("prefix_table", x["prefix_table"][0], ValueError),
                             ("prefix_table", x["prefix_table"].cpu(), TypeError),
                             ("page_table", x["page_table"][:1].contiguous(), ValueError)):
        with pytest.raises(error):
            run(kda, {**x, name: bad}, par)
    with pytest.raises(kda.KDAError):
        run(kda, x, par, workspace=torch.empty(256, dtype=torch.uint8, device="cuda"))


def test_streams_and_graphs(kda):
    """A captured call on a side stream, replayed on new inputs, lengths and tables."""
    N, M, H, Hkv, d, page = 6, 2, 8, 2, 128, 16
    make = lambda seed, plens, seqs: ref.prefix_inputs(N, M, H, Hkv, d, page, [9, 0, 50, 3, 1, 2], plens, seqs, BF,
                                                       np.random.default_rng(seed))
    par = tree_ref.parents(N, M, "chain", np.random.default_rng(1))
    x, parent = cu(make(1, [500, 100], [0, 4, 6])), i32(par)
    ws = workspace(kda, x, N, M, H, Hkv, d, page, BF)
    call = lambda: kda.kda_prefix_attention(x["q"], x["k_new"], x["v_new"], x["k_cache"], x["v_cache"], x["prefix_table"],
                                            x["prefix_lens"], x["prefix_seqs"], x["page_table"], x["cache_lens"], parent,
                                            want_lse=True, workspace=ws)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        call()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out, lse = call()
    for seed, plens, seqs in ((2, [100, 500], [0, 1, 6]), (3, [0, 320], [2, 3, 5])):
        new = make(seed, plens, seqs)
        for n in new:
            if n in ("page_table", "prefix_table"):
                x[n].zero_()
                w = min(x[n].shape[1], new[n].shape[1])
                x[n][:, :w] = new[n][:, :w].cuda()
            elif n.endswith("_cache"):
                x[n][:len(new[n])] = new[n].cuda()[:len(x[n])]
            else:
                x[n].copy_(new[n])
        graph.replay()
        torch.cuda.synchronize()
        assert kda.kda_get_device_status(ws) == kda.KDA_DEVICE_OK
        check_attention((out, lse), plain(new, par, d ** -0.5), BF, f"replay {seed}")
