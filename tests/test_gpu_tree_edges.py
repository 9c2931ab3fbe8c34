"""Tree-drafted decoding at the edges of its definition: tiles whose readers run
far apart, values that are not finite or close to the largest number, lengths
out of range.  Plain fp64 implementations: tests/tree_ref.py; tolerances:
tests/test_gpu_tree.py."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from tests import tree_ref as ref
from tests.kda_testlib import f64
from tests.test_gpu_tree import (BF, F32, check_attention, check_verify, cu, draft_inputs, i32, ref_attention,
                                 run_attention, run_verify)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.mark.parametrize("M,H,Hkv,d", [(11, 96, 8, 128), (5, 32, 8, 128), (11, 96, 8, 64)])
def test_tree_attention_short_units_in_a_row(kda, M, H, Hkv, d):
    """Several units per CTA, their tiles of two, one and one steps of 64 keys in turn: the readers of
    the ring are furthest apart.  Every run gives the same bits."""
    rng = np.random.default_rng(M + d)
    lens = np.where(np.arange(64) % 2 == 0, 150, 20)
    x, par = ref.cache_inputs(64, M, H, Hkv, d, 16, lens, BF, rng), ref.parents(64, M, "tree", rng)
    c = cu(x)
    ws = torch.empty(kda.kda_tree_attention_workspace_size(H, Hkv, d, BF, 64, M, 16, x["page_table"].shape[1]),
                     dtype=torch.uint8, device="cuda")
    got = run_attention(kda, c, par, workspace=ws)
    check_attention(got, ref_attention(x, par, d ** -0.5), BF, "short units")
    assert kda.kda_get_device_status(ws) == kda.KDA_DEVICE_OK
    for _ in range(20):
        again = run_attention(kda, c, par, workspace=ws)
        assert torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])


@pytest.mark.parametrize("V", [5000, 20000, 131075])
@pytest.mark.parametrize("with_draft", [False, True])
def test_verify_drafts_with_walks_of_all_lengths(kda, V, with_draft):
    """Two, four and eight CTAs to a sequence, chains that are kept whole beside sequences without a
    node: the CTAs of a cluster meet whatever each had to do first.  Every run gives the same."""
    rng = np.random.default_rng(V)
    p, q, tokens, par, u = draft_inputs(11, 12, V, "chain", with_draft, F32, rng)
    par[1::3] = -2                                 # no node at all
    u[::3] = 0.0                                   # kept as far as the target has mass there
    check_verify(kda, p, q, tokens, par, u)
    first = run_verify(kda, p, q, tokens, par, u)
    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(first, run_verify(kda, p, q, tokens, par, u)))


@pytest.mark.parametrize("dtype,page", [(BF, 16), (F32, 16), (BF, 20)])
@pytest.mark.parametrize("M", [1, 3])
def test_tree_attention_keeps_what_is_no_number(kda, dtype, page, M):
    """A key, a query or a value that is not finite shows in every row that sees it, wherever the
    keys are cut (with few tiles each is a piece of its own), and in no other."""
    rng = np.random.default_rng(page + M)
    H, Hkv, d = 4, 2, 128
    x, par = ref.cache_inputs(2, M, H, Hkv, d, page, [640, 700], dtype, rng), ref.parents(2, M, "chain", rng)
    want = run_attention(kda, cu(x), par)
    clone = lambda: {n: t.clone() for n, t in x.items()}
    nan, inf = float("nan"), float("inf")

    def check(c, seen, lse=True):
        """seen: of sequence 1's rows, [M, H]"""
        out, l = run_attention(kda, cu(c), par)
        assert torch.equal(out[:M], want[0][:M]) and torch.equal(l[:M], want[1][:M])
        seen = seen.cuda()
        if lse:
            assert torch.isnan(out[M:][seen]).all() and torch.isnan(l[M:][seen]).all()
            assert torch.equal(l[M:][~seen], want[1][M:][~seen])
        else:
            assert not torch.isfinite(out[M:][seen]).any()
        assert torch.equal(out[M:][~seen], want[0][M:][~seen])

    for lens in ([640, 700], [640, 640]):
        x["cache_lens"] = torch.tensor(lens, dtype=torch.int32)
        want = run_attention(kda, cu(x), par)
        heads = torch.zeros(M, H, dtype=torch.bool)
        heads[:, :2] = True                        # those that read cache head 0
        c = clone()
        c["k_new"][M, 0] = nan                     # the root's key, in the last tile
        check(c, heads)
        c = clone()
        c["q"][M:, 1] = nan
        one = torch.zeros(M, H, dtype=torch.bool)
        one[:, 1] = True
        check(c, one)
        c = clone()
        for pos in range(256, 384):                # whole tiles of the cache
            c["k_cache"][c["page_table"][1, pos // page], 0, pos % page] = nan
        check(c, heads)
        c = clone()                                # an infinite value under a weight that underflows
        c["q"][M:, :2] = 4.0
        c["k_cache"][c["page_table"][1, 130 // page], 0, 130 % page] = -8.0
        c["v_cache"][c["page_table"][1, 130 // page], 0, 130 % page] = inf
        x2 = dict(c, v_cache=x["v_cache"])
        want = run_attention(kda, cu(x2), par)
        check(c, heads, lse=False)


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (BF, 32), (BF, 16), (F32, 128), (F32, 16)])
@pytest.mark.parametrize("M", [6, 20, 64])
def test_decode_tree_rows_of_no_node_are_zeros_for_any_state(kda, dtype, d, M):
    """Whatever the state holds: the rows of no node are zeros, the rows of other sequences and heads as
    they were, and the nodes' rows are not finite in the columns that are not."""
    rng = np.random.default_rng(d + M)
    N, H = 3, 2
    x, par = ref.kda_inputs(N, M, H, d, dtype, rng), ref.parents(N, M, "holes", rng)
    par[1, 0], par[1, M // 2] = -1, -2
    args = lambda c: (c["q"], c["k"], c["v"], c["g"], c["beta"], c["state"], i32(par))
    want = kda.kda_decode_tree(*args(cu(x)))
    node = torch.tensor([[bool(l) for l in ref.lines(p)] for p in par], device="cuda")
    for bad in (float("nan"), float("inf"), float("-inf")):
        c = dict(x, state=x["state"].clone())
        c["state"][1, 0, :, 3] = bad
        got = kda.kda_decode_tree(*args(cu(c))).view(N, M, H, d)
        assert (got[~node] == 0).all()
        rest = torch.ones(N, H, d, dtype=torch.bool, device="cuda")
        rest[1, 0, 3] = False
        rest = rest[:, None].expand(N, M, H, d)
        assert torch.equal(got[rest], want.view(N, M, H, d)[rest])
        assert not torch.isfinite(got[1, node[1], 0, 3]).any()


@pytest.mark.parametrize("dtype,page,d", [(F32, 16, 128), (F32, 16, 32), (BF, 16, 128), (BF, 20, 128), (BF, 16, 16)])
def test_tree_attention_ignores_the_largest_numbers_in_masked_rows(kda, dtype, page, d):
    """The type's largest and lowest values in the rows of no node and of a leaf reach no other row; a
    row that sees nothing but such a value returns it."""
    rng = np.random.default_rng(page + d)
    N, M, H, Hkv = 2, 9, 4, 2
    x, par = ref.cache_inputs(N, M, H, Hkv, d, page, [200, 5], dtype, rng), ref.parents(N, M, "star", rng)
    par[:, 4] = -2
    want = run_attention(kda, cu(x), par)
    big = torch.finfo(dtype).max
    for value in (big, -big):
        c = {n: t.clone() for n, t in x.items()}
        for n in range(N):
            for row in (n * M + 4, n * M + 8):
                for name in ("q", "k_new", "v_new"):
                    c[name][row] = value
        keep = torch.ones(N * M, dtype=torch.bool)
        keep[[8, M + 8]] = False
        got = run_attention(kda, cu(c), par)
        assert torch.equal(got[0][keep.cuda()], want[0][keep.cuda()])
        assert torch.equal(got[1][keep.cuda()], want[1][keep.cuda()])
        one = ref.cache_inputs(1, 1, H, Hkv, d, page, [0], dtype, rng)
        one["v_new"][:] = value
        out, _ = run_attention(kda, cu(one), np.array([[-1]]))
        assert (out == value).all()


@pytest.mark.parametrize("with_path", [False, True])
def test_cache_append_leaves_a_negative_length_alone(kda, with_path):
    """Nothing is written for a sequence whose length is below zero, and its length stays below zero, so
    that the next attention reports it."""
    rng = np.random.default_rng(41)
    N, M, H, d, page = 5, 6, 2, 64, 4
    x = ref.cache_inputs(N, M, H, H, d, page, [9] * N, BF, rng, spare=0)
    x["k_cache"].nan_to_num_()
    x["v_cache"].nan_to_num_()
    lens, accept = np.array([3, -1, -2 ** 31, -4, 0], np.int32), np.array([4, 6, 6, 2, 6], np.int32)
    path = np.tile(np.arange(M), (N, 1)) if with_path else None
    c = cu(x)
    got = kda.kda_cache_append(c["k_new"], c["v_new"], c["k_cache"], c["v_cache"], c["page_table"], i32(lens),
                               path=None if path is None else i32(path), accept=i32(accept))
    keep = [0, 4]
    k, v, _ = ref.append(torch.cat([x["k_new"][n * M:n * M + M] for n in keep]),
                         torch.cat([x["v_new"][n * M:n * M + M] for n in keep]), x["k_cache"], x["v_cache"],
                         x["page_table"].numpy()[keep], lens[keep], None if path is None else path[keep], accept[keep])
    assert torch.equal(c["k_cache"].cpu(), k) and torch.equal(c["v_cache"].cpu(), v)
    assert got[0].item() == 7 and got[4].item() == 6 and (got[1:4] < 0).all()
    assert got[3].item() == -2                     # the length and the accepted tokens, while that is negative
    ws = torch.empty(kda.kda_tree_attention_workspace_size(H, H, d, BF, N, M, page, c["page_table"].shape[1]),
                     dtype=torch.uint8, device="cuda")
    run_attention(kda, dict(c, cache_lens=got), ref.parents(N, M, "chain", rng), workspace=ws)
    assert kda.kda_get_device_status(ws) == kda.KDA_DEVICE_BAD_LENGTH


@pytest.mark.parametrize("dtype,d", [(BF, 128), (BF, 64), (BF, 32), (BF, 16), (F32, 64)])
def test_decode_tree_pseudo_values_past_the_types_range(kda, dtype, d):
    """v - S^T k of a leaf lies past bf16's largest number (and below fp32's): the leaf's row is right and
    no other row changes.  The leaf's row: a product of its own weight, checked to 2^-7 of its size."""
    rng = np.random.default_rng(d)
    N, M, H = 2, 12, 2
    x, par = ref.kda_inputs(N, M, H, d, dtype, rng), ref.parents(N, M, "star", rng)
    leaf = [5, M + 9]
    for n, row in enumerate(leaf):
        x["g"][n * M], x["g"][row] = 0.0, 0.0
        k = x["k"][row, :, :].float()
        x["state"][n, :, :, 3] = -8e35 * k / (k * k).sum(-1, keepdim=True)
        x["k"][n * M] = 0.0                        # the root leaves the state alone
        x["v"][row, :, 3] = torch.finfo(BF).max
    args = lambda c: (c["q"], c["k"], c["v"], c["g"], c["beta"], c["state"], i32(par))
    got = kda.kda_decode_tree(*args(cu(x)))
    other = dict(x, v=x["v"].clone())
    for row in leaf:
        other["v"][row, :, 3] = 0.0
    want = kda.kda_decode_tree(*args(cu(other)))
    keep = torch.ones(N * M, dtype=torch.bool)
    keep[leaf] = False
    assert torch.equal(got[keep.cuda()], want[keep.cuda()])
    full = ref.decode_tree(*(f64(x[n]) for n in ("q", "k", "v", "g", "beta", "state")), par)[leaf][:, :, 3]
    assert (np.abs(f64(got)[leaf][:, :, 3] - full) <= 2.0 ** -7 * np.abs(full) + 2.0 ** -7 * 8e35).all()


def test_example_reports_a_sequence_past_its_pages(kda):
    spec = importlib.util.spec_from_file_location("tree_speculation", os.path.join(ROOT, "examples",
                                                                                   "tree_speculation.py"))
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    model = example.Hybrid(2, max_tokens=32, seed=1)
    prompt = torch.randint(0, example.VOCAB, (2, 20), generator=torch.Generator().manual_seed(1)).int().cuda()
    model.feed(prompt)
    model.feed(prompt)                             # 40 tokens, room for 32
    model.check()
    model.feed(prompt)
    with pytest.raises(kda.KDAError, match="length"):
        model.check()


@pytest.mark.parametrize("M,G,Hkv,d,page,dtype", [(7, 24, 2, 128, 16, BF), (5, 17, 3, 64, 64, BF), (3, 64, 1, 128, 32, BF),
                                                  (9, 96, 2, 128, 16, BF), (4, 128, 1, 64, 128, BF),
                                                  (64, 128, 1, 128, 16, BF), (3, 129, 1, 128, 16, BF),
                                                  (2, 200, 2, 64, 24, BF), (4, 40, 2, 128, 16, F32),
                                                  (3, 130, 1, 32, 16, F32)])
def test_tree_attention_many_query_heads_to_a_cache_head(kda, M, G, Hkv, d, page, dtype):
    """More than 16: few nodes to a row tile, down to one, then the other form."""
    rng = np.random.default_rng(M * G)
    x, par = ref.cache_inputs(2, M, G * Hkv, Hkv, d, page, [131, 40], dtype, rng), ref.parents(2, M, "holes", rng)
    check_attention(run_attention(kda, cu(x), par), ref_attention(x, par, d ** -0.5), dtype, f"{M} x {G}")
