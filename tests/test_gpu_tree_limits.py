"""Tree-drafted decoding on tensors past 2^31 elements: the far ends against
plain fp64 implementations.  Tolerances: tests/test_gpu_tree.py."""
import numpy as np
import pytest
import torch

from tests import tree_ref as ref
from tests.kda_testlib import f64
from tests.test_gpu_tree import check_attention, check_kda

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]
BF = torch.bfloat16
i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


@pytest.mark.parametrize("page", [64, 20])
def test_attention_over_the_last_pages(kda, page):
    """A cache of 2.3e9 elements; 64-token pages take the tensor-core path, 20 the other."""
    rng = np.random.default_rng(page)
    H, Hkv, d, M, L = 8, 8, 64, 5, 210
    pages = 2_300_000_000 // (Hkv * page * d)
    x = ref.cache_inputs(1, M, H, Hkv, d, page, [L], BF, rng, spare=0)
    par = ref.parents(1, M, "tree", rng)
    used = x["k_cache"].shape[0]
    cache = []
    for c in ("k_cache", "v_cache"):
        big = torch.empty((pages, Hkv, page, d), dtype=BF, device="cuda")
        big[pages - used:] = x[c].cuda()
        cache.append(big)
    assert cache[0].numel() > 2 ** 31
    table = x["page_table"] + (pages - used)
    out, lse = kda.kda_tree_attention(x["q"].cuda(), x["k_new"].cuda(), x["v_new"].cuda(), *cache, table.cuda(),
                                      x["cache_lens"].cuda(), i32(par), want_lse=True)
    want = ref.attention(*(f64(x[n]) for n in ("q", "k_new", "v_new", "k_cache", "v_cache")),
                         x["page_table"].numpy(), x["cache_lens"].numpy(), par, d ** -0.5)
    check_attention((out, lse), want, BF, f"page {page}")
    # and the append to the very last page
    room = used * page - L
    acc = min(M, room)
    if acc:
        kda.kda_cache_append(x["k_new"].cuda(), x["v_new"].cuda(), *cache, table.cuda(), x["cache_lens"].cuda(),
                             accept=i32([acc]))
        pos = np.arange(L, L + acc)
        got = cache[0][table[0].long()[pos // page].cuda(), :, torch.from_numpy(pos % page).cuda()]
        assert torch.equal(got.cpu(), x["k_new"][:acc])


def test_states_past_2_31(kda):
    N, H, d = 1400, 96, 128
    state = torch.zeros((N, H, d, d), device="cuda")
    assert state.numel() > 2 ** 31
    rng = np.random.default_rng(3)
    x = ref.kda_inputs(1, 1, H, d, BF, rng)
    state[-1] = x["state"][0].cuda()
    big = {n: torch.zeros((N, *x[n].shape[1:]), dtype=x[n].dtype, device="cuda") for n in ("q", "k", "v", "g", "beta")}
    for n in big:
        big[n][-1] = x[n][0].cuda()
    par = i32(np.full((N, 1), -1))
    out = kda.kda_decode_tree(big["q"], big["k"], big["v"], big["g"], big["beta"], state, par)
    args = [f64(x[n]) for n in ("q", "k", "v", "g", "beta", "state")]
    check_kda(out[-1:], ref.decode_tree(*args, np.array([[-1]])), BF, "last tree")
    kda.kda_decode_commit(big["k"], big["v"], big["g"], big["beta"], state, i32(np.zeros((N, 1))), i32(np.ones(N)))
    check_kda(state[-1:], ref.decode_commit(*args[1:], np.array([[0]]), np.array([1])), BF, "last state")


def test_verify_past_2_31(kda):
    """40 x 64 rows of 900,001 tokens: the last sequence's rows are certain."""
    N, M, V = 40, 64, 900_001
    p = torch.empty((N, M, V), dtype=BF, device="cuda")
    assert p.numel() > 2 ** 31
    p[-1] = 0
    want = np.random.default_rng(4).integers(0, V, M)
    for m in range(M):
        p[-1, m, int(want[m])] = 1.0
    tokens = np.zeros((N, M), np.int32)
    tokens[-1, 1:] = want[:-1]
    tokens[-1, 40] = (tokens[-1, 40] + 1) % V            # the walk ends at node 39
    par = np.full((N, M), -2, np.int32)
    par[-1] = np.arange(M) - 1
    accept, path, token = kda.kda_verify_drafts(p, i32(tokens), i32(par), torch.full((N, M + 1), 0.5, device="cuda"))
    assert accept[-1].item() == 40 and path[-1, :40].tolist() == list(range(40)) and token[-1].item() == want[39]
    assert (accept[:-1] == 0).all() and (token[:-1] == -1).all() and (path[:-1] == -1).all()
