"""Tree-drafted decoding at the edges of its definition: tiles whose readers run
far apart, values that are not finite or close to the largest number, lengths
out of range.  Plain fp64 implementations: tests/tree_ref.py; tolerances:
tests/test_gpu_tree.py."""
import numpy as np
import pytest
import torch

from tests import tree_ref as ref
from tests.test_gpu_tree import (BF, F32, check_attention, check_verify, cu, draft_inputs, ref_attention, run_attention,
                                 run_verify)

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
