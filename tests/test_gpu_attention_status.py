"""The status word of the attention calls where several findings come together: of a bounded wait that
ran out, offsets, a page and a length the first is reported."""
import numpy as np
import pytest
import torch

from tests import serving_ref as ref
from tests import tree_ref
from tests.test_gpu_prefix import run, workspace
from tests.test_gpu_tree import BF, F32, cu, i32

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]
FORMS = [(BF, 16), (BF, 20), (F32, 16)]
LENGTH = ("prefix_lens", 0, -1), ("cache_lens", 2, -1)
PAGE = ("prefix_table", (1, 2), -1), ("page_table", (0, 0), 2 ** 31 - 1)
OFFSETS = ("prefix_seqs", 0, -1)


@pytest.mark.parametrize("dtype,page", FORMS)
def test_findings_of_the_prefix_call(kda, dtype, page):
    rng = np.random.default_rng(9)
    N, M, H, Hkv, d = 4, 2, 4, 2, 64
    x = ref.prefix_inputs(N, M, H, Hkv, d, page, [30, 0, 7, 9], [300, 150], [0, 2, 4], dtype, rng)
    par, ws = tree_ref.parents(N, M, "chain", rng), workspace(kda, x, N, M, H, Hkv, d, page, dtype)

    def status(*changes):
        c = cu({n: t.clone() for n, t in x.items()})
        for n, at, value in changes:
            c[n][at] = value
        run(kda, c, par, workspace=ws)
        return kda.kda_get_device_status(ws)

    for length in LENGTH:
        assert status(length) == kda.KDA_DEVICE_BAD_LENGTH
        assert status(OFFSETS, length) == kda.KDA_DEVICE_BAD_OFFSETS, length
        for page_ in PAGE:
            assert status(page_, length) == kda.KDA_DEVICE_BAD_PAGE, (page_, length)
    for page_ in PAGE:
        assert status(page_) == kda.KDA_DEVICE_BAD_PAGE
        assert status(page_, OFFSETS) == kda.KDA_DEVICE_BAD_OFFSETS, page_
    assert status(*LENGTH, *PAGE, OFFSETS) == kda.KDA_DEVICE_BAD_OFFSETS
    assert status(*LENGTH, *PAGE) == kda.KDA_DEVICE_BAD_PAGE
    assert status() == kda.KDA_DEVICE_OK


@pytest.mark.parametrize("dtype,page", FORMS)
@pytest.mark.parametrize("N", [4, 50])
def test_findings_of_the_tree_call(kda, dtype, page, N):
    rng = np.random.default_rng(N)
    M, H, Hkv, d = 2, 4, 2, 64
    x = tree_ref.cache_inputs(N, M, H, Hkv, d, page, [30, 0, 700, 9] + [40] * (N - 4), dtype, rng)
    par = i32(tree_ref.parents(N, M, "chain", rng))
    size = kda.kda_tree_attention_workspace_size(H, Hkv, d, dtype, N, M, page, x["page_table"].shape[1])
    ws = torch.full((size,), 255, dtype=torch.uint8, device="cuda")

    def status(*changes):
        c = cu({n: t.clone() for n, t in x.items()})
        for n, at, value in changes:
            c[n][at] = value
        kda.kda_tree_attention(c["q"], c["k_new"], c["v_new"], c["k_cache"], c["v_cache"], c["page_table"],
                               c["cache_lens"], par, workspace=ws)
        return kda.kda_get_device_status(ws)

    bad_length, first, last = ("cache_lens", 1, -1), ("page_table", (0, 0), -1), ("page_table", (N - 1, 0), 2 ** 31 - 1)
    assert status(bad_length) == kda.KDA_DEVICE_BAD_LENGTH
    for bad_page in (first, last):
        assert status(bad_page) == kda.KDA_DEVICE_BAD_PAGE
        assert status(bad_page, bad_length) == kda.KDA_DEVICE_BAD_PAGE
    assert status() == kda.KDA_DEVICE_OK
