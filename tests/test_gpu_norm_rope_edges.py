"""kda_head_norm_rope at values that are not finite, against the formula, and in place."""
import numpy as np
import pytest
import torch

from tests.kda_testlib import f64
from tests.test_gpu_norm_rope import BF, F32, freqs, inputs

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.mark.parametrize("n", [0, 1, 3, 8, 16, 24, 31, 32])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_an_infinity_stays_in_its_pair(kda, n, pairs, dtype):
    """A row with an infinity has a root of infinity: its finite channels are zeros, rotated ones beside
    the infinity no numbers, and one that is not rotated touches no other channel."""
    d, T = 64, 64
    q, k, w = inputs(T, 2, 1, d, dtype, False, seed=n)
    for t in range(T):
        q[t, 1, t], k[t, 0, t] = float("inf"), float("-inf")
    kept = q[:, 0].clone()
    pos = torch.arange(T, dtype=torch.int32, device="cuda") + 1
    qo, ko = kda.kda_head_norm_rope(q, k, pos, freqs(n), w[0], w[1], interleaved=pairs)
    alone, _ = kda.kda_head_norm_rope(kept[:, None].contiguous(), None, pos, freqs(n), w[0], interleaved=pairs)
    assert torch.equal(qo[:, :1], alone)
    for t in range(T):
        bad = {t}
        if t < 2 * n:
            bad.add(t ^ 1 if pairs else (t + n if t < n else t - n))
        for got in (f64(qo)[t, 1], f64(ko)[t, 0]):
            assert set(np.flatnonzero(np.isnan(got))) == bad, (t, n)
            assert (got[[c for c in range(d) if c not in bad]] == 0).all()


@pytest.mark.parametrize("n", [0, 3, 16, 32])
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_in_place_gives_the_same(kda, n, pairs, dtype):
    """Bit for bit, rows with infinities among them, for one token and for many out of a projection."""
    for T in (1, 700):
        q, k, w = inputs(T, 7, 2, 64, dtype, True, seed=n)
        q[T // 2, 3, 40], k[T // 2, 1, 5], q[0, 6, 63] = float("inf"), float("-inf"), float("inf")
        pos, f = torch.arange(T, dtype=torch.int32, device="cuda") * 371, freqs(n)
        want = kda.kda_head_norm_rope(q, k, pos, f, w[0], w[1], interleaved=pairs)
        got = kda.kda_head_norm_rope(q, k, pos, f, w[0], w[1], interleaved=pairs, q_out=q, k_out=k)
        for a, b in zip(got, want):
            assert torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(a.nan_to_num(), b.nan_to_num())
