"""kda_sample where one filter's border meets another's, and where the row is shared by a
cluster, against the plain fp64 form (tests/serving_ref.py); tolerances as tests/test_gpu_sample.py."""
import numpy as np
import pytest
import torch

from tests.test_gpu_sample import BF, F32, check, rows, uniform

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N", [3, 60])
def test_a_large_k_of_which_a_mask_leaves_fewer(kda, dtype, N):
    """All that the mask leaves stays, and goes on to top-p; rows over clusters of several CTAs, many times."""
    V, k, p = 40000, 5000, 0.9
    x = rows(N, V, dtype, 11 + N)
    gen = torch.Generator(device="cuda").manual_seed(N)
    x[torch.rand(N, V, generator=gen, device="cuda") > 0.08] = -float("inf")        # some 3,200 are left
    assert int((x > -float("inf")).sum(-1).max()) < k
    check(kda, x, uniform(N, 2), k=np.full(N, k), p=np.full(N, p))
    u = torch.from_numpy(uniform(N, 3)).cuda()
    kw = dict(top_k=torch.full((N,), k, dtype=torch.int32, device="cuda"), top_p=torch.full((N,), p, device="cuda"))
    token, probs = kda.kda_sample(x, u, want_probs=True, **kw)
    plain, alone = kda.kda_sample(x, u, want_probs=True, top_p=kw["top_p"])
    assert torch.equal(token, plain) and torch.equal(probs, alone)
    for _ in range(50):
        again, out = kda.kda_sample(x, u, want_probs=True, **kw)
        assert torch.equal(again, token) and torch.equal(out, probs)
