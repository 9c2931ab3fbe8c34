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


@pytest.mark.parametrize("more", [0, 300, 3000])
def test_neighbouring_logits_at_the_border_of_min_p(kda, more):
    """Two fp32 logits one step apart whose rounded weights come in the wrong order, with min-p between
    them: of the few that top-k leaves the beginning of the order stays, whichever of the two that ends with."""
    word = lambda *bits: np.array(bits, np.uint32).view(np.float32)
    x = np.concatenate([word(0), word(0xbe88544e, 0xbe88544f), np.float32([-50.0])])
    m = float(word(0x3f4427e3)[0])
    x = np.concatenate([x, np.full(more, -50.0, np.float32)])       # (from 300 on the few are sorted; 3,000 go by histograms)
    logits = torch.from_numpy(x)[None].repeat(4, 1).cuda()
    dev = lambda v, t=F32: torch.full((4,), v, dtype=t, device="cuda")
    u = torch.tensor([0.0, 0.3, 0.7, 0.999], device="cuda")
    token, probs = kda.kda_sample(logits, u, top_k=dev(3 + more // 2, torch.int32), min_p=dev(m), want_probs=True)
    w = np.exp(x.astype(np.float64))
    got = probs.cpu().numpy().astype(np.float64)
    for n in range(4):
        stay = got[n] > 0
        assert stay[0] and not stay[3:].any() and (stay[1] or not stay[2]), got[n][:4]
        want = w * stay / (w * stay).sum()
        assert (np.abs(got[n] - want) <= 2.0 ** -22 * want).all(), (got[n][:4], want[:4])
        assert int(token[n]) == int(np.searchsorted(np.cumsum(want), float(u[n]), side="right"))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [60, 900, 30000])
@pytest.mark.parametrize("k", [0, 50, 800, 1500])
def test_min_p_far_below_one(kda, dtype, V, k):
    """Weights on both sides of m, however small m is: of the distribution only those that reach it are there."""
    N = 6
    gen = torch.Generator(device="cuda").manual_seed(V)
    x = -torch.rand(N, V, generator=gen, device="cuda") * 60                       # weights from 1 to 10^-26
    x[:, V // 3] = 0.0
    m = np.float32([1e-3, 1e-9, 1e-12, 1e-13, 1e-20, 1e-24])
    check(kda, x.to(dtype), uniform(N, 5), m=m, k=np.full(N, k))
    check(kda, x.to(dtype), uniform(N, 6), m=m, k=np.full(N, k), p=np.full(N, 0.5), T=np.linspace(0.5, 3.0, N))
    check(kda, x.to(dtype), uniform(N, 7), m=m, k=np.full(N, k), T=np.linspace(0.5, 3.0, N))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [7, 200, 20000])
def test_min_p_from_one_on_keeps_the_largest(kda, dtype, V):
    """m above one counts as one: the logits equal to the largest stay, all of them."""
    x = rows(4, V, dtype, V)
    x[:, [1, V // 2, V - 1]] = 20.0
    for k in (0, 2, 5, V // 2):
        check(kda, x, uniform(4, 1), m=[1.0, 1.5, float("inf"), 3e38], k=np.full(4, k))
    _, probs = kda.kda_sample(x, want_probs=True, min_p=torch.tensor([1.0, 1.5, float("inf"), 3e38], device="cuda"))
    assert torch.equal(probs > 0, x == 20.0)
