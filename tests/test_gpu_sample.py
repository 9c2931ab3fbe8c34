"""kda_sample against the plain fp64 form (tests/serving_ref.py).

A weight is right to 2^-24 of itself (the logarithm's fraction, rounded once to 2^-25,
the series, the whole multiples of 2^-42 for weights above 2^-18 of the largest, whose
share of a sum is what counts), and so is a sum.  So a token has to be the plain form's
unless u times the sum lies within 2^-22 of it of the border between two tokens, and
what stays has to be the plain form's unless p times the weight does.  probs: fp32
2^-22 of themselves (weight, sum, product), bf16 half a step more.
"""
import numpy as np
import pytest
import torch

from tests import serving_ref as ref
from tests.kda_testlib import f64, half_ulp_bf16

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]
BF, F32 = torch.bfloat16, torch.float32
TOL = 2.0 ** -22


def check(kda, logits, u, T=None, k=None, p=None, m=None, probs_dtype=F32, what=""):
    """Runs the rows at once and compares each; returns the tokens."""
    dev = lambda a, t: None if a is None else torch.as_tensor(np.asarray(a), dtype=t).cuda()
    args = dict(temperature=dev(T, F32), top_k=dev(k, torch.int32), top_p=dev(p, F32), min_p=dev(m, F32))
    N, V = logits.shape
    out = torch.full((N, V), 7.0, dtype=probs_dtype, device="cuda")
    token, probs = kda.kda_sample(logits, dev(u, F32), probs=out, **args)
    again, none = kda.kda_sample(logits, dev(u, F32), **args)
    nodraw, alone = kda.kda_sample(logits, probs=torch.empty_like(out), **args)
    assert probs is out and none is None and nodraw is None and torch.equal(alone, probs)
    assert torch.equal(token, again), what
    at = lambda name, n, d: d if args[name] is None else float(args[name][n])
    x, got, tok = f64(logits), f64(probs), token.tolist()
    for n in range(N):
        kw = dict(T=at("temperature", n, 1.0), k=int(at("top_k", n, 0)), p=at("top_p", n, 1.0), m=at("min_p", n, 0.0))
        for tol in (0.0, TOL, -TOL):
            t, want = ref.sample_row(x[n], **kw, tol=tol)
            if np.array_equal(want > 1e-37, got[n] > 1e-37):
                break
        else:
            # The sums' errors put the border anywhere within 2^-22 of p times the weight, not at the ends of that
            # range alone (with p = 1 - 2^-24 it holds the last thousand of a row's tokens).
            if kw["p"] < 1 and kw["m"] <= 0:
                kept = int((got[n] > 1e-37).sum())
                few, many = (int((ref.sample_row(x[n], **kw, tol=z)[1] > 1e-37).sum()) for z in (-TOL, TOL))
                assert few <= kept <= many, (what, n, kw, few, kept, many)
                t, want = ref.sample_row(x[n], **kw, first=kept)
        bound = TOL * want + (half_ulp_bf16(want) * 1.01 if probs_dtype == BF else 0.0) + 1e-37
        diff = np.abs(got[n] - want)
        assert (diff <= bound).all(), (what, n, kw, int((want > 0).sum()), int((got[n] > 0).sum()), float((diff - bound).max()))
        if t == -1:
            assert tok[n] == -1 and not got[n].any()
            continue
        cum, ui = np.cumsum(want), float(np.float32(u[n]))
        assert 0 <= tok[n] < V and want[tok[n]] > 0, (what, n, kw, tok[n])
        assert cum[tok[n]] - want[tok[n]] <= ui + TOL and ui - TOL <= cum[tok[n]], (what, n, kw, tok[n], ui)
    return tok


def rows(N, V, dtype, seed, scale=3.0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(N, V, generator=gen, device="cuda") * scale).to(dtype)


def uniform(N, seed):
    return np.random.default_rng(seed).random(N).astype(np.float32)


SIZES = [(3, 1), (3, 2), (4, 7), (5, 33), (3, 255), (2, 1000), (3, 4097), (2, 50257), (2, 131072)]


@pytest.mark.parametrize("N,V", SIZES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_each_filter(kda, N, V, dtype):
    x = rows(N, V, dtype, V)
    rng = np.random.default_rng(V)
    for i, kw in enumerate((dict(), dict(T=rng.uniform(0.3, 2.0, N)), dict(k=rng.integers(0, 60, N)),
                            dict(k=rng.integers(0, V + 2, N)), dict(p=rng.uniform(0.05, 1.0, N)),
                            dict(p=rng.uniform(0.9, 1.0, N), T=np.full(N, 3.0)), dict(m=rng.uniform(0.0, 0.3, N)),
                            dict(T=rng.uniform(0.3, 2.0, N), k=rng.integers(1, 300, N), p=rng.uniform(0.3, 1.0, N),
                                 m=rng.uniform(0.0, 0.1, N)))):
        check(kda, x, uniform(N, i), **kw, probs_dtype=(F32, BF)[i % 2], what=f"{i}")


@pytest.mark.parametrize("dtype", [BF, F32])
def test_edges_of_the_settings(kda, dtype):
    x = rows(12, 3001, dtype, 5)
    nan, inf = float("nan"), float("inf")
    big = np.arange(12)
    check(kda, x, uniform(12, 1), T=[0.0, -1.0, nan, 1e-30, 1e-4, inf, 1e30, 1.0, 1e-44, 0.01, 50.0, 3e38])
    check(kda, x, uniform(12, 2), k=[0, -5, 1, 2, 3000, 3001, 3002, 2 ** 31 - 1, -2 ** 31, 7, 600, 2500])
    check(kda, x, uniform(12, 3), p=[0.0, -1.0, nan, 1.0, 2.0, inf, -inf, 1e-30, 0.5, 0.9999999, 0.999, 1e-7])
    check(kda, x, uniform(12, 4), m=[0.0, -1.0, nan, 1.0, 2.0, inf, -inf, 1e-30, 0.5, 0.9999999, 1e-7, 1e-13])
    check(kda, x, np.where(big % 2 == 0, 0.0, np.float32(1 - 2.0 ** -24)).astype(np.float32), p=np.full(12, 0.9))
    top = x.float().argmax(-1).tolist()
    for kw in (dict(T=np.zeros(12)), dict(k=np.ones(12)), dict(p=np.zeros(12)), dict(T=np.zeros(12), p=np.full(12, 0.1), m=np.full(12, 0.5))):
        first = [int((x[n] == x[n].max()).nonzero()[0]) for n in range(12)]
        assert check(kda, x, uniform(12, 6), **kw) == first
    assert top is not None


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [9, 5000, 40001])
def test_ties_go_to_the_lowest_index(kda, dtype, V):
    """Few values, many of each; all equal; zeros of both signs are equal."""
    gen = torch.Generator(device="cuda").manual_seed(V)
    x = torch.randint(-3, 4, (6, V), generator=gen, device="cuda").to(dtype)
    x[1] = 0.5
    x[2] = torch.where(torch.rand(V, generator=gen, device="cuda") < 0.5, 0.0, -0.0)
    x[3, V // 2] = 9.0
    rng = np.random.default_rng(V)
    for i in range(3):
        check(kda, x, uniform(6, i), k=rng.integers(1, V, 6), p=rng.uniform(0.2, 1.0, 6))
        check(kda, x, uniform(6, i), k=rng.integers(1, min(V, 900), 6))
        check(kda, x, uniform(6, i), p=rng.uniform(0.01, 1.0, 6))
    tok, probs = kda.kda_sample(x[1:2].contiguous(), torch.tensor([0.5], device="cuda"), want_probs=True,
                                top_p=torch.tensor([0.5], device="cuda"))
    assert int((probs > 0).sum()) == (V + 1) // 2 and (probs[0, :(V + 1) // 2] > 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [5, 700, 40000])
def test_values_that_are_not_finite(kda, dtype, V):
    nan, inf = float("nan"), float("inf")
    x = rows(7, V, dtype, V + 1)
    x[0] = -inf
    x[1] = nan
    x[2, 1:] = -inf
    x[3, ::2] = nan
    x[4, V // 2], x[4, V - 1] = inf, inf
    x[5] = torch.where(torch.rand(V, device="cuda") < 0.7, torch.full_like(x[5], -inf), x[5])
    x[5, 0] = 1.0
    x[6] = -torch.finfo(dtype).max
    x[6, V - 2] = torch.finfo(dtype).max
    rng = np.random.default_rng(V)
    for kw in (dict(), dict(T=np.zeros(7)), dict(k=np.full(7, 3)), dict(p=np.full(7, 0.6)), dict(m=np.full(7, 0.2)),
               dict(T=rng.uniform(0.5, 2, 7), k=np.full(7, min(V, 500)), p=rng.uniform(0.2, 1, 7), m=np.full(7, 0.01))):
        tok = check(kda, x, uniform(7, 3), **kw)
        assert tok[0] == -1 and tok[1] == -1 and tok[2] == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_scales_of_logits(kda, dtype):
    """Flat, steep and far from zero; a few values among very small ones."""
    x = rows(8, 20000, F32, 9, 1.0) * torch.tensor([1e-30, 1e-6, 1e-3, 0.1, 30.0, 1e4, 1e30, 1.0], device="cuda")[:, None]
    x[7] += 1e5
    x = x.to(dtype)
    rng = np.random.default_rng(3)
    for kw in (dict(), dict(k=rng.integers(1, 2000, 8)), dict(k=np.full(8, 15000)), dict(p=rng.uniform(0.1, 1, 8)),
               dict(k=np.full(8, 9000), p=rng.uniform(0.1, 1, 8))):
        check(kda, x, uniform(8, 4), **kw)


@pytest.mark.parametrize("N,V,dtype", [(300, 3000 + 1, BF), (700, 501, F32), (65, 32000, F32), (5, 262144, F32),
                                       (3, 262143, BF), (40, 131075, BF)])
def test_many_rows_and_large_vocabularies(kda, N, V, dtype):
    x = rows(N, V, dtype, N + V)
    rng = np.random.default_rng(N)
    kw = dict(T=np.where(rng.random(N) < 0.1, 0.0, rng.uniform(0.5, 1.5, N)), k=rng.choice([0, 1, 40, 200, 1000, 5000], N),
              p=rng.uniform(0.5, 1.0, N), m=rng.uniform(0, 0.05, N))
    check(kda, x, uniform(N, 1), **kw)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("copies,V", [(1, 70001), (14, 40000)])
def test_rows_that_fill_lists(kda, dtype, copies, V):
    """Flat rows, few values, shares close to one: more candidates than the kernel lists, in few and in many CTAs."""
    gen = torch.Generator(device="cuda").manual_seed(V)
    scales = torch.tensor([1e-3, 0.05, 0.3, 1.0, 1.0, 1.0, 2.0, 3.0, 1.0, 1.0, 1.0, 1.0], device="cuda")
    x = torch.randn(12, V, generator=gen, device="cuda") * scales[:, None]
    x[8] = torch.randint(0, 3, (V,), generator=gen, device="cuda") * 0.5      # three values
    x[9] = 0.25                                                               # one
    x[10] = torch.where(torch.rand(V, generator=gen, device="cuda") < 0.5, x[10], -float("inf"))
    x[11, V // 3] = 12.0                                                      # one far above the others
    x = x.to(dtype).repeat(copies, 1)
    N = len(x)
    for i, kw in enumerate((dict(p=0.5), dict(p=0.9), dict(p=0.999), dict(p=0.99999), dict(p=1 - 2.0 ** -24), dict(p=1e-5),
                            dict(p=0.7, m=0.05), dict(p=0.95, m=0.3), dict(p=0.6, m=1e-4), dict(m=0.2), dict(p=0.8, T=0.2),
                            dict(p=0.8, T=5.0), dict(p=0.9, k=V - 9), dict(p=0.5, k=1025), dict(p=0.99, k=1024), dict(k=20000))):
        check(kda, x[:12] if copies == 1 else x, uniform(N, i), **{a: np.full(N, b) for a, b in kw.items()}, what=str(kw))
        if i == 0 and copies > 1:
            # as many rows as fill the GPU, or one at a time: the same bits
            u = torch.rand(N, generator=gen, device="cuda")
            p = torch.full((N,), 0.9, device="cuda")
            tok, probs = kda.kda_sample(x, u, top_p=p, want_probs=True)
            for n in range(12):
                t, q = kda.kda_sample(x[n:n + 1], u[n:n + 1], top_p=p[:1], want_probs=True)
                assert int(t) == int(tok[n]) and torch.equal(q[0], probs[n]), n


@pytest.mark.parametrize("V", [30000, 200000])
def test_far_from_zero(kda, V):
    """Logits whose distances are near their rounding: the bounds of a bin take in many more than the bin has."""
    x = rows(6, V, F32, V, 0.3) + torch.tensor([1e4, 1e5, 1e6, -1e5, -1e6, 3e6], device="cuda")[:, None]
    for i, kw in enumerate((dict(p=1e-6), dict(p=1e-3), dict(p=0.5), dict(p=1e-5, m=1e-3), dict(p=0.9, m=0.5), dict(k=30), dict(k=900),
                            dict(k=9000, p=0.3), dict(m=0.9), dict(p=1e-6, T=0.1))):
        check(kda, x, uniform(6, i), **{a: np.full(6, b) for a, b in kw.items()}, what=str(kw))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_strided_rows_and_alignment(kda, dtype):
    """Rows of a wider tensor, at every alignment, whose other columns are never looked at."""
    wide = torch.full((9, 1500), float("nan"), dtype=dtype, device="cuda")
    for lo, V in ((0, 1000), (8, 1001), (16, 777), (24, 1470)):
        x = wide[:, lo:lo + V]
        x.copy_(rows(9, V, dtype, lo))
        check(kda, x, uniform(9, lo), k=np.full(9, 20), p=np.full(9, 0.8))
        wide.fill_(float("inf"))
    flat = torch.randn(50 * 333, device="cuda").to(dtype)
    check(kda, flat.view(50, 333), uniform(50, 1), p=np.full(50, 0.7))       # rows at odd addresses


def test_draws_follow_the_distribution(kda):
    """40,000 draws from one row: counts within five standard deviations."""
    x = rows(1, 50, F32, 2, 1.0)
    n = 40000
    tok, _ = kda.kda_sample(x.expand(n, 50).contiguous(), torch.rand(n, device="cuda"),
                            top_k=torch.full((n,), 20, dtype=torch.int32, device="cuda"))
    _, want = ref.sample_row(f64(x)[0], k=20)
    got = np.bincount(tok.cpu().numpy(), minlength=50)
    assert (np.abs(got - n * want) <= 5 * np.sqrt(n * want * (1 - want)) + 1e-9).all()


def test_empty_and_refusals(kda):
    x, u = rows(3, 100, F32, 1), torch.rand(3, device="cuda")
    tok, probs = kda.kda_sample(x[:0], u[:0], want_probs=True)
    assert tok.shape == (0,) and probs.shape == (0, 100)
    for bad, error in ((dict(uniforms=u[:2].contiguous()), ValueError), (dict(temperature=u.double()), TypeError),
                       (dict(top_k=u), TypeError), (dict(top_p=u.cpu()), TypeError), (dict(min_p=u[None]), ValueError),
                       (dict(token=torch.empty(3, dtype=torch.int64, device="cuda")), TypeError),
                       (dict(probs=torch.empty(3, 99, device="cuda")), ValueError),
                       (dict(probs=torch.empty(3, 100, device="cuda").half()), TypeError)):
        with pytest.raises(error):
            kda.kda_sample(x, **{"uniforms": u, **bad})
    with pytest.raises(ValueError):
        kda.kda_sample(x[0], u)
    with pytest.raises(ValueError):
        kda.kda_sample(x.t(), u)
    with pytest.raises(TypeError):
        kda.kda_sample(x.half(), u)
    for args in ((x,), (x, None, None, None, None, None, torch.empty(3, dtype=torch.int32, device="cuda"))):
        with pytest.raises(kda.KDAError):
            kda.kda_sample(*args)
    with pytest.raises(kda.KDAError):
        kda.kda_sample(torch.empty(1, 262145, device="cuda"), u[:1].contiguous())


def test_streams_and_graphs(kda):
    x, u = rows(9, 5000, BF, 4), torch.rand(9, device="cuda")
    k, p = torch.full((9,), 50, dtype=torch.int32, device="cuda"), torch.full((9,), 0.9, device="cuda")
    want, wp = kda.kda_sample(x, u, top_k=k, top_p=p, want_probs=True)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got, gp = kda.kda_sample(x, u, top_k=k, top_p=p, want_probs=True)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(gp, wp)
    with torch.cuda.graph(graph):
        got, gp = kda.kda_sample(x, u, top_k=k, top_p=p, want_probs=True)
    for seed in (5, 6):
        x.copy_(rows(9, 5000, BF, seed))
        k.fill_(seed)
        graph.replay()
        want, wp = kda.kda_sample(x, u, top_k=k, top_p=p, want_probs=True)
        assert torch.equal(got, want) and torch.equal(gp, wp)


def test_past_2_31_elements(kda):
    N, V = 8300, 262144
    x = torch.empty(N, V, dtype=BF, device="cuda")
    for i in range(0, N, 100):
        x[i:i + 100].normal_()
    k = torch.full((N,), 30, dtype=torch.int32, device="cuda")
    u = torch.rand(N, device="cuda")
    tok, _ = kda.kda_sample(x, u, top_k=k)
    for n in (0, 1, 8191, 8192, 8193, N - 1):
        want, _ = kda.kda_sample(x[n:n + 1].contiguous(), u[n:n + 1].contiguous(), top_k=k[:1].contiguous())
        assert int(tok[n]) == int(want)
        t, probs = ref.sample_row(f64(x[n]), float(u[n]), k=30)
        assert probs[int(tok[n])] > 0
