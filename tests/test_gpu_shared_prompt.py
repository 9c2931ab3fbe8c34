"""examples/shared_prompt.py: the calls around the softmax layers together, as a serving
loop makes them, against the same model run without sharing and against plain forms."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from tests import serving_ref as ref
from tests.kda_testlib import f64

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("shared_prompt", os.path.join(ROOT, "examples", "shared_prompt.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def prompt(example, T, seed=2):
    return torch.randint(0, example.VOCAB, (T,), generator=torch.Generator().manual_seed(seed)).cuda()


def test_example_runs(example, kda):
    example.main()


@pytest.mark.parametrize("T", [1, 64, 200, 333])
def test_a_shared_prompt_is_as_good_as_everyones_own(example, kda, T):
    """The same tokens fed to one model of five sequences and to five of one: the logits differ by
    roundings alone (bf16 values through four layers and the head, in products of other shapes and sums
    cut elsewhere): at most fifteen of 2^-8."""
    tokens, steps = prompt(example, T), 5
    together = example.Hybrid(n=5, seed=4)
    first = together.prompt(tokens)
    fed = torch.randint(0, example.VOCAB, (steps, 5), generator=torch.Generator().manual_seed(T)).int().cuda()
    got = [together.step(fed[i]) for i in range(steps)]
    together.check()
    assert together.lens.tolist() == [steps] * 5 and together.prefix_lens.tolist() == [T]
    for n in range(5):
        alone = example.Hybrid(n=1, seed=4)
        assert torch.equal(alone.prompt(tokens)[0], first[n])
        for i in range(steps):
            want = alone.step(fed[i, n:n + 1])
            scale = float(want.square().mean().sqrt())
            assert float((got[i][n] - want[0]).abs().max()) <= 15 * 2.0 ** -8 * scale, (n, i)


def test_softmax_layer_against_the_plain_form(example, kda):
    """A step's queries and keys out of the projection, through norm, rotation, pages and attention."""
    model, T = example.Hybrid(n=3, seed=5), 150
    model.prompt(prompt(example, T))
    x = torch.randn(3, example.HIDDEN, device="cuda")
    HQ, HKV, DA = example.HQ, example.HKV, example.DA
    for step in range(3):
        pos = model.prefix_lens + model.lens
        q, k, v = model._softmax_inputs(x, pos)
        out, lse = kda.kda_prefix_attention(q, k, v, model.k_cache, model.v_cache, model.prefix_table, model.prefix_lens,
                                            model.prefix_seqs, model.table, model.lens, model.root, want_lse=True)
        qkv = f64((model._norm(x).bfloat16() @ model.qkv).view(3, HQ + 2 * HKV, DA))
        for got, rows, w in ((q, qkv[:, :HQ], model.q_norm), (k, qkv[:, HQ:HQ + HKV], model.k_norm)):
            want, size = ref.norm_rope(rows, f64(pos), f64(model.inv_freq), f64(w))
            assert (np.abs(f64(got) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * size).all()
        want, w_lse, wt = ref.prefix_attention(f64(q), f64(k), f64(v), f64(model.k_cache), f64(model.v_cache),
                                               model.prefix_table.cpu().numpy(), [T], [0, 3], model.table.cpu().numpy(),
                                               model.lens.tolist(), np.full((3, 1), -1), DA ** -0.5)
        assert (np.abs(f64(out) - want) <= 2.0 ** -8 * (np.abs(want) + wt) + 1e-7).all()
        assert (np.abs(f64(lse) - w_lse) <= 2e-5 + 2e-6 * np.abs(w_lse)).all()
        model.lens = kda.kda_cache_append(k, v, model.k_cache, model.v_cache, model.table, model.lens)


def test_greedy_is_the_largest_logit_and_steps_can_be_captured(example, kda):
    """A step captured into a graph and replayed gives what the loop gives."""
    per = lambda x: torch.full((4,), x, device="cuda")
    tokens = prompt(example, 70)
    eager = example.generate(example.Hybrid(n=4, seed=6), tokens, 8, temperature=per(0.0))
    model = example.Hybrid(n=4, seed=6)
    logits = model.prompt(tokens)
    token, lens = torch.zeros(4, dtype=torch.int32, device="cuda"), model.lens
    u, zero = torch.zeros(4, device="cuda"), per(0.0)

    def step():
        kda.kda_sample(logits, u, temperature=zero, token=token)
        model.lens = lens
        logits.copy_(model.step(token))
        lens.copy_(model.lens)

    kept = [t.clone() for t in (*model.state, model.k_cache, model.v_cache, lens, logits)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    for t, was in zip((*model.state, model.k_cache, model.v_cache, lens, logits), kept):
        t.copy_(was)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(8):
        want = logits.argmax(-1).int()
        graph.replay()
        assert torch.equal(token, want) and torch.equal(token, eager[:, i])


def test_distributions_for_the_verification(kda):
    """Target and draft distributions from kda_sample, as kda_verify_drafts takes them: a chain whose draft
    has the target's logits is kept whole, and tokens outside the target's top-k never are."""
    N, M, V = 6, 5, 997
    gen = torch.Generator(device="cuda").manual_seed(8)
    logits = torch.randn(N * M, V, generator=gen, device="cuda") * 3
    k, p = torch.full((N * M,), 20, dtype=torch.int32, device="cuda"), torch.full((N * M,), 0.9, device="cuda")
    u = torch.rand(N * M, generator=gen, device="cuda")
    drawn, probs = kda.kda_sample(logits, u, top_k=k, top_p=p, want_probs=True)
    tokens = torch.cat([torch.zeros(N, 1, dtype=torch.int32, device="cuda"), drawn.view(N, M)[:, :-1]], 1).contiguous()
    par = torch.arange(M, dtype=torch.int32, device="cuda").expand(N, M).contiguous() - 1
    uni = torch.rand(N, M + 1, generator=gen, device="cuda")
    target = probs.view(N, M, V)
    accept, path, nxt = kda.kda_verify_drafts(target, tokens, par, uni, draft_probs=target.clone())
    assert accept.tolist() == [M] * N
    last = probs.view(N, M, V)[:, -1]
    assert (last[torch.arange(N), nxt.long()] > 0).all()
    wrong = tokens.clone()
    wrong[:, 1] = (target[:, 0] == 0).float().argmax(-1).int()
    accept, _, nxt = kda.kda_verify_drafts(target, wrong, par, uni, draft_probs=target.clone())
    assert accept.tolist() == [1] * N and (target[:, 0][torch.arange(N), nxt.long()] > 0).all()
