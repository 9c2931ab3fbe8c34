"""The tree-drafted decoding loop of examples/tree_speculation.py: the states
and pages that the steps leave are those of the same tokens fed as a chain."""
import importlib.util
import os

import pytest
import torch

from tests.kda_testlib import rms

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(kda):
    spec = importlib.util.spec_from_file_location("tree_speculation", os.path.join(ROOT, "examples",
                                                                                   "tree_speculation.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_steps_leave_what_the_tokens_leave(example):
    """Eight tree steps, then every sequence's kept tokens as one chain through a
    fresh copy of the model: lengths equal, states and pages within 2e-2 of their
    RMS in the mean and ten times that at worst (bf16 activations pass different
    kernels' roundings through four layers)."""
    n, T = 3, 9
    prompt = torch.randint(0, example.VOCAB, (n, T), generator=torch.Generator().manual_seed(5)).int().cuda()
    model = example.Hybrid(n, seed=1)
    tokens, mean = example.generate(model, prompt, steps=8, seed=7)
    assert mean >= 1.0                                   # node 0 is always kept
    assert all(0 <= t < example.VOCAB for row in tokens for t in row)
    for i in range(n):
        fed = torch.tensor([tokens[i][:-1]], dtype=torch.int32, device="cuda")
        assert int(model.lens[i]) == fed.shape[1] <= 64
        alone = example.Hybrid(1, seed=1)
        alone.feed(fed)
        for a, b in zip(alone.state, model.state):
            worst = (a[0] - b[i]).abs().max().item()
            assert worst <= 2e-1 * rms(a[0].cpu().numpy()) and \
                (a[0] - b[i]).square().mean().sqrt().item() <= 2e-2 * rms(a[0].cpu().numpy())
        L = fed.shape[1]
        pos = torch.arange(L, device="cuda")
        pages = lambda m, j: m.k_cache[m.table[j, pos // example.PAGE].long(), :, pos % example.PAGE].float()
        want = pages(alone, 0)
        assert (pages(model, i) - want).square().mean().sqrt() <= 2e-2 * want.square().mean().sqrt()
    # the same seed gives the same tokens
    again, _ = example.generate(example.Hybrid(n, seed=1), prompt, steps=8, seed=7)
    assert again == tokens


def test_steps_can_be_captured(kda, example):
    """One step of the five calls in a CUDA graph gives the eager step's results."""
    n = 2
    prompt = torch.randint(0, example.VOCAB, (n, 6), generator=torch.Generator().manual_seed(6)).int().cuda()
    model = example.Hybrid(n, seed=2)
    model.feed(prompt)
    tokens, parent = example.draft(example.successors(model, 3), prompt[:, -1], example.SHAPE)
    u = torch.rand(n, len(example.SHAPE) + 1, device="cuda")
    before = [s.clone() for s in model.state], model.k_cache.clone(), model.lens.clone()

    def step():
        probs, kept = model.forward(tokens, parent)
        accept, path, nxt = kda.kda_verify_drafts(probs, tokens, parent, u)
        model.commit(kept, path, accept)
        return accept, path, nxt, model.lens

    want = [t.clone() for t in step()]
    state = [s.clone() for s in model.state]

    def restore():
        for s, b in zip(model.state, before[0]):
            s.copy_(b)
        model.k_cache.copy_(before[1])

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        restore()
        model.lens = before[2]
        step()                                           # warm up off the default stream
    torch.cuda.current_stream().wait_stream(side)
    restore()
    model.lens = before[2]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    restore()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for a, b in zip(model.state, state):
        assert torch.equal(a, b)
