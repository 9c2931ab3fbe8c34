"""Argument checks of the tree-drafted decoding calls, before anything reaches
the GPU, and the plain implementations against each other (no GPU)."""
import ctypes

import numpy as np
import pytest

from tests import tree_ref as ref

FAKE = 0x10000     # 16-byte aligned, never dereferenced: the checks fail first


def dims(kda, H=96, d=128, dt=1):
    return kda.kda_dims(H, d, d, dt)


@pytest.fixture
def ptrs():
    return ctypes.c_void_p(FAKE), ctypes.c_void_p(FAKE + 4)


def test_decode_tree_argument_checks(kda, ptrs):
    p, mis = ptrs
    call = lambda **o: kda.lib.kda_decode_tree(o.get("q", p), p, p, p, p, p, o.get("parent", p), o.get("N", 2),
                                               o.get("M", 8), o.get("d", dims(kda)), o.get("out", p), None)
    assert call(N=0) == kda.KDA_OK
    assert call(N=-1) == kda.KDA_ERR_INVALID
    assert call(M=0) == kda.KDA_ERR_INVALID
    assert call(M=65) == kda.KDA_ERR_UNSUPPORTED and "64" in kda.kda_last_error()
    assert call(N=2 ** 30, M=8) == kda.KDA_ERR_INVALID
    assert call(q=None) == kda.KDA_ERR_INVALID and "q" in kda.kda_last_error()
    assert call(parent=None) == kda.KDA_ERR_INVALID and "parent" in kda.kda_last_error()
    assert call(out=mis) == kda.KDA_ERR_INVALID
    assert call(d=dims(kda, d=48)) == kda.KDA_ERR_UNSUPPORTED
    assert call(d=dims(kda, dt=3)) == kda.KDA_ERR_UNSUPPORTED


def test_decode_commit_argument_checks(kda, ptrs):
    p, mis = ptrs
    call = lambda **o: kda.lib.kda_decode_commit(p, p, p, p, o.get("s", p), o.get("path", p), o.get("acc", p),
                                                 o.get("N", 2), o.get("M", 8), o.get("P", 4), dims(kda), p, None)
    assert call(N=0) == kda.KDA_OK
    assert call(N=-1) == kda.KDA_ERR_INVALID
    assert call(M=0) == kda.KDA_ERR_INVALID and call(P=0) == kda.KDA_ERR_INVALID
    assert call(N=2 ** 30, P=4) == kda.KDA_ERR_INVALID
    assert call(s=mis) == kda.KDA_ERR_INVALID
    assert call(path=None) == kda.KDA_ERR_INVALID and call(acc=None) == kda.KDA_ERR_INVALID


def test_tree_attention_argument_checks(kda, ptrs):
    p, mis = ptrs
    size = lambda **o: kda.lib.kda_tree_attention_workspace_size(
        o.get("d", dims(kda)), o.get("Hkv", 8), o.get("N", 2), o.get("M", 8), o.get("page", 16), o.get("mp", 10))
    assert size() >= 256
    assert size(Hkv=7) == 0 and size(page=0) == 0 and size(mp=0) == 0 and size(M=65) == 0 and size(N=0) == 0
    call = lambda **o: kda.lib.kda_tree_attention(
        o.get("q", p), p, p, p, p, o.get("table", p), p, p, o.get("N", 2), o.get("M", 8), o.get("Hkv", 8),
        o.get("np", 20), o.get("page", 16), o.get("mp", 10), o.get("scale", 0.1), o.get("d", dims(kda)), p,
        o.get("lse", None), o.get("ws", p), o.get("wsb", 1 << 40), None)
    assert call(N=0) == kda.KDA_OK
    assert call(Hkv=7) == kda.KDA_ERR_INVALID and call(Hkv=0) == kda.KDA_ERR_INVALID
    assert call(M=65) == kda.KDA_ERR_UNSUPPORTED
    assert call(np=0) == kda.KDA_ERR_INVALID and call(page=0) == kda.KDA_ERR_INVALID
    assert call(mp=0) == kda.KDA_ERR_INVALID and call(page=2 ** 20, mp=2 ** 20) == kda.KDA_ERR_INVALID
    for s in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=s) == kda.KDA_ERR_INVALID
    assert call(q=None) == kda.KDA_ERR_INVALID and call(q=mis) == kda.KDA_ERR_INVALID
    assert call(table=None) == kda.KDA_ERR_INVALID and call(ws=None) == kda.KDA_ERR_INVALID
    assert call(lse=ctypes.c_void_p(FAKE + 2)) == kda.KDA_ERR_INVALID
    assert call(wsb=size() - 1) == kda.KDA_ERR_INVALID and "workspace" in kda.kda_last_error()


def test_verify_and_append_argument_checks(kda, ptrs):
    p, mis = ptrs
    ver = lambda **o: kda.lib.kda_verify_drafts(o.get("t", p), o.get("q", None), p, p, o.get("u", p), o.get("N", 2),
                                                o.get("M", 8), o.get("V", 100), o.get("dt", 0), p, p, p, None)
    assert ver(N=0) == kda.KDA_OK and ver(N=-1) == kda.KDA_ERR_INVALID
    assert ver(V=0) == kda.KDA_ERR_INVALID and ver(M=65) == kda.KDA_ERR_UNSUPPORTED
    assert ver(dt=2) == kda.KDA_ERR_UNSUPPORTED
    assert ver(t=mis) == kda.KDA_ERR_INVALID and ver(q=mis) == kda.KDA_ERR_INVALID
    assert ver(u=None) == kda.KDA_ERR_INVALID
    q = ctypes.c_void_p(FAKE + 4096)
    app = lambda **o: kda.lib.kda_cache_append(o.get("k", p), p, o.get("path", None), None, p, o.get("lens", p),
                                               o.get("N", 2), o.get("M", 8), o.get("P", 8), 20, o.get("page", 16),
                                               10, dims(kda), p, p, o.get("out", q), None)
    assert app(N=0) == kda.KDA_OK and app(N=-1) == kda.KDA_ERR_INVALID and app(N=70000) == kda.KDA_ERR_INVALID
    assert app(P=9) == kda.KDA_ERR_INVALID           # more than M without a path
    assert app(page=0) == kda.KDA_ERR_INVALID and app(k=mis) == kda.KDA_ERR_INVALID
    assert app(out=p) == kda.KDA_ERR_INVALID and "alias" in kda.kda_last_error()


def test_plain_tree_is_the_plain_chain_of_each_line():
    rng = np.random.default_rng(1)
    x = {k: v.double().numpy() for k, v in ref.kda_inputs(2, 9, 2, 16, __import__("torch").float32, rng).items()}
    par = ref.parents(2, 9, "holes", rng)
    out = ref.decode_tree(*(x[n] for n in ("q", "k", "v", "g", "beta", "state")), par)
    for n in range(2):
        for m, line in enumerate(ref.lines(par[n])):
            path, row = np.full((2, 9), -1), n * 9 + m
            path[n, :len(line)] = line
            accept = np.array([0, 0])
            accept[n] = len(line)
            S = ref.decode_commit(*(x[k] for k in ("k", "v", "g", "beta", "state")), path, accept)[n]
            want = np.einsum("hk,hkv->hv", x["q"][row], S) if line else 0 * out[row]
            assert np.allclose(out[row], want, atol=1e-12)


def test_plain_verify_on_certain_cases():
    p = np.zeros((1, 3, 4), np.float32)
    p[0, 0, 2] = p[0, 1, 1] = p[0, 2, 3] = 1
    par, u = np.array([[-1, 0, 1]]), np.full((1, 4), 0.5, np.float32)
    assert [a.tolist() for a in ref.verify(p, np.array([[9, 2, 1]]), par, u)] == [[3], [[0, 1, 2]], [3]]
    assert [a.tolist() for a in ref.verify(p, np.array([[9, 2, 0]]), par, u)] == [[2], [[0, 1, -1]], [1]]
    assert [a.tolist() for a in ref.verify(p, np.array([[9, 0, 1]]), par, u, p)] == [[1], [[0, -1, -1]], [2]]
