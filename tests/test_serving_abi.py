"""Argument checks of the calls around the softmax layers, before anything
reaches the GPU (no GPU)."""
import ctypes

import pytest
import torch

FAKE = 0x10000     # 16-byte aligned, never dereferenced: the checks fail first


def dims(kda, H=96, d=128, dt=1):
    return kda.kda_dims(H, d, d, dt)


@pytest.fixture
def ptrs():
    return ctypes.c_void_p(FAKE), ctypes.c_void_p(FAKE + 4)


def test_head_norm_rope_argument_checks(kda, ptrs):
    p, mis = ptrs
    o = ctypes.c_void_p(FAKE + 4096)
    call = lambda **a: kda.lib.kda_head_norm_rope(
        a.get("q", p), a.get("qs", 96 * 128), a.get("k", p), a.get("ks", 1024), a.get("pos", p), a.get("f", p),
        a.get("n", 64), a.get("w", None), None, a.get("T", 3), a.get("Hkv", 8), a.get("d", dims(kda)), 0,
        a.get("eps", 1e-6), a.get("qo", o), a.get("qos", 96 * 128), a.get("ko", o), a.get("kos", 1024), None)
    assert call(T=0) == kda.KDA_OK
    assert call(T=-1) == kda.KDA_ERR_INVALID and call(T=2 ** 31) == kda.KDA_ERR_INVALID
    assert call(Hkv=-1) == kda.KDA_ERR_INVALID
    assert call(n=-1) == kda.KDA_ERR_INVALID and call(n=65) == kda.KDA_ERR_INVALID
    for eps in (-1.0, float("nan")):
        assert call(eps=eps) == kda.KDA_ERR_INVALID
    assert call(q=None) == kda.KDA_ERR_INVALID and call(k=None) == kda.KDA_ERR_INVALID
    assert call(qo=None) == kda.KDA_ERR_INVALID and call(ko=mis) == kda.KDA_ERR_INVALID
    assert call(q=mis) == kda.KDA_ERR_INVALID and call(w=mis) == kda.KDA_ERR_INVALID
    assert call(pos=None) == kda.KDA_ERR_INVALID and call(f=None) == kda.KDA_ERR_INVALID
    assert call(pos=ctypes.c_void_p(FAKE + 2)) == kda.KDA_ERR_INVALID
    assert call(qs=96 * 128 + 4) == kda.KDA_ERR_INVALID and "16 bytes" in kda.kda_last_error()
    assert call(qs=95 * 128) == kda.KDA_ERR_INVALID and call(kos=512) == kda.KDA_ERR_INVALID
    assert call(qo=p, qs=97 * 128) == kda.KDA_ERR_INVALID and "in place" in kda.kda_last_error()
    assert call(d=dims(kda, d=256)) == kda.KDA_ERR_UNSUPPORTED
    assert call(d=dims(kda, dt=2)) == kda.KDA_ERR_UNSUPPORTED


def test_prefix_attention_argument_checks(kda, ptrs):
    p, mis = ptrs
    size = lambda **a: kda.lib.kda_prefix_attention_workspace_size(
        a.get("d", dims(kda)), a.get("Hkv", 8), a.get("N", 2), a.get("M", 8), a.get("P", 1), a.get("page", 16),
        a.get("mpp", 9), a.get("mp", 10))
    assert size() >= 256 and size(P=0) >= 256 and size(P=0, mpp=0) >= 256
    for bad in (dict(Hkv=7), dict(page=0), dict(mp=0), dict(mpp=0), dict(M=65), dict(N=0), dict(P=-1), dict(P=65536)):
        assert size(**bad) == 0
    call = lambda **a: kda.lib.kda_prefix_attention(
        a.get("q", p), p, p, p, p, a.get("pt", p), a.get("pl", p), a.get("ps", p), a.get("table", p), p, p,
        a.get("N", 2), a.get("M", 8), a.get("P", 1), a.get("Hkv", 8), a.get("np", 20), a.get("page", 16),
        a.get("mpp", 9), a.get("mp", 10), a.get("scale", 0.1), a.get("d", dims(kda)), p, a.get("lse", None),
        a.get("ws", p), a.get("wsb", 1 << 40), None)
    assert call(N=0) == kda.KDA_OK
    for bad in (dict(Hkv=7), dict(Hkv=0), dict(np=0), dict(page=0), dict(mp=0), dict(mpp=0), dict(P=-1), dict(P=65536),
                dict(mpp=2 ** 28), dict(q=None), dict(q=mis), dict(pt=None), dict(pl=None), dict(ps=None),
                dict(table=None), dict(ws=None), dict(ws=mis), dict(ws=ctypes.c_void_p(FAKE + 16)), dict(lse=ctypes.c_void_p(FAKE + 2)), dict(wsb=size() - 1),
                dict(N=2 ** 20, M=8), dict(scale=0.0), dict(scale=float("nan"))):
        assert call(**bad) == kda.KDA_ERR_INVALID, bad
    assert call(M=65) == kda.KDA_ERR_UNSUPPORTED and call(d=dims(kda, d=96)) == kda.KDA_ERR_UNSUPPORTED


def test_sample_argument_checks(kda, ptrs):
    p, mis = ptrs
    call = lambda **a: kda.lib.kda_sample(a.get("x", p), a.get("s", 100), a.get("T", None), a.get("k", None), None,
                                          a.get("m", None), a.get("u", p), a.get("N", 2), a.get("V", 100),
                                          a.get("dt", 0), a.get("pd", 0), a.get("tok", p), a.get("probs", None), None)
    assert call(N=0) == kda.KDA_OK
    for bad in (dict(N=-1), dict(N=2 ** 28), dict(V=0), dict(s=99), dict(tok=None), dict(x=None), dict(x=ctypes.c_void_p(FAKE + 2)),
                dict(u=None), dict(probs=ctypes.c_void_p(FAKE + 2)), dict(T=ctypes.c_void_p(FAKE + 2)), dict(k=ctypes.c_void_p(FAKE + 1)),
                dict(m=ctypes.c_void_p(FAKE + 3))):
        assert call(**bad) == kda.KDA_ERR_INVALID, bad
    assert call(V=262145, s=262145) == kda.KDA_ERR_UNSUPPORTED and call(dt=2) == kda.KDA_ERR_UNSUPPORTED
    assert call(probs=p, pd=5) == kda.KDA_ERR_UNSUPPORTED


def test_tensors_of_another_device_are_refused(kda, monkeypatch):
    class On:
        def __init__(self, device):
            self.device = device

        def get_device(self):
            return self.device

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    kda._here(On(1), None, On(1))
    with pytest.raises(ValueError, match="cuda:0"):
        kda._here(On(1), None, On(0))
