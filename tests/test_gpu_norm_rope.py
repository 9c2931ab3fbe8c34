"""kda_head_norm_rope against the plain fp64 form (tests/serving_ref.py).

Tolerance per element, from the roundings made: the fp32 sum of squares of d
channels (at most 16 + 3 sums in a row, halved by the root), the root's own
rounding, two products, cosine and sine (2 ulp each and 2^-26 of angle), the
rotation's products and sum: 22 steps of 2^-24 of |a| + |b|, the sizes of the
element's pair; then half a step of the output's type.
"""
import numpy as np
import pytest
import torch

from tests import serving_ref as ref
from tests.kda_testlib import f64, half_ulp_bf16

pytestmark = [pytest.mark.gpu, pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]
BF, F32 = torch.bfloat16, torch.float32


def check(got, x, positions, inv_freq, weight, what, **kw):
    rows = f64(x)
    want, size = ref.norm_rope(rows, f64(positions), f64(inv_freq), None if weight is None else f64(weight), **kw)
    bound = 22 * 2.0 ** -24 * size + (half_ulp_bf16(np.abs(want) + 22 * 2.0 ** -24 * size) if got.dtype == BF else 0.0)
    diff = np.abs(f64(got) - want)
    assert np.isfinite(f64(got)).all() and (diff <= bound).all(), (what, float((diff - bound).max()))


def freqs(n, base=10000.0):
    return torch.from_numpy((base ** (-np.arange(n) / max(n, 1))).astype(np.float32)).cuda()


def inputs(T, H, Hkv, d, dtype, fused, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if fused:
        qkv = (torch.randn(T, H + 2 * Hkv, d, generator=gen, device="cuda") * 2).to(dtype)
        q, k = qkv[:, :H], qkv[:, H:H + Hkv]
    else:
        q, k = ((torch.randn(T, h, d, generator=gen, device="cuda") * 2).to(dtype) for h in (H, Hkv))
    w = [1 + 0.2 * torch.randn(d, generator=gen, device="cuda") for _ in range(2)]
    return q, k, w


CASES = [(1, 1, 1, 128, 64, False, BF, False), (1, 32, 8, 128, 64, False, BF, False),
         (5, 12, 4, 64, 16, True, F32, True), (33, 7, 3, 64, 17, False, BF, True),
         (9, 96, 8, 128, 64, False, BF, True), (17, 5, 1, 32, 16, False, F32, False),
         (3, 40, 1, 16, 8, False, BF, False), (3, 6, 2, 16, 8, True, F32, False), (4, 33, 11, 16, 3, False, F32, True),
         (2, 3, 3, 128, 24, False, F32, True), (2, 3, 3, 128, 40, False, BF, True), (6, 10, 2, 128, 1, True, BF, False),
         (6, 10, 2, 32, 0, False, BF, False), (700, 3, 1, 128, 64, True, BF, True), (40, 9, 2, 32, 11, False, BF, False)]


@pytest.mark.parametrize("T,H,Hkv,d,n,pairs,dtype,fused", CASES)
def test_norm_rope(kda, T, H, Hkv, d, n, pairs, dtype, fused):
    q, k, w = inputs(T, H, Hkv, d, dtype, fused, seed=T * 100 + d)
    kept = [q.clone(), k.clone()]
    pos = torch.from_numpy(np.random.default_rng(T).integers(0, 262144, T).astype(np.int32)).cuda()
    f = freqs(n)
    qo, ko = kda.kda_head_norm_rope(q, k, pos, f, q_weight=w[0], k_weight=w[1], interleaved=pairs)
    assert qo.is_contiguous() and ko.is_contiguous()
    check(qo, q, pos, f, w[0], "q", interleaved=pairs)
    check(ko, k, pos, f, w[1], "k", interleaved=pairs)
    assert torch.equal(q, kept[0]) and torch.equal(k, kept[1])
    # without weights and keys; and in place of a projection's slices, whose values stay
    qo, none = kda.kda_head_norm_rope(q, None, pos, f, eps=1e-3, interleaved=pairs)
    assert none is None
    check(qo, q, pos, f, None, "q alone", eps=1e-3, interleaved=pairs)
    again, _ = kda.kda_head_norm_rope(q, k, pos, f, eps=1e-3, interleaved=pairs, q_out=q, k_out=k)
    assert again is q and torch.equal(q, qo)


@pytest.mark.parametrize("pairs", [False, True])
def test_far_and_negative_positions(kda, pairs):
    pos = torch.tensor([0, 1, -1, 262143, 2 ** 31 - 1, -2 ** 31, 123456789], dtype=torch.int32).cuda()
    q, k, w = inputs(len(pos), 2, 1, 64, F32, False)
    f = torch.tensor([1.0, 0.5, 0.1, 1e-3, 1e-9, 1e-30, 1e-40, 0.0, -0.3, 1.7, 3.0, 0.999], device="cuda")
    qo, ko = kda.kda_head_norm_rope(q, k, pos, f, w[0], w[1], interleaved=pairs)
    check(qo, q, pos, f, w[0], "q", interleaved=pairs)
    check(ko, k, pos, f, w[1], "k", interleaved=pairs)


def test_rows_do_not_reach_each_other(kda):
    """Zero rows stay zero; a row with NaN or infinity leaves all others as they are."""
    q, k, w = inputs(4, 9, 2, 128, BF, False, seed=3)
    pos, f = torch.arange(4, dtype=torch.int32, device="cuda"), freqs(64)
    want, wantk = kda.kda_head_norm_rope(q, k, pos, f, w[0], w[1])
    q[1, 3], q[2, 0, 5], q[2, 8, 127], k[3, 0, 0] = 0.0, float("nan"), float("inf"), float("-inf")
    got, gotk = kda.kda_head_norm_rope(q, k, pos, f, w[0], w[1])
    assert (got[1, 3] == 0).all() and torch.isnan(got[2, 0]).any() and torch.isnan(got[2, 8]).any()
    for t, h in ((1, 3), (2, 0), (2, 8)):
        got[t, h] = want[t, h]
    gotk[3, 0] = wantk[3, 0]
    assert torch.equal(got, want) and torch.equal(gotk, wantk)


def test_empty_and_refusals(kda):
    q, k, w = inputs(3, 4, 2, 64, BF, False)
    pos, f = torch.arange(3, dtype=torch.int32, device="cuda"), freqs(32)
    qo, ko = kda.kda_head_norm_rope(q[:0], k[:0], pos[:0], f)
    assert qo.shape == (0, 4, 64) and ko.shape == (0, 2, 64)
    with pytest.raises(TypeError):
        kda.kda_head_norm_rope(q, k, pos.long(), f)
    with pytest.raises(TypeError):
        kda.kda_head_norm_rope(q, k.float(), pos, f)
    with pytest.raises(ValueError):
        kda.kda_head_norm_rope(q.transpose(0, 1).contiguous().transpose(0, 1), k, pos, f)
    with pytest.raises(ValueError):
        kda.kda_head_norm_rope(q[:, :, ::2], k, pos, f)
    with pytest.raises(ValueError):
        kda.kda_head_norm_rope(q, k, pos, f, q_weight=w[0][:32].contiguous().new_ones(63))
    with pytest.raises(kda.KDAError):
        kda.kda_head_norm_rope(q, k, pos, freqs(33))
    odd = torch.randn(3, 4 * 64 + 4, device="cuda").bfloat16()[:, :256].view(3, 4, 64)       # 8 bytes off
    with pytest.raises(kda.KDAError):
        kda.kda_head_norm_rope(odd, k, pos, f)


def test_past_2_31_elements(kda):
    T, H, Hkv, d = 150000, 112, 8, 128
    qkv = torch.empty(T, H + Hkv, d, dtype=BF, device="cuda")
    for i in range(0, T, 10000):
        qkv[i:i + 10000].normal_()
    q, k = qkv[:, :H], qkv[:, H:]
    pos, f = torch.arange(T, dtype=torch.int32, device="cuda"), freqs(64)
    rows = torch.tensor([0, 1, 139810, 139811, 149000, T - 1], device="cuda")
    was = q[rows].clone(), k[rows].clone()
    kda.kda_head_norm_rope(q, k, pos, f, q_out=q, k_out=k)
    check(q[rows], was[0], pos[rows], f, None, "q")
    check(k[rows], was[1], pos[rows], f, None, "k")
