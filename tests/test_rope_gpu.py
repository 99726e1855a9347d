"""GPU parity of attn_rope and attn_rope_bwd against the float64 oracle.

Tolerance, element by element: the result is rounded to bf16 once (half a step,
2^-8 of the value), after an fp32 rotation whose errors scale with |a| + |b| of
the pair: the remainder of the turns is good to 2^-33 and its radians, below pi,
round to fp32 (pi 2^-24, 1.9e-7), the fast sine and cosine are good to 2^-21
(4.8e-7) over [-pi, pi], the factor m, the two products and their sum round
once each (4 x 2^-24): 9.1e-7 m (|a| + |b|) in all, taken as 1e-6.
"""
import numpy as np
import pytest
import torch

from exact_softmax_attention_fwd_b200 import (AttnError, attn_get_device_error, attn_rope,
                                             attn_rope_bwd, rope_frequencies)
from exact_softmax_attention_fwd_b200 import workloads as W
from oracle import serving as S

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def close(got, x, positions, freq, interleaved, mscale, what=""):
    want = S.rotate(x, positions, freq, interleaved, mscale)
    n = len(freq)
    tol = np.abs(want) * 2.0 ** -8 + 1e-6 * abs(mscale) * S.pair_weight(x, n, interleaved)
    tol[..., 2 * n:] = 0.0  # copied
    bad = np.abs(S.f64(got) - want) > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} elements off"


CASES = [
    # B, Hq, Hkv, S, d, rotary, interleaved, scaling, start, step
    (1, 1, 1, 1, 64, 64, False, "none", 0, 1),
    (1, 32, 8, 1, 128, 128, True, "none", 777, 1),
    (3, 4, 2, 33, 64, 16, False, "none", 0, 1),
    (2, 5, 3, 129, 128, 48, True, "linear", 100, 3),
    (1, 8, 8, 257, 128, 128, False, "ramp", 1000000, 1),
    (2, 3, 1, 65, 64, 64, True, "base", -500, 7),
    (1, 2, 2, 31, 128, 112, False, "none", 2 ** 31 - 40, 1),
    (70, 2, 1, 3, 64, 32, False, "none", 5, 1),
]


def _positions(start, step, n):
    return torch.tensor([start + step * i for i in range(n)], dtype=torch.int32)


@pytest.mark.parametrize("bwd", [False, True])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_parity(case, bwd):
    B, Hq, Hkv, n, d, rot, inter, scaling, start, step = case
    freq, m = rope_frequencies(rot, scaling=scaling, factor=1.0 if scaling == "none" else 8.0)
    pos = _positions(start, step, n)
    q = W.randn_bf16((B, Hq, n, d), 31)
    k = W.randn_bf16((B, Hkv, n, d), 32)
    fn = attn_rope_bwd if bwd else attn_rope
    qo, ko = fn(q.to(DEV), k.to(DEV), freq.to(DEV), pos.to(DEV), interleaved=inter, mscale=m)
    at = -pos.double() if bwd else pos
    close(qo, q, at, freq, inter, m, "q")
    close(ko, k, at, freq, inter, m, "k")
    assert qo.is_contiguous() and ko.is_contiguous()


@pytest.mark.parametrize("interleaved", [False, True])
def test_views_of_a_fused_projection_and_back(interleaved):
    B, Hq, Hkv, n, d = 2, 6, 2, 50, 128
    freq, _ = rope_frequencies(64)
    qkv = W.randn_bf16((B, n, Hq + 2 * Hkv, d), 33)
    dev = qkv.to(DEV)
    q, k = dev[:, :, :Hq].transpose(1, 2), dev[:, :, Hq:Hq + Hkv].transpose(1, 2)
    qo, ko = attn_rope(q, k, freq.to(DEV), interleaved=interleaved)
    pos = torch.arange(n)
    close(qo, qkv[:, :, :Hq].transpose(1, 2), pos, freq, interleaved, 1.0)
    close(ko, qkv[:, :, Hq:Hq + Hkv].transpose(1, 2), pos, freq, interleaved, 1.0)
    assert torch.equal(dev.cpu(), qkv)
    # the gradients, into slices of the projection's gradient; its V part stays
    to = torch.full_like(dev, 7.0)
    attn_rope_bwd(qo, ko, freq.to(DEV), interleaved=interleaved,
                  q_out=to[:, :, :Hq].transpose(1, 2), k_out=to[:, :, Hq:Hq + Hkv].transpose(1, 2))
    close(to[:, :, :Hq].transpose(1, 2), qo.cpu(), -pos.double(), freq, interleaved, 1.0)
    assert bool((to[:, :, Hq + Hkv:] == 7.0).all())
    # turned there and back: two roundings of half a step each
    err = (to[:, :, :Hq + Hkv].cpu().float() - qkv[:, :, :Hq + Hkv].float()).abs()
    pair = torch.tensor(S.pair_weight(qkv[:, :, :Hq + Hkv], 32, interleaved))
    assert bool((err <= 2.0 ** -8 * (2 * pair + qkv[:, :, :Hq + Hkv].abs()) + 1e-6).all())


def test_packed_tokens_and_positions_of_each_row():
    x = W.randn_bf16((37, 4, 64), 34)
    freq, _ = rope_frequencies(32)
    pos = torch.randint(0, 5000, (37,), dtype=torch.int32, generator=torch.Generator().manual_seed(1))
    qo, none = attn_rope(x.to(DEV).transpose(0, 1)[None], None, freq.to(DEV), pos.to(DEV))
    assert none is None
    close(qo[0], x.transpose(0, 1), pos, freq, False, 1.0)
    # positions [B, S], the rows of a wider table
    q = W.randn_bf16((3, 2, 9, 64), 35)
    wide = torch.randint(0, 99, (3, 20), dtype=torch.int32, generator=torch.Generator().manual_seed(2))
    qo, _ = attn_rope(q.to(DEV), None, freq.to(DEV), wide.to(DEV)[:, 5:14])
    close(qo, q, wide[:, None, 5:14], freq, False, 1.0)
    # a broadcast input (one head read by several)
    qo, _ = attn_rope(q[:, :1].to(DEV).expand(3, 4, 9, 64), None, freq.to(DEV))
    close(qo, q[:, :1].expand(3, 4, 9, 64), torch.arange(9), freq, False, 1.0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_in_place_gives_the_same_bits(interleaved):
    q, k = W.randn_bf16((2, 4, 70, 128), 36).to(DEV), W.randn_bf16((2, 2, 70, 128), 37).to(DEV)
    freq = rope_frequencies(96)[0].to(DEV)
    qo, ko = attn_rope(q, k, freq, interleaved=interleaved)
    q2, k2 = attn_rope(q, k, freq, interleaved=interleaved, q_out=q, k_out=k)
    assert q2 is q and k2 is k
    assert torch.equal(q, qo) and torch.equal(k, ko)


def test_values_that_are_not_finite_stay_in_their_pair():
    q = torch.ones(1, 1, 4, 64, dtype=torch.bfloat16)
    q[0, 0, 1, 3], q[0, 0, 2, 40] = float("nan"), float("inf")
    qo, _ = attn_rope(q.to(DEV), None, rope_frequencies(32)[0].to(DEV))
    odd = ~torch.isfinite(qo.cpu()[0, 0])
    assert odd.nonzero().tolist() in ([[1, 3], [1, 19], [2, 40]],)


def test_empty_rows_and_refusals():
    freq = rope_frequencies(64)[0].to(DEV)
    q = torch.zeros(2, 4, 0, 64, dtype=torch.bfloat16, device=DEV)
    qo, _ = attn_rope(q, None, freq)
    assert qo.shape == q.shape
    x = torch.zeros(2, 4, 8, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError):
        attn_rope(x.float(), None, freq)
    with pytest.raises(ValueError):
        attn_rope(x, None, freq.float())
    with pytest.raises(ValueError):
        attn_rope(x, None, rope_frequencies(128)[0].to(DEV))
    with pytest.raises(ValueError):
        attn_rope(x, x[:, :, :4], freq)
    with pytest.raises(ValueError):
        attn_rope(x, None, freq, torch.zeros(7, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError):
        attn_rope(x, None, freq, torch.zeros(8, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        attn_rope(x.transpose(2, 3), None, freq)
    with pytest.raises(ValueError):
        attn_rope(x, None, freq, q_out=x[:, :2])
    with pytest.raises(ValueError):
        attn_rope(x, None, freq.cpu())
    with pytest.raises(AttnError):   # 24 turned elements
        attn_rope(x, None, freq[:12])
    with pytest.raises(AttnError):   # every head to the same rows
        attn_rope(x, None, freq, q_out=x[:, :1].expand(2, 4, 8, 64))
    odd = torch.zeros(2 * 4 * 8 * 64 + 8, dtype=torch.bfloat16, device=DEV)[4:-4].view(2, 4, 8, 64)
    with pytest.raises(AttnError):   # rows that do not start on 16 bytes
        attn_rope(odd, None, freq)
    assert attn_get_device_error()[0] == 0


def test_other_stream_and_graph():
    q = W.randn_bf16((2, 4, 300, 128), 38).to(DEV)
    freq = rope_frequencies(128)[0].to(DEV)
    want, _ = attn_rope(q, None, freq)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got, _ = attn_rope(q, None, freq, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        attn_rope(q, None, freq, q_out=out)
    q.copy_(W.randn_bf16((2, 4, 300, 128), 39))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, attn_rope(q, None, freq)[0])
