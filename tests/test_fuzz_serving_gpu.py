"""Randomized sweeps of the rotary, append and window-with-first-tokens calls against the float64
oracle: shapes, lengths, windows, pages and layouts drawn from seeded generators around the
kernels' edges (16-token chunks, 128-key tiles, 256-row units, page ends)."""
import math
import random

import numpy as np
import pytest
import torch

from exact_softmax_attention_fwd_b200 import (attn_append_paged, attn_bwd_window_sinks,
                                             attn_decode_paged_window,
                                             attn_decode_paged_window_fp8, attn_fwd_paged_window,
                                             attn_fwd_window_sinks, attn_get_device_error,
                                             attn_rope, rope_frequencies)
from exact_softmax_attention_fwd_b200 import workloads as W
from oracle import serving as S
from oracle.kv_fp8 import dequantize

from parity import check_grad
from window_parity import check_rows

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
EDGES = [1, 2, 15, 16, 17, 31, 32, 33, 127, 128, 129, 255, 256, 257, 384, 500]


def _n(rng, top=500):
    return min(top, rng.choice(EDGES) if rng.random() < 0.6 else rng.randint(1, top))


def _heads(rng, groups=(1, 2, 3, 4, 8)):
    kv = rng.choice([1, 2, 3])
    return kv * rng.choice(groups), kv


def _mask(rng):
    window = rng.choice([0, 1, 16, 100, 127, 128, 129, 300, rng.randint(1, 600)])
    return window, rng.choice([0, 1, 4, 31, 32, 33, 128, 129, rng.randint(0, 400)])


def _ok(what):
    st, flags = attn_get_device_error()
    assert st == 0, f"{what}: device error flags {flags:#x}"


@pytest.mark.parametrize("seed", range(24))
def test_window_forward_and_backward(seed):
    rng = random.Random(1000 + seed)
    Hq, Hkv = _heads(rng)
    B, d = rng.choice([1, 2]), rng.choice([64, 128])
    sq = _n(rng)
    sk = sq if rng.random() < 0.5 else _n(rng, 700)
    window, sinks = _mask(rng)
    q, k, v = W.prefill_inputs(B, Hq, Hkv, sq, sk, d, 2000 + seed)
    lens = torch.tensor([rng.randint(0, sk) for _ in range(B)], dtype=torch.int32) \
        if rng.random() < 0.5 else None
    what = f"{(B, Hq, Hkv, sq, sk, d, window, sinks, lens)}"
    scale = 1 / math.sqrt(d)
    qd, kd, vd = q.to(DEV), k.to(DEV), v.to(DEV)
    ld = None if lens is None else lens.to(DEV)
    o, lse = attn_fwd_window_sinks(qd, kd, vd, scale, window, sinks, k_lens=ld)
    check_rows(o, lse, S.window_fwd(q, k, v, scale, window, sinks, lens, bound=True), what)
    do = W.grad_output(B, Hq, sq, d, 2000 + seed)
    got = attn_bwd_window_sinks(qd, kd, vd, o, lse, do.to(DEV), scale, window, sinks, k_lens=ld)
    grads = S.window_grads(q, k, v, do, scale, window, sinks, lens)
    # Where every row sees one key at most, P is 1, O is that key's value and dS = dP - D is 0:
    # the kernel takes the difference of two fp32 sums of the same d products dO_i v_i, each
    # within (d + 2) 2^-24 sum |dO_i v_i|, and a key's dK adds group * Sq such rows.
    most = lambda x: float(x.float().abs().max())  # noqa: E731
    floor = 1.01 * 2 * (d + 2) * 2.0 ** -24 * float(do.float().abs().sum(-1).max()) * most(v) * \
        scale * (Hq // Hkv) * sq * max(most(q), most(k))
    for name, g, r in zip(("dq", "dk", "dv"), got, grads):
        if np.any(r) or name == "dv":
            check_grad(g, r, what=f"{name} {what}")
        else:
            assert float(g.float().abs().max()) <= floor, f"{name} {what}"
    _ok(what)


def _lengths(rng, new):
    return [max(n, 1) + rng.choice([0, 0, 1, rng.randint(0, 900)]) for n in new]


@pytest.mark.parametrize("seed", range(24))
def test_paged_chunks(seed):
    rng = random.Random(3000 + seed)
    Hq, Hkv = _heads(rng, (1, 2, 3, 4, 8, 16))
    d, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    new = [rng.choice([0, 1, _n(rng, 300)]) for _ in range(rng.randint(1, 5))]
    if sum(new) == 0:
        new[0] = 3
    total = _lengths(rng, new)
    window, sinks = _mask(rng)
    q, cu, c = W.paged_prefill_inputs(new, total, Hq, Hkv, d, page, 4000 + seed)
    kc, vc = c.k_cache.clone(), c.v_cache.clone()
    for b, n in enumerate(total):
        if n % page:
            last = int(c.block_table[b, n // page])
            kc[last, n % page:], vc[last, n % page:] = float("nan"), float("nan")
    what = f"{(new, total, Hq, Hkv, d, page, window, sinks)}"
    scale = 1 / math.sqrt(d)
    args = [x.to(DEV) for x in (q, kc, vc, c.block_table, cu, c.seq_lens)]
    o, lse = attn_fwd_paged_window(*args, max(new), scale, window, sinks)
    check_rows(o, lse, S.paged_window(q, c.k_cache, c.v_cache, c.block_table, cu, c.seq_lens, scale,
                                      window, sinks, bound=True), what)
    _ok(what)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("seed", range(20))
def test_single_tokens(seed, fp8):
    rng = random.Random(5000 + seed)
    Hq, Hkv = _heads(rng, (1, 2, 3, 5, 8))
    d, page = rng.choice([64, 128]), rng.choice([16, 48, 64, 256])
    B = rng.choice([1, 2, 7, 60])
    lens = [rng.choice([0, 1, _n(rng, 1500), rng.randint(0, 1500)]) for _ in range(B)]
    window, sinks = _mask(rng)
    make = W.fp8_paged_inputs if fp8 else W.paged_inputs
    c = make(torch.tensor(lens, dtype=torch.int32), Hq, Hkv, d, page, 6000 + seed)
    what = f"{(lens, Hq, Hkv, d, page, window, sinks)}"
    scale = 1 / math.sqrt(d)
    t = [x.to(DEV) for x in (c.q, c.k_cache, c.v_cache)]
    if fp8:
        o, lse = attn_decode_paged_window_fp8(*t, c.k_scale.to(DEV), c.v_scale.to(DEV),
                                              c.block_table.to(DEV), c.seq_lens.to(DEV), scale,
                                              window, sinks)
        kc, vc = (dequantize(x.numpy(), s.numpy()) for x, s in
                  ((c.k_cache, c.k_scale), (c.v_cache, c.v_scale)))
    else:
        o, lse = attn_decode_paged_window(*t, c.block_table.to(DEV), c.seq_lens.to(DEV), scale,
                                          window, sinks)
        kc, vc = c.k_cache, c.v_cache
    check_rows(o, lse, S.paged_window(c.q, kc, vc, c.block_table, None, lens, scale, window, sinks,
                                      bound=True), what)
    _ok(what)


@pytest.mark.parametrize("seed", range(20))
def test_rotation_and_append(seed):
    rng = random.Random(7000 + seed)
    Hq, Hkv = _heads(rng)
    d, page = rng.choice([64, 128]), rng.choice([16, 48, 64, 256])
    rot = 16 * rng.randint(1, d // 16)
    inter = rng.random() < 0.5
    freq, m = rope_frequencies(rot, scaling=rng.choice(["linear", "ramp"]), factor=rng.choice([1.0, 8.0]))
    new = [rng.choice([0, 1, _n(rng, 200)]) for _ in range(rng.randint(1, 40))]
    if sum(new) == 0:
        new[0] = 3
    total = _lengths(rng, new)
    c = W.paged_inputs(torch.tensor(total, dtype=torch.int32), 1, Hkv, d, page, 8000 + seed,
                       extra_pages=2)
    cu = W.cu_seqlens(new)
    qkv = W.randn_bf16((sum(new), Hq + 2 * Hkv, d), 8100 + seed)
    split = lambda x: (x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:])  # noqa: E731
    dev = qkv.to(DEV)
    q, k, v = split(dev)
    kc, vc = c.k_cache.to(DEV), c.v_cache.to(DEV)
    got = attn_append_paged(k, v, kc, vc, c.block_table.to(DEV), c.seq_lens.to(DEV), cu.to(DEV), q=q,
                            inv_freq=freq.to(DEV), interleaved=inter, mscale=m)
    qo, kr, vr, places = S.append_paged(*split(qkv), c.k_cache, c.v_cache, c.block_table, c.seq_lens,
                                        cu, freq, inter, m)
    tok, page_of, row = (np.array([p[i] for p in places]) for i in (0, 3, 4))
    n = len(freq)
    hq, hk, hv = split(qkv)

    def near(a, want, x):
        tol = np.abs(want) * 2.0 ** -8 + 1e-6 * abs(m) * S.pair_weight(x, n, inter)
        assert (np.abs(S.f64(a) - want) <= tol).all(), seed

    near(got, qo, hq)
    near(kc.cpu()[page_of, row], kr[page_of, row], hk[tok])
    assert torch.equal(vc.cpu()[page_of, row], hv[tok])
    left = np.ones(kc.shape[:2], dtype=bool)
    left[page_of, row] = False
    for have, was in ((kc, c.k_cache), (vc, c.v_cache)):
        assert torch.equal(have.cpu()[torch.tensor(left)], was[torch.tensor(left)])
    # the same tokens through the rotation alone
    pos = torch.tensor([p[2] for p in places], dtype=torch.int32)
    qr, kr2 = attn_rope(q.transpose(0, 1)[None], k.transpose(0, 1)[None], freq.to(DEV), pos.to(DEV),
                        interleaved=inter, mscale=m)
    assert torch.equal(qr[0].transpose(0, 1), got)
    assert torch.equal(kr2[0].transpose(0, 1).cpu(), kc.cpu()[page_of, row])
    _ok(seed)
