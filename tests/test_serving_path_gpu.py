"""The new operators run together, as a serving loop and a training step use them, each against
the float64 oracle of the whole path.

Serving: prompts are projected (here: drawn), their Q and K rotated, K and V appended to a paged
cache and attended with a window and first tokens; more chunks follow, then single tokens, with
the calls of a decode step captured into one CUDA graph and replayed.  The oracle keeps its own
float64 history of every sequence's rotated keys and values.

The cache holds bf16 (or E4M3) roundings of the rotated keys, which the oracle's attention
reads back from the cache that the kernels filled; the append itself is compared with the
oracle's rotation at its own tolerance (tests/test_append_gpu.py).  So every stage is checked
against what it was given.
"""
import math

import numpy as np
import pytest
import torch

from exact_softmax_attention_fwd_b200 import (attn_append_paged, attn_append_paged_fp8,
                                             attn_bwd_window_sinks, attn_decode_paged,
                                             attn_decode_paged_window,
                                             attn_decode_paged_window_fp8, attn_fwd_paged,
                                             attn_fwd_paged_window, attn_fwd_window_sinks,
                                             attn_get_device_error, attn_rope, attn_rope_bwd,
                                             rope_frequencies)
from exact_softmax_attention_fwd_b200 import workloads as W
from oracle import serving as S
from oracle.kv_fp8 import dequantize

from parity import check_grad
from window_parity import check_rows

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
HQ, HKV, D, PAGE, WINDOW, SINKS = 8, 2, 128, 16, 70, 4
SCALE = 1 / math.sqrt(D)


def _ok():
    st, flags = attn_get_device_error()
    assert st == 0, f"device error flags {flags:#x}"


def _split(qkv):
    return qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:]


def _rows_close(got, x, pos, freq):
    """got [n, H, d] is x turned at positions pos [n], to the rotation's tolerance."""
    want = S.rotate(S.f64(x).transpose(1, 0, 2), pos, freq).transpose(1, 0, 2)
    tol = np.abs(want) * 2.0 ** -8 + 1e-6 * S.pair_weight(x, len(freq))
    assert (np.abs(S.f64(got) - want) <= tol).all()


def test_chunks_then_tokens_over_a_bf16_cache():
    lens = [0, 0, 0]
    chunks = [[100, 17, 1], [60, 0, 33], [9, 200, 40]]
    steps = 4
    most = max(sum(c[b] for c in chunks) for b in range(3)) + steps
    per = -(-most // PAGE)
    perm = torch.randperm(3 * per, generator=torch.Generator().manual_seed(9))
    table = perm.view(3, per).to(torch.int32)
    kc = torch.full((3 * per, PAGE, HKV, D), float("nan"), dtype=torch.bfloat16, device=DEV)
    vc = torch.full_like(kc, float("nan"))
    freq = rope_frequencies(D)[0]
    tabled, freqd = table.to(DEV), freq.to(DEV)
    history = [[] for _ in range(3)]   # (unrotated k, v) of each sequence

    def cache_matches():
        for b, h in enumerate(history):
            if not h:
                continue
            k, v = torch.cat([x[0] for x in h]), torch.cat([x[1] for x in h])
            n = k.shape[0]
            got = S.gather_pages(S.f64(kc), table[b], n), S.gather_pages(S.f64(vc), table[b], n)
            _rows_close(got[0], k, np.arange(n), freq)
            assert np.array_equal(got[1], S.f64(v))

    for i, new in enumerate(chunks):
        lens = [a + n for a, n in zip(lens, new)]
        qkv = W.randn_bf16((sum(new), HQ + 2 * HKV, D), 300 + i)
        cu = W.cu_seqlens(new)
        q, k, v = _split(qkv.to(DEV))
        seq = torch.tensor(lens, dtype=torch.int32)
        qr = attn_append_paged(k, v, kc, vc, tabled, seq.to(DEV), cu.to(DEV), q=q, inv_freq=freqd)
        pos = np.concatenate([np.arange(t - n, t) for n, t in zip(new, lens)])
        _rows_close(qr, _split(qkv)[0], pos, freq)
        for b in range(3):
            history[b].append(tuple(x[int(cu[b]):int(cu[b + 1])] for x in _split(qkv)[1:]))
        o, lse = attn_fwd_paged_window(qr, kc, vc, tabled, cu.to(DEV), seq.to(DEV), max(new), SCALE,
                                       WINDOW, SINKS)
        _ok()
        cache_matches()
        check_rows(o, lse, S.paged_window(qr, kc, vc, table, cu, lens, SCALE, WINDOW, SINKS,
                                          bound=True), f"chunk {i}")
    # decode: append and attend, captured once; the lengths live on the device
    qkv = torch.zeros(3, HQ + 2 * HKV, D, dtype=torch.bfloat16, device=DEV)
    seq = torch.tensor(lens, dtype=torch.int32, device=DEV)

    def step():
        q, k, v = _split(qkv)
        qr = attn_append_paged(k, v, kc, vc, tabled, seq, q=q, inv_freq=freqd)
        return (qr,) + attn_decode_paged_window(qr, kc, vc, tabled, seq, SCALE, WINDOW, SINKS)

    seq += 1                                     # the place of the first decoded token
    first = W.randn_bf16(tuple(qkv.shape), 400)
    qkv.copy_(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qr, o, lse = step()
    for i in range(steps):
        host = W.randn_bf16(tuple(qkv.shape), 400 + i)
        qkv.copy_(host)
        if i:
            seq += 1
        lens = [n + 1 for n in lens]
        graph.replay()
        torch.cuda.synchronize()
        assert seq.tolist() == lens
        _rows_close(qr, _split(host)[0], np.array(lens) - 1, freq)
        for b in range(3):
            history[b].append(tuple(x[b:b + 1] for x in _split(host)[1:]))
        cache_matches()
        check_rows(o, lse, S.paged_window(qr, kc, vc, table, None, lens, SCALE, WINDOW, SINKS,
                                          bound=True), f"token {i}")
    _ok()


def test_the_cache_serves_the_calls_that_were_there():
    """A cache filled by the append, slots behind the ends zeroed, read by the full-attention
    prefill and decode."""
    new, total = [50, 7], [50, 30]
    c = W.paged_inputs(torch.tensor(total, dtype=torch.int32), HQ, HKV, D, PAGE, 302)
    kc, vc = torch.zeros_like(c.k_cache).to(DEV), torch.zeros_like(c.v_cache).to(DEV)
    table, freq = c.block_table.to(DEV), rope_frequencies(D)[0].to(DEV)
    full = W.randn_bf16((sum(total), HQ + 2 * HKV, D), 303)
    q, k, v = _split(full.to(DEV))
    lens = torch.tensor(total, dtype=torch.int32, device=DEV)
    attn_append_paged(k, v, kc, vc, table, lens, W.cu_seqlens(total).to(DEV), inv_freq=freq)
    cu = W.cu_seqlens(new)
    o, lse = attn_fwd_paged(q[:57].contiguous(), kc, vc, table, cu.to(DEV), lens, 50, True, SCALE)
    check_rows(o, lse, S.paged_window(q[:57], kc, vc, c.block_table, cu, total, SCALE, 0, 0,
                                      bound=True))
    o, lse = attn_decode_paged(q[:2].contiguous(), kc, vc, table, lens, SCALE)
    check_rows(o, lse, S.paged_window(q[:2], kc, vc, c.block_table, None, total, SCALE, 0, 0,
                                      bound=True))
    _ok()


def test_tokens_over_an_e4m3_cache():
    total = [90, 33, 16]
    c = W.fp8_paged_inputs(torch.tensor(total, dtype=torch.int32), HQ, HKV, D, PAGE, 304)
    kc, vc = torch.full_like(c.k_cache, 0x7F).to(DEV), torch.full_like(c.v_cache, 0x7F).to(DEV)
    ks, vs, table = c.k_scale.to(DEV), c.v_scale.to(DEV), c.block_table.to(DEV)
    freq = rope_frequencies(D)[0].to(DEV)
    qkv = W.randn_bf16((sum(total), HQ + 2 * HKV, D), 305)
    q, k, v = _split(qkv.to(DEV))
    lens = torch.tensor(total, dtype=torch.int32, device=DEV)
    qr = attn_append_paged_fp8(k, v, kc, vc, ks, vs, table, lens, W.cu_seqlens(total).to(DEV), q=q,
                               inv_freq=freq)
    last = W.cu_seqlens(total)[1:].long() - 1
    ql = qr[last.to(DEV)].contiguous()
    o, lse = attn_decode_paged_window_fp8(ql, kc, vc, ks, vs, table, lens, SCALE, WINDOW, SINKS)
    _ok()
    kd, vd = dequantize(kc.cpu().numpy(), ks.cpu().numpy()), dequantize(vc.cpu().numpy(), vs.cpu().numpy())
    check_rows(o, lse, S.paged_window(ql, kd, vd, c.block_table, None, total, SCALE, WINDOW, SINKS,
                                      bound=True))


@pytest.mark.parametrize("interleaved", [False, True])
def test_training_step_gradients(interleaved):
    """qkv -> rotation -> attention -> sum(dO * O), and back into one buffer of d(qkv), against
    the oracle's gradients of the same chain (from the unrounded rotation: the rotated Q and K
    carry a bf16 rounding of 2^-8, which the gradients' bar of 5e-3 in norm covers: a rounding
    error is uniform, 2^-8 / sqrt(3) = 2.3e-3 of its value's norm at most)."""
    n = 300
    qkv = W.randn_bf16((2, n, HQ + 2 * HKV, D), 306)
    do = W.grad_output(2, HQ, n, D, 307)
    freq, m = rope_frequencies(64, scaling="linear", factor=2.0)
    pos = torch.arange(n, dtype=torch.int32)
    dev, freqd, posd = qkv.to(DEV), freq.to(DEV), pos.to(DEV)
    kw = dict(interleaved=interleaved, mscale=m)
    heads = lambda x, a, b: x[:, :, a:b].transpose(1, 2)  # noqa: E731
    q, k = attn_rope(heads(dev, 0, HQ), heads(dev, HQ, HQ + HKV), freqd, posd, **kw)
    v = heads(dev, HQ + HKV, HQ + 2 * HKV).contiguous()
    o, lse = attn_fwd_window_sinks(q, k, v, SCALE, WINDOW, SINKS)
    grad = torch.full_like(dev, float("nan"))
    dq, dk, dv = attn_bwd_window_sinks(q, k, v, o, lse, do.to(DEV), SCALE, WINDOW, SINKS)
    attn_rope_bwd(dq, dk, freqd, posd, **kw, q_out=heads(grad, 0, HQ), k_out=heads(grad, HQ, HQ + HKV))
    heads(grad, HQ + HKV, HQ + 2 * HKV).copy_(dv)
    torch.cuda.synchronize()
    _ok()
    hq, hk = heads(qkv, 0, HQ), heads(qkv, HQ, HQ + HKV)
    rq, rk = (S.rotate(x, pos, freq, interleaved, m) for x in (hq, hk))
    rdq, rdk, rdv = S.window_grads(rq, rk, heads(qkv, HQ + HKV, HQ + 2 * HKV), do, SCALE, WINDOW, SINKS)
    back = -pos.double()
    want = [S.rotate(rdq, back, freq, interleaved, m), S.rotate(rdk, back, freq, interleaved, m), rdv]
    got = [heads(grad, 0, HQ), heads(grad, HQ, HQ + HKV), heads(grad, HQ + HKV, HQ + 2 * HKV)]
    for name, g, w in zip(("dq", "dk", "dv"), got, want):
        if name == "dv":
            check_grad(g, w, name)
            continue
        # the rounding of Q, K (through P and dS) and of dQ, dK before the rotation back come
        # on top of the backward's own error: three independent errors of at most 5e-3, 2.3e-3
        # (dS meets the rounded operand) and 2.3e-3 of the norm
        g, w = S.f64(g), np.asarray(w)
        assert np.linalg.norm(g - w) <= math.sqrt(5e-3 ** 2 + 2 * 2.3e-3 ** 2) * np.linalg.norm(w), name


def test_two_streams_at_once():
    """The same calls on two streams with work of different sizes in flight together, many times:
    the bits of each stream's results are those of the calls alone (units that a CTA takes over,
    clusters and workspaces belong to their own launch)."""
    def work(seed, n, window):
        q, k, v = (x.to(DEV) for x in W.prefill_inputs(1, 8, 2, n, n, 128, seed))
        do = W.grad_output(1, 8, n, 128, seed).to(DEV)
        c = W.paged_inputs(torch.tensor([n, 33, 700], dtype=torch.int32), 8, 2, 128, 16, seed)
        paged = [x.to(DEV) for x in (c.q, c.k_cache, c.v_cache, c.block_table, c.seq_lens)]
        freq = rope_frequencies(128)[0].to(DEV)

        def run(stream):
            a, b = attn_rope(q, k, freq, stream=stream)
            o, lse = attn_fwd_window_sinks(a, b, v, 0.088, window, 4, stream=stream)
            grads = attn_bwd_window_sinks(a, b, v, o, lse, do, 0.088, window, 4, stream=stream)
            return (o, lse) + grads + attn_decode_paged_window(*paged, 0.088, window, 4, stream=stream)

        return run

    calls = [work(311, 3000, 200), work(312, 900, 64)]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    want = []
    for call, s in zip(calls, streams):
        torch.cuda.synchronize()
        want.append(call(s))
        torch.cuda.synchronize()
    for _ in range(10):
        got = [[call(s) for _ in range(3)] for call, s in zip(calls, streams)]
        torch.cuda.synchronize()
        for runs, ref in zip(got, want):
            for r in runs:
                assert all(torch.equal(x, y) for x, y in zip(r, ref))
    _ok()
