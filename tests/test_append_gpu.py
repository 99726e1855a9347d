"""GPU parity of attn_append_paged and attn_append_paged_fp8 against the float64 oracle.

bf16 caches and the rotated queries: the tolerance of the rotation (half a bf16
step plus 1e-6 of the pair's |a| + |b|).  E4M3 caches hold the value nearest to
x / scale: half a step (2^-4 of the value, 2^-10 below the smallest normal),
plus the rotation's and the fp32 division's error.  Every other slot of the
cache keeps its bits.
"""
import numpy as np
import pytest
import torch

from exact_softmax_attention_fwd_b200 import (AttnError, attn_append_paged, attn_append_paged_fp8,
                                             attn_get_device_error, rope_frequencies)
from exact_softmax_attention_fwd_b200 import _binding as B
from exact_softmax_attention_fwd_b200 import workloads as W
from oracle import serving as S
from oracle.kv_fp8 import e4m3_to_float

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _case(new, total, Hq, Hkv, d, page, seed, extra=0, fp8=False, single=False):
    """(q, k, v views of a fused projection, cache inputs, cu_seqlens or None) on the host."""
    make = W.fp8_paged_inputs if fp8 else W.paged_inputs
    c = make(total, 1, Hkv, d, page, seed, extra_pages=3, max_pages_per_seq=None)
    n = (len(total) if single else sum(new)) + extra
    qkv = W.randn_bf16((n, Hq + 2 * Hkv, d), seed + 7)
    return qkv, c, None if single else W.cu_seqlens(new)


def _split(qkv, Hq, Hkv):
    return qkv[:, :Hq] if Hq else None, qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]


def _run(qkv, c, cu, Hq, Hkv, freq, inter, m, pos=None, fp8=False, q_out=None):
    q, k, v = _split(qkv.to(DEV), Hq, Hkv)
    kc, vc = c.k_cache.to(DEV), c.v_cache.to(DEV)
    args = dict(cu_seqlens=None if cu is None else cu.to(DEV), q=q,
                inv_freq=None if freq is None else freq.to(DEV), interleaved=inter, mscale=m,
                positions=None if pos is None else pos.to(DEV), q_out=q_out)
    table, lens = c.block_table.to(DEV), c.seq_lens.to(DEV)
    if fp8:
        got = attn_append_paged_fp8(k, v, kc, vc, c.k_scale.to(DEV), c.v_scale.to(DEV), table, lens,
                                    **args)
    else:
        got = attn_append_paged(k, v, kc, vc, table, lens, **args)
    torch.cuda.synchronize()
    return got, kc.cpu(), vc.cpu()


def _check(qkv, c, cu, Hq, Hkv, freq, inter, m, pos, fp8, got, kc, vc, table=None):
    q, k, v = _split(qkv, Hq, Hkv)
    table = c.block_table if table is None else table
    value = e4m3_to_float if fp8 else S.f64
    n = 0 if freq is None else len(freq)
    scales = dict(k_scale=c.k_scale.numpy(), v_scale=c.v_scale.numpy()) if fp8 else {}
    qo, kr, vr, places = S.append_paged(q, k, v, value(c.k_cache), value(c.v_cache), table,
                                        c.seq_lens, cu, freq, inter, m, pos, **scales)
    written = np.zeros(kc.shape[:2], dtype=bool)
    for tok, _, _, page, row in places:
        written[page, row] = True
        weight = S.pair_weight(k[tok], n, inter) * abs(m) * 1e-6
        if fp8:
            z, zv = kr[page, row], vr[page, row]
            ks, vs = (scales[x][page][:, None].astype(np.float64) for x in ("k_scale", "v_scale"))
            exact_k = S.rotate(S.f64(k[tok])[:, None], [0], np.zeros(0))[:, 0] if n == 0 else \
                S.rotate(S.f64(k[tok])[:, None],
                         [S.f64(pos)[tok] if pos is not None else _key(c, cu, tok)], freq, inter,
                         m)[:, 0]
            for got8, near, x, sc, w in ((kc, z, exact_k, ks, weight), (vc, zv, S.f64(v[tok]), vs, 0.0)):
                y = np.clip(np.where(sc != 0, x / np.where(sc != 0, sc, 1.0), 0.0), -448, 448)
                err = np.abs(y) * 2.0 ** -22 + \
                    np.where(sc != 0, w / np.where(sc != 0, np.abs(sc), 1.0), 0.0)
                tol = np.maximum(np.abs(y) * 2.0 ** -4, 2.0 ** -10) + err
                have = value(got8[page, row].numpy())
                assert (np.abs(have - y) <= tol).all(), (tok, page, row)
                # and the very code, unless the value lies within its error of the border
                # (the middle) between the two: bf16 values over a scale of amax / 448 often do
                border = np.abs((have + near) / 2 - y) <= err
                assert ((have == near) | border).all(), (tok, page, row)
        else:
            tol = np.abs(kr[page, row]) * 2.0 ** -8 + weight
            tol[:, 2 * n:] = 0.0
            assert (np.abs(S.f64(kc[page, row]) - kr[page, row]) <= tol).all(), (tok, page, row)
            assert torch.equal(vc[page, row], v[tok])
        if q is not None:
            tol = np.abs(qo[tok]) * 2.0 ** -8 + 1e-6 * abs(m) * S.pair_weight(q[tok], n, inter)
            tol[:, 2 * n:] = 0.0
            assert (np.abs(S.f64(got[tok]) - qo[tok]) <= tol).all(), tok
    for have, was in ((kc, c.k_cache), (vc, c.v_cache)):
        left = torch.tensor(~written)
        assert torch.equal(have[left].view(torch.uint8), was[left].view(torch.uint8))
    return places


def _key(c, cu, tok):
    if cu is None:
        return int(c.seq_lens[tok]) - 1
    b = int((cu[1:] <= tok).sum())
    return int(c.seq_lens[b]) - (int(cu[b + 1]) - tok)


CASES = [
    # new tokens, lengths with them, Hq, Hkv, d, page, rotary (0: none), interleaved, scaling
    ([1], [1], 1, 1, 64, 16, 64, False, "none"),
    ([5, 0, 17], [5, 40, 33], 4, 2, 128, 16, 128, False, "none"),
    ([33, 1, 64, 2], [100, 129, 64, 257], 8, 2, 64, 32, 32, True, "linear"),
    ([130], [1000], 2, 1, 128, 128, 48, True, "ramp"),
    ([3, 3], [16, 48], 0, 4, 128, 48, 128, False, "none"),
    ([40, 9], [40, 300], 3, 1, 64, 256, 0, False, "none"),
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", CASES, ids=str)
def test_ragged_tokens(case, fp8):
    new, total, Hq, Hkv, d, page, rot, inter, scaling = case
    freq, m = rope_frequencies(rot, scaling=scaling, factor=1.0 if scaling == "none" else 4.0) \
        if rot else (None, 1.0)
    qkv, c, cu = _case(new, total, Hq, Hkv, d, page, 51, fp8=fp8)
    got = _run(qkv, c, cu, Hq, Hkv, freq, inter, m, fp8=fp8)
    _check(qkv, c, cu, Hq, Hkv, freq, inter, m, None, fp8, *got)
    assert (got[0] is None) == (Hq == 0)
    assert attn_get_device_error()[0] == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_single_tokens_and_idle_rows(fp8):
    total = [1, 0, 16, 17, 900, 0, 32]
    Hq, Hkv, d = 8, 2, 128
    freq, m = rope_frequencies(128)
    qkv, c, _ = _case(None, total, Hq, Hkv, d, 16, 52, fp8=fp8, single=True)
    q_out = torch.full((7, Hq, d), 3.0, dtype=torch.bfloat16, device=DEV)
    got = _run(qkv, c, None, Hq, Hkv, freq, False, m, fp8=fp8, q_out=q_out)
    places = _check(qkv, c, None, Hq, Hkv, freq, False, m, None, fp8, *got)
    assert [p[0] for p in places] == [0, 2, 3, 4, 6]
    assert bool((got[0][[1, 5]] == 3.0).all())
    assert attn_get_device_error()[0] == 0


def test_many_sequences_and_positions_of_their_own():
    g = torch.Generator().manual_seed(3)
    new = torch.randint(0, 4, (300,), generator=g).tolist()
    total = [n + int(x) for n, x in zip(new, torch.randint(0, 60, (300,), generator=g))]
    total = [max(t, 1) for t in total]
    qkv, c, cu = _case(new, total, 2, 1, 64, 16, 53)
    pos = torch.randint(-1000, 10 ** 6, (sum(new),), generator=g, dtype=torch.int32)
    freq, m = rope_frequencies(64)
    got = _run(qkv, c, cu, 2, 1, freq, True, m, pos=pos)
    _check(qkv, c, cu, 2, 1, freq, True, m, pos, False, *got)


def test_tokens_behind_the_last_sequence_are_left_alone():
    new, total = [4, 3], [20, 3]
    qkv, c, cu = _case(new, total, 2, 2, 64, 16, 54, extra=5)
    q_out = torch.full((12, 2, 64), -2.0, dtype=torch.bfloat16, device=DEV)
    freq, m = rope_frequencies(64)
    got = _run(qkv, c, cu, 2, 2, freq, False, m, q_out=q_out)
    _check(qkv, c, cu, 2, 2, freq, False, m, None, False, *got)
    assert bool((got[0][7:] == -2.0).all())
    assert attn_get_device_error()[0] == 0


def test_bad_pages_are_skipped_and_flagged():
    new, total = [20, 4], [20, 4]
    qkv, c, cu = _case(new, total, 2, 1, 64, 16, 55)
    for bad in (-1, c.num_pages, 2 ** 31 - 1):
        c2 = W.PagedInputs(c.q, c.k_cache, c.v_cache, c.block_table.clone(), c.seq_lens, 16)
        good = int(c.block_table[0, 1])
        c2.block_table[0, 1] = bad
        freq, m = rope_frequencies(64)
        qo, kc, vc = _run(qkv, c2, cu, 2, 1, freq, False, m)
        st, flags = attn_get_device_error()
        assert st == B.ATTN_ERR_DEVICE and flags == B.DEVERR_BAD_PAGE
        full, kf, vf = _run(qkv, c, cu, 2, 1, freq, False, m)
        assert torch.equal(qo, full)          # the queries do not need the page
        assert torch.equal(kc[good].view(torch.uint8), c.k_cache[good].view(torch.uint8))
        rest = [p for p in range(c.num_pages) if p != good]
        assert torch.equal(kc[rest], kf[rest]) and torch.equal(vc[rest], vf[rest])


@pytest.mark.parametrize("lens,offsets", [
    ([3, 9], None),            # 4 new tokens in a sequence of 3
    ([-1, 9], None),
    ([10 ** 6, 9], None),      # beyond the block table
    ([20, 9], [0, 4, 3]),      # offsets that decrease
    ([20, 9], [0, 4, 99]),     # beyond the tokens
])
def test_bad_lengths_are_skipped_and_flagged(lens, offsets):
    qkv, c, cu = _case([4, 3], [20, 9], 2, 1, 64, 16, 56)
    cu2 = cu if offsets is None else torch.tensor(offsets, dtype=torch.int32)
    c2 = W.PagedInputs(c.q, c.k_cache, c.v_cache, c.block_table,
                       torch.tensor(lens, dtype=torch.int32), 16)
    freq, m = rope_frequencies(64)
    q_out = torch.full((7, 2, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    qo, kc, vc = _run(qkv, c2, cu2, 2, 1, freq, False, m, q_out=q_out)
    st, flags = attn_get_device_error()
    assert st == B.ATTN_ERR_DEVICE and flags == B.DEVERR_BAD_LENGTH
    bad = 0 if offsets is None else 1
    ids = [p for p in c.block_table[bad].tolist() if p >= 0]
    assert torch.equal(kc[ids].view(torch.uint8), c.k_cache[ids].view(torch.uint8))
    assert torch.equal(vc[ids].view(torch.uint8), c.v_cache[ids].view(torch.uint8))
    rows = slice(0, 4) if bad == 0 else slice(4, 7)
    assert bool((qo[rows] == 5.0).all())


def test_scales_of_zero_and_below_and_saturation():
    qkv, c, cu = _case([3, 2, 2, 3], [3, 18, 2, 5], 0, 2, 64, 16, 57, fp8=True)
    c.k_scale[int(c.block_table[0, 0])] = 0.0
    c.v_scale[int(c.block_table[1, 1])] *= -1.0
    c.v_scale[int(c.block_table[2, 0])] *= 2.0 ** -6     # most values beyond 448
    c.k_scale[int(c.block_table[3, 0])] *= 2.0 ** 12     # subnormal codes and zeros
    freq, m = rope_frequencies(64)
    got = _run(qkv, c, cu, 0, 2, freq, False, m, fp8=True)
    _check(qkv, c, cu, 0, 2, freq, False, m, None, True, *got)
    page = int(c.block_table[2, 0])
    assert int((got[2][page, :2] & 0x7F == 0x7E).sum()) > 100


def test_queries_in_place_and_other_stream_and_graph():
    new, total = [6, 1], [30, 17]
    Hq, Hkv, d = 4, 2, 128
    qkv, c, cu = _case(new, total, Hq, Hkv, d, 16, 58)
    freq, m = rope_frequencies(128)
    want, kw, vw = _run(qkv, c, cu, Hq, Hkv, freq, False, m)
    q, k, v = (x.contiguous().to(DEV) for x in _split(qkv, Hq, Hkv))
    table, lens, cud, f = c.block_table.to(DEV), c.seq_lens.to(DEV), cu.to(DEV), freq.to(DEV)
    kc, vc = c.k_cache.to(DEV), c.v_cache.to(DEV)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    q2 = q.clone()
    side.wait_stream(torch.cuda.current_stream())
    got = attn_append_paged(k, v, kc, vc, table, lens, cud, q=q2, inv_freq=f, q_out=q2, stream=side)
    side.synchronize()
    assert got is q2 and torch.equal(q2, want)
    assert torch.equal(kc.cpu(), kw) and torch.equal(vc.cpu(), vw)
    with pytest.raises(ValueError):
        attn_append_paged(k, v, kc, vc, table, lens, cud, q=qkv.to(DEV)[:, :Hq], inv_freq=f,
                          q_out=qkv.to(DEV)[:, :Hq])
    # captured: the next step's lengths, in the same buffers
    kc.copy_(c.k_cache)
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        attn_append_paged(k, v, kc, vc, table, lens, cud, q=q, inv_freq=f, q_out=out)
    lens += 1
    kc.copy_(c.k_cache)
    vc.copy_(c.v_cache)
    g.replay()
    torch.cuda.synchronize()
    c2 = W.PagedInputs(c.q, c.k_cache, c.v_cache, c.block_table, c.seq_lens + 1, 16)
    want, kw, vw = _run(qkv, c2, cu, Hq, Hkv, freq, False, m)
    assert torch.equal(out, want) and torch.equal(kc.cpu(), kw) and torch.equal(vc.cpu(), vw)


@pytest.mark.parametrize("fp8", [False, True])
def test_pool_beyond_32_bit_offsets(fp8):
    pages, page, Hkv, d = 140000, 16, 8, 128      # 2.3e9 elements
    free, _ = torch.cuda.mem_get_info()
    if free < 14 << 30:
        pytest.skip("needs 14 GB of free device memory")
    dtype = torch.uint8 if fp8 else torch.bfloat16
    kc = torch.zeros(pages, page, Hkv, d, dtype=dtype, device=DEV)
    vc = torch.zeros_like(kc)
    table = torch.tensor([[pages - 1], [3]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([16, 2], dtype=torch.int32, device=DEV)
    k = torch.ones(2, Hkv, d, dtype=torch.bfloat16, device=DEV)
    if fp8:
        scale = torch.ones(pages, Hkv, device=DEV)
        attn_append_paged_fp8(k, k, kc, vc, scale, scale, table, lens)
        kc, vc = kc.view(torch.float8_e4m3fn), vc.view(torch.float8_e4m3fn)
    else:
        attn_append_paged(k, k, kc, vc, table, lens)
    for cache in (kc, vc):
        assert bool((cache[pages - 1, 15].float() == 1.0).all())
        assert bool((cache[3, 1].float() == 1.0).all())
        written = cache.view(torch.uint8).view(pages, -1).amax(1)
        assert written.nonzero().flatten().tolist() == [3, pages - 1]


def test_binding_refusals():
    qkv, c, cu = _case([2, 1], [2, 5], 2, 1, 64, 16, 59)
    q, k, v = _split(qkv.to(DEV), 2, 1)
    kc, vc = c.k_cache.to(DEV), c.v_cache.to(DEV)
    table, lens, cud = c.block_table.to(DEV), c.seq_lens.to(DEV), cu.to(DEV)
    f = rope_frequencies(64)[0].to(DEV)
    with pytest.raises(ValueError):
        attn_append_paged(k, v, kc, vc, table, lens)              # 3 tokens, 2 sequences
    with pytest.raises(ValueError):
        attn_append_paged(k.float(), v, kc, vc, table, lens, cud)
    with pytest.raises(ValueError):
        attn_append_paged(k, v, kc.float(), vc.float(), table, lens, cud)
    with pytest.raises(ValueError):
        attn_append_paged(k, v, kc, vc, table.long(), lens, cud)
    with pytest.raises(ValueError):
        attn_append_paged(k, v, kc, vc, table, lens[:1], cud)
    with pytest.raises(ValueError):
        attn_append_paged(k, v, kc, vc, table, lens, cud, q=q[:2], inv_freq=f)
    with pytest.raises(ValueError):
        attn_append_paged(k, v, kc, vc, table, lens, cud, inv_freq=f.float())
    with pytest.raises(ValueError):
        attn_append_paged(k, v, kc, vc, table, lens, cud, q_out=torch.empty(3, 2, 64, device=DEV))
    with pytest.raises(ValueError):
        attn_append_paged(k, v, kc, vc, table.cpu(), lens, cud)
    with pytest.raises(ValueError):
        attn_append_paged_fp8(k, v, kc, vc, f, f, table, lens, cud)
    with pytest.raises(AttnError):
        attn_append_paged(k, v, kc, vc, table, lens, cud, inv_freq=f[:4])   # 8 turned elements
    assert torch.equal(kc.cpu(), c.k_cache)


def test_q_out_at_the_address_of_strided_queries_is_refused():
    """q as a view of the fused projection, q_out contiguous from the same address: other rows
    of q would be overwritten before they are read."""
    Hq, Hkv, d, total = 4, 2, 64, [40, 9]
    qkv, c, _ = _case([1, 1], total, Hq, Hkv, d, 16, 61, single=True)
    x = qkv.to(DEV)
    q, k, v = _split(x, Hq, Hkv)
    q_out = x.view(-1)[:2 * Hq * d].view(2, Hq, d)
    assert q_out.is_contiguous() and q_out.data_ptr() == q.data_ptr()
    kc, vc = c.k_cache.to(DEV), c.v_cache.to(DEV)
    with pytest.raises(ValueError, match="itself"):
        attn_append_paged(k, v, kc, vc, c.block_table.to(DEV), c.seq_lens.to(DEV), q=q, q_out=q_out)
    assert torch.equal(x.cpu(), qkv) and torch.equal(kc.cpu(), c.k_cache)
