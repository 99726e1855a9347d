"""GPU parity of single-token attention over a paged cache with a sliding window and visible
first tokens (bf16 and E4M3 caches) against the float64 oracle, at the bar of
tests/window_parity.py (the E4M3 kernel rounds its weights to f16, finer than the bar's bf16)."""
import math
from dataclasses import replace

import pytest
import torch

from exact_softmax_attention_fwd_b200 import (AttnError, attn_decode_paged, attn_decode_paged_fp8,
                                             attn_decode_paged_window,
                                             attn_decode_paged_window_fp8, attn_get_device_error)
from exact_softmax_attention_fwd_b200 import _binding as B
from exact_softmax_attention_fwd_b200 import workloads as W
from oracle import serving as S
from oracle.kv_fp8 import dequantize

from window_parity import check_rows

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _ok():
    st, flags = attn_get_device_error()
    assert st == 0, f"device error flags {flags:#x}"


def _make(lens, Hq, Hkv, d, page, seed, fp8, **kw):
    lens = torch.tensor(lens, dtype=torch.int32)
    return (W.fp8_paged_inputs if fp8 else W.paged_inputs)(lens, Hq, Hkv, d, page, seed, **kw)


def _call(c, scale, window, sinks, fp8, kc=None, vc=None, table=None, lens=None, **kw):
    kc, vc = c.k_cache if kc is None else kc, c.v_cache if vc is None else vc
    table, lens = c.block_table if table is None else table, c.seq_lens if lens is None else lens
    q, kc, vc, table, lens = (x.to(DEV) for x in (c.q, kc, vc, table, lens))
    if fp8:
        return attn_decode_paged_window_fp8(q, kc, vc, c.k_scale.to(DEV), c.v_scale.to(DEV), table,
                                            lens, scale, window, sinks, **kw)
    return attn_decode_paged_window(q, kc, vc, table, lens, scale, window, sinks, **kw)


def _ref(c, scale, window, sinks, fp8):
    kc, vc = (dequantize(c.k_cache.numpy(), c.k_scale.numpy()),
              dequantize(c.v_cache.numpy(), c.v_scale.numpy())) if fp8 else (c.k_cache, c.v_cache)
    return S.paged_window(c.q, kc, vc, c.block_table, None, c.seq_lens, scale, window, sinks,
                          bound=True)


CASES = [
    # lengths, Hq, Hkv, d, page, window, sinks
    ([1], 1, 1, 64, 16, 1, 1),
    ([0, 1, 15, 16, 17, 33], 8, 2, 128, 16, 16, 4),
    ([100, 700, 0, 1500], 8, 1, 128, 16, 100, 4),
    ([100, 700, 333], 6, 2, 64, 48, 64, 20),
    ([500, 37], 4, 4, 128, 256, 1, 0),
    ([40, 50, 60, 70], 4, 2, 64, 32, 30, 25),          # first tokens and window in one chunk
    ([900], 4, 2, 128, 64, 128, 300),                  # many first tokens
    ([900, 20], 4, 2, 64, 16, 17, 2000),               # all keys are first tokens
    ([900, 20], 4, 2, 64, 16, 5000, 4),                # the window is every key
    ([900, 0], 4, 2, 128, 16, 0, 4),                   # no window
    ([900, 33], 4, 2, 64, 16, 2 ** 40, 2 ** 35),       # counts beyond an int
    ([5000], 2, 1, 64, 16, 4500, 4),                   # more chunks than one round of the warps holds
    ([2100] * 40, 8, 8, 64, 16, 2000, 5),              # several rounds in a cluster of one
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: str(c)[:60])
def test_parity(case, fp8):
    lens, Hq, Hkv, d, page, window, sinks = case
    c = _make(lens, Hq, Hkv, d, page, 211, fp8)
    scale = 1 / math.sqrt(d)
    o, lse = _call(c, scale, window, sinks, fp8)
    torch.cuda.synchronize()
    _ok()
    check_rows(o, lse, _ref(c, scale, window, sinks, fp8), str(case))
    again = _call(c, scale, window, sinks, fp8)
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("fp8", [False, True])
def test_every_length_around_the_edges(fp8):
    """Lengths 0..70 with a window of 20 and 3 first tokens: every place of the window's two
    ends in a chunk of 16."""
    c = _make(list(range(71)), 2, 1, 64, 16, 212, fp8)
    o, lse = _call(c, 0.2, 20, 3, fp8)
    _ok()
    check_rows(o, lse, _ref(c, 0.2, 20, 3, fp8))


@pytest.mark.parametrize("fp8", [False, True])
def test_slots_that_are_not_visible_may_hold_anything(fp8):
    lens, page, window, sinks = [300, 77, 16], 16, 60, 5
    c = _make(lens, 4, 2, 128, page, 213, fp8)
    kc, vc = c.k_cache.clone(), c.v_cache.clone()
    junk = 0x7F if fp8 else float("nan")
    table = c.block_table.clone()
    for b, n in enumerate(lens):
        for t in range(-(-n // page) * page):
            if not (t < n and (t >= n - window or t < sinks)):
                at = int(c.block_table[b, t // page]), t % page
                kc[at], vc[at] = junk, junk
        # pages without any visible key are not looked up
        for pg in range(table.shape[1]):
            seen = any(t < n and (t >= n - window or t < sinks) for t in range(pg * page, pg * page + page))
            if not seen:
                table[b, pg] = -7
    o, lse = _call(c, 0.1, window, sinks, fp8, kc=kc, vc=vc, table=table)
    _ok()
    check_rows(o, lse, _ref(c, 0.1, window, sinks, fp8))


@pytest.mark.parametrize("B_,window,sinks", [(1, 0, 0), (1, 200, 4), (40, 200, 4)])
@pytest.mark.parametrize("where", ["query", "keys"])
def test_nan_in_what_a_row_sees_reaches_its_result(where, B_, window, sinks):
    """A query of NaN, or a run of visible keys of NaN (all that some warps see): the rows that
    see them are NaN, O and LSE, and the others as ever."""
    c = _make([500] + [300] * (B_ - 1), 4, 2, 64, 16, 216, False)
    o0, lse0 = _call(c, 0.2, window, sinks, False)
    q, kc = c.q.clone(), c.k_cache.clone()
    hit = torch.zeros(B_, 4, dtype=torch.bool)
    if where == "query":
        q[0, 2] = float("nan")
        hit[0, 2] = True
    else:
        for t in range(448, 480, 16):
            kc[int(c.block_table[0, t // 16]), :, 1] = float("nan")
        hit[0, 2:] = True
    o, lse = _call(replace(c, q=q), 0.2, window, sinks, False, kc=kc)
    _ok()
    assert torch.isnan(o.cpu()[hit]).all() and torch.isnan(lse.cpu()[hit]).all()
    assert torch.equal(o.cpu()[~hit], o0.cpu()[~hit])
    assert torch.equal(lse.cpu()[~hit], lse0.cpu()[~hit])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 2.0])
def test_odd_scales(scale, fp8):
    c = _make([200, 40], 4, 2, 64, 16, 214, fp8)
    o, lse = _call(c, scale, 50, 4, fp8)
    check_rows(o, lse, _ref(c, scale, 50, 4, fp8))


def test_scales_of_zero_below_zero_and_far_apart():
    c = _make([2000], 4, 1, 128, 16, 215, True)
    g = torch.Generator().manual_seed(1)
    c.v_scale.mul_(torch.exp2(torch.randint(-8, 9, c.v_scale.shape, generator=g).float()))
    c.v_scale[::3] *= -1
    c.v_scale[::7] = 0.0
    c.k_scale[::5] = 0.0
    o, lse = _call(c, 0.09, 1500, 4, True)
    _ok()
    check_rows(o, lse, _ref(c, 0.09, 1500, 4, True))


@pytest.mark.parametrize("fp8", [False, True])
def test_a_window_of_everything_agrees_with_the_plain_decode(fp8):
    c = _make([1000, 513, 64], 16, 4, 128, 16, 216, fp8)
    o, lse = _call(c, 0.088, 0, 0, fp8)
    q, kc, vc, table, lens = (x.to(DEV) for x in (c.q, c.k_cache, c.v_cache, c.block_table, c.seq_lens))
    if fp8:
        o2, lse2 = attn_decode_paged_fp8(q, kc, vc, c.k_scale.to(DEV), c.v_scale.to(DEV), table, lens,
                                         0.088)
    else:
        o2, lse2 = attn_decode_paged(q, kc, vc, table, lens, 0.088)
    ref = _ref(c, 0.088, 0, 0, fp8)
    check_rows(o, lse, ref)
    check_rows(o2, lse2, ref)


def test_bad_pages_and_lengths_are_flagged():
    c = _make([200, 40], 4, 2, 64, 16, 217, False)
    table = c.block_table.clone()
    table[0, 11] = c.num_pages        # in the window
    o, lse = _call(c, 0.1, 50, 2, False, table=table)
    assert attn_get_device_error() == (B.ATTN_ERR_DEVICE, B.DEVERR_BAD_PAGE)
    assert bool(torch.isfinite(o).all())
    good, _ = _call(c, 0.1, 50, 2, False)
    assert torch.equal(o[1], good[1])
    _ok()
    cap = c.block_table.shape[1] * 16
    for bad in (-1, cap + 1):
        lens = c.seq_lens.clone()
        lens[1] = bad
        c2 = W.PagedInputs(c.q, c.k_cache, c.v_cache, c.block_table.clone().clamp(min=0), lens, 16)
        o, lse = _call(c2, 0.1, 50, 2, False)
        assert attn_get_device_error() == (B.ATTN_ERR_DEVICE, B.DEVERR_BAD_LENGTH)
        assert torch.equal(o[0], good[0])
        if bad < 0:                   # read as an empty sequence
            assert bool((o[1] == 0).all()) and bool(torch.isneginf(lse[1]).all())


def test_other_stream_two_graphs_and_growing_lengths():
    c = _make([300, 9], 8, 2, 128, 16, 218, False, max_pages_per_seq=40)
    c.block_table.clamp_(min=0)
    q, kc, vc, table, lens = (x.to(DEV) for x in (c.q, c.k_cache, c.v_cache, c.block_table, c.seq_lens))
    call = lambda **kw: attn_decode_paged_window(q, kc, vc, table, lens, 0.1, 100, 4, **kw)  # noqa: E731
    want = call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = call(stream=side)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call())
        graphs.append(g)
    for _ in range(3):
        lens += 5
        want = call()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for out in outs:
            assert torch.equal(want[0], out[0]) and torch.equal(want[1], out[1])
    _ok()


@pytest.mark.parametrize("fp8", [False, True])
def test_pool_beyond_32_bit_offsets(fp8):
    pages, page, Hkv, d = 140000, 16, 8, 128      # 2.3e9 elements
    free, _ = torch.cuda.mem_get_info()
    if free < 14 << 30:
        pytest.skip("needs 14 GB of free device memory")
    dtype = torch.uint8 if fp8 else torch.bfloat16
    kc = torch.zeros(pages, page, Hkv, d, dtype=dtype, device=DEV)
    vc = torch.zeros_like(kc)
    one = torch.ones((), device=DEV).to(torch.float8_e4m3fn).view(torch.uint8) if fp8 else 1.0
    vc[pages - 1] = one
    table = torch.tensor([[5, pages - 1]], dtype=torch.int32, device=DEV)
    lens = torch.tensor([32], dtype=torch.int32, device=DEV)
    q = torch.ones(1, 16, d, dtype=torch.bfloat16, device=DEV)
    if fp8:
        scale = torch.ones(pages, Hkv, device=DEV)
        o, _ = attn_decode_paged_window_fp8(q, kc, vc, scale, scale, table, lens, 0.1, 16, 16)
    else:
        o, _ = attn_decode_paged_window(q, kc, vc, table, lens, 0.1, 16, 16)
    assert bool((o == 0.5).all())     # half of the weight on each page
    _ok()


def test_refusals():
    c = _make([20, 9], 4, 2, 64, 16, 219, False)
    q, kc, vc, table, lens = (x.to(DEV) for x in (c.q, c.k_cache, c.v_cache, c.block_table, c.seq_lens))
    for window, sinks in ((-1, 0), (4, -1)):
        with pytest.raises(AttnError):
            attn_decode_paged_window(q, kc, vc, table, lens, 0.1, window, sinks)
    with pytest.raises(ValueError):
        attn_decode_paged_window(q.float(), kc, vc, table, lens, 0.1, 4, 1)
    with pytest.raises(ValueError):
        attn_decode_paged_window(q, kc.float(), vc, table, lens, 0.1, 4, 1)
    with pytest.raises(ValueError):
        attn_decode_paged_window(q, kc, vc, table[:1], lens, 0.1, 4, 1)
    with pytest.raises(ValueError):
        attn_decode_paged_window(q, kc, vc, table, lens.long(), 0.1, 4, 1)
    with pytest.raises(ValueError):
        attn_decode_paged_window(q, kc, vc, table.cpu(), lens, 0.1, 4, 1)
    with pytest.raises(ValueError):
        attn_decode_paged_window_fp8(q, kc, vc, None, None, table, lens, 0.1, 4, 1)
    with pytest.raises(AttnError):   # 9 query heads per KV head
        attn_decode_paged_window(torch.zeros(2, 18, 64, dtype=torch.bfloat16, device=DEV), kc, vc,
                                 table, lens, 0.1, 4, 1)
    _ok()


@pytest.mark.parametrize("small", [1e-5, 1e-6, 1e-8])
@pytest.mark.parametrize("first", ["scale 0", "values 0"])
def test_fp8_small_v_scales_behind_a_run_of_zeros(first, small):
    """One sequence of 32 x 1536 tokens: 32 warps (8 CTAs of 4), each with three rounds of 512
    tokens, the first of which adds nothing to the sums (V scales of 0, or of 1 over codes of 0, as a
    page that was never quantised has them).  The scales of the others are small: their weights keep
    their precision, as in the plain decode, which takes 512 tokens at a time."""
    n, page = 32 * 1536, 64
    c = _make([n], 4, 1, 64, page, 220, True)
    c.v_scale.fill_(small)
    for t in range(0, n, page):
        if t % 1536 < 512:
            pg = int(c.block_table[0, t // page])
            c.v_scale[pg] = 0.0 if first == "scale 0" else 1.0
            if first == "values 0":
                c.v_cache[pg] = 0
    ref = _ref(c, 0.125, 0, 0, True)
    q, kc, vc, table, lens = (x.to(DEV) for x in (c.q, c.k_cache, c.v_cache, c.block_table, c.seq_lens))
    plain = attn_decode_paged_fp8(q, kc, vc, c.k_scale.to(DEV), c.v_scale.to(DEV), table, lens, 0.125)
    check_rows(*plain, ref, "plain decode")
    o, lse = _call(c, 0.125, 0, 0, True)
    _ok()
    check_rows(o, lse, ref)


@pytest.mark.parametrize("spread", [16, 1e3, 1e6, 1e11])
@pytest.mark.parametrize("lens,window", [([3000, 40], 0), ([900] * 40, 700)])
def test_fp8_v_scales_far_apart_within_a_warps_run(lens, window, spread):
    """V scales of pages next to one another that differ by up to `spread`, zeros and both signs
    among them: as the plain decode."""
    c = _make(lens, 4, 2, 128, 16, 221, True)
    g = torch.Generator().manual_seed(222)
    f = torch.tensor([0.0, 1.0, -1.0, 1 / spread, -1 / spread, spread ** -0.5])
    c.v_scale.mul_(f[torch.randint(0, len(f), c.v_scale.shape, generator=g)])
    o, lse = _call(c, 0.088, window, 4, True)
    _ok()
    check_rows(o, lse, _ref(c, 0.088, window, 4, True), f"spread {spread}")
