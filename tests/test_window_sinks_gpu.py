"""GPU parity of attention with a sliding window and visible first tokens (dense forward and
backward, and over a paged cache) against the float64 oracle, at the bar of tests/parity.py."""
import math

import numpy as np
import pytest
import torch

from exact_softmax_attention_fwd_b200 import (AttnError, attn_bwd_window, attn_bwd_window_sinks,
                                             attn_bwd_window_sinks_workspace_size, attn_fwd_masked,
                                             attn_fwd_paged_window, attn_fwd_window,
                                             attn_fwd_window_sinks, attn_get_device_error)
from exact_softmax_attention_fwd_b200 import _binding as B
from exact_softmax_attention_fwd_b200 import workloads as W
from oracle import serving as S

from parity import check_grad
from window_parity import check_rows

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _ok():
    st, flags = attn_get_device_error()
    assert st == 0, f"device error flags {flags:#x}"


def _dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


CASES = [
    # B, Hq, Hkv, Sq, Sk, d, window, sinks, k_lens
    (1, 1, 1, 1, 1, 64, 1, 1, None),
    (1, 2, 1, 1, 700, 128, 100, 4, None),            # one query row
    (1, 4, 2, 700, 700, 128, 100, 4, None),          # head pairs, a gap of several tiles
    (1, 3, 1, 700, 700, 128, 100, 4, None),          # 256-row units
    (2, 3, 3, 513, 513, 64, 1, 1, None),
    (1, 2, 1, 900, 900, 64, 128, 128, None),         # first tokens of a whole tile
    (1, 3, 1, 900, 900, 64, 129, 129, None),         # and one more
    (1, 4, 2, 800, 800, 128, 37, 300, None),         # three tiles of first tokens
    (1, 2, 1, 640, 640, 128, 64, 1000, None),        # first tokens are all tokens
    (1, 2, 1, 640, 640, 128, 5000, 3, None),         # the window is all tokens
    (1, 4, 1, 640, 640, 128, 0, 7, None),            # no window
    (1, 6, 3, 300, 1100, 128, 130, 5, None),         # queries at the end of longer keys
    (3, 4, 2, 600, 600, 128, 50, 9, [600, 333, 1]),  # rows with no key
    (2, 3, 1, 400, 400, 64, 20, 200, [0, 150]),      # an empty sequence; fewer keys than first tokens
    (2, 2, 2, 1100, 300, 64, 40, 6, None),           # more queries than keys
]


def _inputs(case, seed=191):
    B_, Hq, Hkv, Sq, Sk, d, window, sinks, lens = case
    q, k, v = W.prefill_inputs(B_, Hq, Hkv, Sq, Sk, d, seed)
    lens = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    return q, k, v, lens, 1 / math.sqrt(d)


@pytest.mark.parametrize("case", CASES, ids=str)
def test_forward(case):
    q, k, v, lens, scale = _inputs(case)
    window, sinks = case[6:8]
    o, lse = attn_fwd_window_sinks(*_dev(q, k, v), scale, window, sinks, k_lens=_dev(lens)[0])
    torch.cuda.synchronize()
    _ok()
    check_rows(o, lse, S.window_fwd(q, k, v, scale, window, sinks, lens, bound=True), str(case))


@pytest.mark.parametrize("case", CASES, ids=str)
def test_backward(case):
    q, k, v, lens, scale = _inputs(case)
    window, sinks = case[6:8]
    do = W.grad_output(case[0], case[1], case[3], case[5], 192)
    qd, kd, vd, ld, dod = _dev(q, k, v, lens, do)
    o, lse = attn_fwd_window_sinks(qd, kd, vd, scale, window, sinks, k_lens=ld)
    out = [torch.full_like(x, float("nan")) for x in (qd, kd, vd)]
    got = attn_bwd_window_sinks(qd, kd, vd, o, lse, dod, scale, window, sinks, k_lens=ld,
                                dq=out[0], dk=out[1], dv=out[2])
    torch.cuda.synchronize()
    _ok()
    for name, g, r in zip(("dq", "dk", "dv"), got, S.window_grads(q, k, v, do, scale, window, sinks,
                                                                 lens)):
        check_grad(g, r, what=f"{name} {case}")
    # deterministic, and the partial sums do not depend on what the workspace held
    need = attn_bwd_window_sinks_workspace_size(*case[:6], window, sinks)
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device=DEV)
    again = attn_bwd_window_sinks(qd, kd, vd, o, lse, dod, scale, window, sinks, k_lens=ld,
                                  workspace=ws)
    assert all(torch.equal(a, b) for a, b in zip(got, again))


def test_gradients_by_differences():
    """dL/dx of L = sum(dO * O) along random directions: the directional derivative by
    central differences of the float64 oracle equals the kernel's gradient product within
    the gradient's own tolerance (relative 5e-3 in norm, so that times the direction's)."""
    case = (1, 4, 2, 300, 300, 64, 40, 5, None)
    q, k, v, _, scale = _inputs(case, 17)
    do = W.grad_output(1, 4, 300, 64, 18)
    qd, kd, vd, dod = _dev(q, k, v, do)
    o, lse = attn_fwd_window_sinks(qd, kd, vd, scale, 40, 5)
    grads = attn_bwd_window_sinks(qd, kd, vd, o, lse, dod, scale, 40, 5)
    g = np.random.default_rng(2)
    base = [S.f64(x) for x in (q, k, v)]
    for which, grad in enumerate(grads):
        grad = S.f64(grad)
        for _ in range(3):
            u = g.standard_normal(grad.shape)
            u /= np.linalg.norm(u)
            vals = []
            for h in (1e-4, -1e-4):
                args = list(base)
                args[which] = args[which] + h * u
                vals.append((S.window_fwd(*args, scale, 40, 5)[0] * S.f64(do)).sum())
            assert abs((vals[0] - vals[1]) / 2e-4 - (grad * u).sum()) <= 5e-3 * np.linalg.norm(grad)


def test_without_first_tokens_the_bits_are_the_window_calls():
    q, k, v = _dev(*W.prefill_inputs(2, 8, 2, 1111, 1111, 128, 193))
    o, lse = attn_fwd_window(q, k, v, 0.088, window=200)
    o2, lse2 = attn_fwd_window_sinks(q, k, v, 0.088, 200, 0)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    do = torch.randn_like(o)
    for a, b in zip(attn_bwd_window(q, k, v, o, lse, do, 0.088, window=200),
                    attn_bwd_window_sinks(q, k, v, o, lse, do, 0.088, 200, 0)):
        assert torch.equal(a, b)
    oc, lc = attn_fwd_masked(q, k, v, True, 0.088)
    o3, l3 = attn_fwd_window_sinks(q, k, v, 0.088, 0, 5)
    assert torch.equal(oc, o3) and torch.equal(lc, l3)


def test_no_keys_and_counts_beyond_an_int():
    q = W.randn_bf16((2, 4, 70, 64), 202).to(DEV)
    none = torch.empty(2, 2, 0, 64, dtype=torch.bfloat16, device=DEV)
    o, lse = attn_fwd_window_sinks(q, none, none, 0.1, 8, 2)
    assert bool((o == 0).all()) and bool(torch.isneginf(lse).all())
    dq, dk, dv = attn_bwd_window_sinks(q, none, none, o, lse, q, 0.1, 8, 2)
    assert bool((dq == 0).all()) and dk.shape == none.shape == dv.shape
    _, k, v = _dev(*W.prefill_inputs(2, 4, 2, 70, 300, 64, 203))
    for far, near in (((2 ** 40 + 3, 2 ** 33), (300, 0)), ((8, 2 ** 32 + 1), (8, 300))):
        a = attn_fwd_window_sinks(q, k, v, 0.1, *far)
        b = attn_fwd_window_sinks(q, k, v, 0.1, *near)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        for x, y in zip(attn_bwd_window_sinks(q, k, v, *a, q, 0.1, *far),
                        attn_bwd_window_sinks(q, k, v, *b, q, 0.1, *near)):
            assert torch.equal(x, y)
    _ok()


@pytest.mark.parametrize("scale", [-0.2, 0.0, 3.0])
def test_odd_scales(scale):
    q, k, v = W.prefill_inputs(1, 2, 1, 400, 400, 64, 194)
    o, lse = attn_fwd_window_sinks(*_dev(q, k, v), scale, 30, 4)
    check_rows(o, lse, S.window_fwd(q, k, v, scale, 30, 4, bound=True), f"scale {scale}")


def test_weights_on_first_tokens_far_above_the_window():
    """The maximum moves between the first tokens' tile and the window's: both orders."""
    for sign in (1.0, -1.0):
        q, k, v = W.prefill_inputs(1, 2, 1, 1000, 1000, 128, 195)
        k[:, :, :4] = sign * 3.0 * q[:, :1, 500:504]
        o, lse = attn_fwd_window_sinks(*_dev(q, k, v), 0.088, 100, 4)
        check_rows(o, lse, S.window_fwd(q, k, v, 0.088, 100, 4, bound=True), f"sign {sign}")


PAGED = [
    # new tokens, lengths with them, Hq, Hkv, d, page, window, sinks
    ([1], [1], 2, 1, 64, 16, 5, 2),
    ([300, 0, 1, 77], [300, 50, 900, 500], 4, 2, 128, 16, 100, 4),
    ([130, 600], [1400, 600], 3, 1, 64, 64, 37, 140),
    ([257, 5], [257, 129], 4, 4, 128, 128, 64, 1),
    ([20, 20], [20, 400], 2, 2, 64, 32, 0, 3),             # no window
    ([1, 33, 200, 64, 7], [700, 33, 450, 64, 2000], 8, 1, 128, 16, 90, 4),   # 8 heads to a tile
    ([1, 9, 140], [40, 700, 300], 16, 1, 64, 64, 50, 33),  # 16
    ([31, 65], [400, 65], 12, 2, 128, 32, 64, 4),          # 6: tiles of one head
    ([5, 9], [3, 9], 2, 1, 64, 16, 4, 2),                  # more queries than keys: empty rows
    ([4, 2, 140], [0, 2, 1], 8, 2, 128, 16, 4, 2),         # no keys, one key
]


@pytest.mark.parametrize("case", PAGED, ids=str)
def test_paged(case):
    new, total, Hq, Hkv, d, page, window, sinks = case
    q, cu, c = W.paged_prefill_inputs(new, total, Hq, Hkv, d, page, 196)
    # slots behind the sequences' ends were never written
    kc, vc = c.k_cache.clone(), c.v_cache.clone()
    for b, n in enumerate(total):
        if n % page:
            last = int(c.block_table[b, n // page])
            kc[last, n % page:], vc[last, n % page:] = float("nan"), float("inf")
    scale = 1 / math.sqrt(d)
    args = _dev(q, kc, vc, c.block_table, cu, c.seq_lens)
    o, lse = attn_fwd_paged_window(*args, max(new), scale, window, sinks)
    torch.cuda.synchronize()
    _ok()
    check_rows(o, lse, S.paged_window(q, c.k_cache, c.v_cache, c.block_table, cu, c.seq_lens, scale,
                                      window, sinks, bound=True), str(case))


def test_paged_rows_behind_the_last_sequence_stay_and_bad_input_is_flagged():
    new, total = [40, 9], [200, 30]
    q, cu, c = W.paged_prefill_inputs(new, total, 2, 1, 64, 16, 197)
    q = torch.cat([q, q[:7]])
    args = _dev(q, c.k_cache, c.v_cache, c.block_table, cu, c.seq_lens)
    out = torch.full((56, 2, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((2, 56), 9.0, device=DEV)
    attn_fwd_paged_window(*args, 40, 0.125, 50, 2, out=out, lse=lse)
    assert bool((out[49:] == 9.0).all()) and bool((lse[:, 49:] == 9.0).all())
    _ok()
    bad = c.seq_lens.clone()
    bad[1] = 10 ** 6
    out.fill_(9.0)
    attn_fwd_paged_window(*args[:5], bad.to(DEV), 40, 0.125, 50, 2, out=out)
    assert attn_get_device_error() == (B.ATTN_ERR_DEVICE, B.DEVERR_BAD_LENGTH)
    assert bool((out[40:] == 9.0).all())
    table = c.block_table.clone()
    table[0, 12] = c.num_pages
    attn_fwd_paged_window(*args[:3], table.to(DEV), *args[4:], 40, 0.125, 50, 2)
    assert attn_get_device_error() == (B.ATTN_ERR_DEVICE, B.DEVERR_BAD_PAGE)
    # a page between the first tokens' tile and the windows is not read, whatever its id
    q, cu, c = W.paged_prefill_inputs([10], [1000], 2, 1, 64, 16, 198)
    args = _dev(q, c.k_cache, c.v_cache, c.block_table, cu, c.seq_lens)
    o, _ = attn_fwd_paged_window(*args, 10, 0.125, 50, 2)
    table = c.block_table.clone()
    table[0, 8:50] = -5
    o2, _ = attn_fwd_paged_window(*args[:3], table.to(DEV), *args[4:], 10, 0.125, 50, 2)
    _ok()
    assert torch.equal(o, o2)


def test_refusals():
    q, k, v = _dev(*W.prefill_inputs(1, 4, 2, 64, 64, 64, 199))
    for window, sinks in ((-1, 0), (0, -1), (5, -2)):
        with pytest.raises(AttnError):
            attn_fwd_window_sinks(q, k, v, 0.1, window, sinks)
    with pytest.raises(ValueError):
        attn_fwd_window_sinks(q.transpose(1, 2), k, v, 0.1, 4, 1)
    with pytest.raises(ValueError):
        attn_fwd_window_sinks(q, k.float(), v, 0.1, 4, 1)
    with pytest.raises(ValueError):
        attn_fwd_window_sinks(q, k, v[:, :1], 0.1, 4, 1)
    with pytest.raises(ValueError):
        attn_fwd_window_sinks(q, k, v, 0.1, 4, 1, out=torch.empty_like(k))
    with pytest.raises(ValueError):
        attn_fwd_window_sinks(q.cpu(), k, v, 0.1, 4, 1)
    with pytest.raises(AttnError):
        attn_fwd_window_sinks(q, k, v, float("nan"), 4, 1)
    o, lse = attn_fwd_window_sinks(q, k, v, 0.1, 4, 1)
    with pytest.raises(AttnError):
        attn_bwd_window_sinks(q, k, v, o, lse, o, 0.1, 4, 1,
                              workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError):
        attn_bwd_window_sinks(q, k, v, o, lse[:, :2], o, 0.1, 4, 1)
    _ok()


def test_other_stream_and_two_graphs():
    q, k, v = _dev(*W.prefill_inputs(1, 4, 2, 900, 900, 64, 200))
    do = W.grad_output(1, 4, 900, 64, 201).to(DEV)

    def step(stream=None):
        o, lse = attn_fwd_window_sinks(q, k, v, 0.125, 60, 3, stream=stream)
        return (o, lse) + attn_bwd_window_sinks(q, k, v, o, lse, do, 0.125, 60, 3, stream=stream)

    want = step()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = step(side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    q.mul_(0.5)
    want = step()
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(a, b) for a, b in zip(want, out))
    _ok()


# new tokens and keys of two sequences, Hq, Hkv, d, page, window, first tokens: gaps of many tiles
# and of less than one, the window's start and the first tokens' end inside a tile and a page,
# one and several blocks of query rows, heads of a group in one tile (2, 4, 16) and not (1, 3)
HIDDEN = [
    ([10, 3], [1000, 700], 2, 1, 64, 16, 50, 4),
    ([10, 3], [1000, 700], 4, 1, 128, 32, 50, 4),
    ([10, 1], [1000, 700], 3, 1, 64, 64, 200, 0),
    ([10, 40], [290, 300], 16, 1, 64, 16, 60, 4),      # the window starts in the tile after the first
    ([5, 6], [120, 125], 1, 1, 128, 16, 20, 4),        # everything in one tile
    ([5, 6], [120, 125], 4, 2, 128, 16, 20, 33),
    ([300, 8], [900, 500], 2, 2, 128, 16, 100, 130),   # several blocks, two tiles of first tokens
    ([300, 8], [900, 500], 8, 2, 64, 128, 100, 40),
]


@pytest.mark.parametrize("what", ["bad ids", "nan"])
@pytest.mark.parametrize("case", HIDDEN, ids=str)
def test_paged_pages_without_a_visible_key_are_not_read(case, what):
    """Every page that lies wholly between the first tokens and the windows has an id outside the
    pool, or holds NaN: the result keeps its bits, and nothing is flagged."""
    new, total, Hq, Hkv, d, page, window, sinks = case
    q, cu, c = W.paged_prefill_inputs(new, total, Hq, Hkv, d, page, 203)
    args = _dev(q, c.k_cache, c.v_cache, c.block_table, cu, c.seq_lens)
    scale = 1 / math.sqrt(d)
    o, lse = attn_fwd_paged_window(*args, max(new), scale, window, sinks)
    _ok()
    check_rows(o, lse, S.paged_window(q, c.k_cache, c.v_cache, c.block_table, cu, c.seq_lens, scale,
                                      window, sinks, bound=True), str(case))
    kc, vc, table = c.k_cache.clone(), c.v_cache.clone(), c.block_table.clone()
    n_hidden = 0
    for b, (n, t) in enumerate(zip(new, total)):
        for pg in range(-(-sinks // page), max(0, t - n - window + 1) // page):
            n_hidden += 1
            if what == "nan":
                kc[int(table[b, pg])] = vc[int(table[b, pg])] = float("nan")
            else:
                table[b, pg] = c.num_pages + 7 if pg % 2 else -1
    assert n_hidden > 0
    o2, lse2 = attn_fwd_paged_window(*_dev(q, kc, vc, table, cu, c.seq_lens), max(new), scale,
                                     window, sinks)
    _ok()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("d,window,sinks", [(128, 1024, 4), (64, 300, 200)])
def test_long_rows_against_the_oracle(d, window, sinks):
    """5000 rows: windows of several tiles, and first tokens whose gradients many query tiles
    share out among units."""
    q, k, v = W.prefill_inputs(1, 2, 1, 5000, 5000, d, 204)
    do = W.grad_output(1, 2, 5000, d, 205)
    scale = 1 / math.sqrt(d)
    assert attn_bwd_window_sinks_workspace_size(1, 2, 1, 5000, 5000, d, window, sinks) > \
        attn_bwd_window_sinks_workspace_size(1, 2, 1, 5000, 5000, d, window, 0)
    qd, kd, vd, dod = _dev(q, k, v, do)
    o, lse = attn_fwd_window_sinks(qd, kd, vd, scale, window, sinks)
    got = attn_bwd_window_sinks(qd, kd, vd, o, lse, dod, scale, window, sinks)
    _ok()
    check_rows(o, lse, S.window_fwd(q, k, v, scale, window, sinks, bound=True))
    for name, g, r in zip(("dq", "dk", "dv"), got, S.window_grads(q, k, v, do, scale, window, sinks)):
        check_grad(g, r, what=name)
