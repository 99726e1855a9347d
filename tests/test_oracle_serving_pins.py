"""Pins of the rotary / append oracle (CPU), and of the host-side frequency tables."""
import math

import numpy as np
import pytest
import torch

from exact_softmax_attention_fwd_b200 import rope_frequencies
from oracle import serving as S
from oracle.kv_fp8 import e4m3_to_float


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("n", [1, 3, 8])
def test_rotate_is_complex_multiplication(interleaved, n):
    g = np.random.default_rng(5)
    x = g.standard_normal((2, 7, 20))
    freq = g.uniform(0.0, 3.0, n)
    pos = np.array([0, 1, -4, 1000000, 7, 8, 123456])
    y = S.rotate(x, pos, freq, interleaved, 1.25)
    head = x[..., :2 * n]
    z = head[..., 0::2] + 1j * head[..., 1::2] if interleaved else head[..., :n] + 1j * head[..., n:]
    z = z * 1.25 * np.exp(1j * pos[:, None] * freq)
    want = x.copy()
    if interleaved:
        want[..., 0:2 * n:2], want[..., 1:2 * n:2] = z.real, z.imag
    else:
        want[..., :n], want[..., n:2 * n] = z.real, z.imag
    np.testing.assert_allclose(y, want, rtol=0, atol=1e-9)
    assert np.array_equal(y[..., 2 * n:], x[..., 2 * n:])
    assert np.array_equal(S.rotate(x, np.zeros(7), freq, interleaved), x)


def test_rotated_products_depend_on_the_distance_alone():
    g = np.random.default_rng(6)
    q, k = g.standard_normal((1, 32)), g.standard_normal((1, 32))
    freq, _ = rope_frequencies(32)
    dots = [S.rotate(q, [p + 9], freq)[0] @ S.rotate(k, [p], freq)[0] for p in (0, 5, 31337)]
    np.testing.assert_allclose(dots, dots[0], rtol=0, atol=1e-9)


@pytest.mark.parametrize("interleaved", [False, True])
def test_turning_back_is_the_gradient(interleaved):
    g = np.random.default_rng(7)
    x, w = g.standard_normal((5, 12)), g.standard_normal((5, 12))
    freq = g.uniform(0.0, 2.0, 4)
    pos = np.arange(5) * 3 - 2
    grad = S.rotate(w, -pos, freq, interleaved, 0.7)
    for _ in range(20):
        i, j = g.integers(5), g.integers(12)
        h = np.zeros_like(x)
        h[i, j] = 1e-3
        num = ((S.rotate(x + h, pos, freq, interleaved, 0.7) -
                S.rotate(x - h, pos, freq, interleaved, 0.7)) * w).sum() / 2e-3
        assert abs(num - grad[i, j]) < 1e-9


def test_e4m3_rounding_matches_the_format():
    codes = e4m3_to_float(np.arange(256))
    values = np.unique(codes[np.isfinite(codes)])
    assert np.array_equal(S.to_e4m3(values), values)
    mids = (values[1:] + values[:-1]) / 2
    for off in (-1e-9, 0.0, 1e-9):
        x = torch.tensor(mids + off * np.maximum(1, np.abs(mids)), dtype=torch.float64)
        want = x.float().to(torch.float8_e4m3fn).double().numpy() if off == 0.0 else \
            values[:-1] if off < 0 else values[1:]
        assert np.array_equal(S.to_e4m3(x.numpy()), want)
    assert S.to_e4m3(np.array([1e9, -460.0]))[0] == 448.0
    assert S.to_e4m3(np.array([1e9, -460.0]))[1] == -448.0


def test_append_places_cross_pages_and_skip_idle_rows():
    table = [[4, 2], [7, 5], [1, 0]]
    got = S.append_places(table, [17, 16, 3], [0, 3, 3, 4], 16)
    assert got == [(0, 0, 14, 4, 14), (1, 0, 15, 4, 15), (2, 0, 16, 2, 0), (3, 2, 2, 1, 2)]
    assert S.append_places(table, [17, 0, 1], None, 16) == [(0, 0, 16, 2, 0), (2, 2, 0, 1, 0)]


def test_frequency_tables():
    f, m = rope_frequencies(128)
    i = np.arange(64)
    assert m == 1.0 and f.dtype == torch.float64
    np.testing.assert_allclose(f.numpy(), 10000.0 ** (-i / 64), rtol=1e-13)
    lin, m = rope_frequencies(128, scaling="linear", factor=4.0)
    np.testing.assert_allclose(lin.numpy(), f.numpy() / 4, rtol=1e-13)
    st, m = rope_frequencies(128, scaling="base", factor=8.0)
    assert m == 1.0
    np.testing.assert_allclose([st[0], st[-1]], [f[0], f[-1] / 8.0], rtol=1e-12)
    ramp, m = rope_frequencies(128, scaling="ramp", factor=16.0, original_length=4096)
    assert m == pytest.approx(0.1 * math.log(16.0) + 1.0)
    turns = 4096 * f.numpy() / (2 * math.pi)
    assert np.allclose(ramp.numpy()[turns >= 32], f.numpy()[turns >= 32], rtol=1e-13)
    assert np.allclose(ramp.numpy()[turns <= 1], f.numpy()[turns <= 1] / 16.0, rtol=1e-13)
    mid = (turns > 1) & (turns < 32)
    share = (turns[mid] - 1) / 31
    np.testing.assert_allclose(ramp.numpy()[mid], f.numpy()[mid] * (share + (1 - share) / 16.0),
                               rtol=1e-12)


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=15), dict(rotary_dim=0), dict(rotary_dim=16, base=1.0),
    dict(rotary_dim=16, base=float("nan")), dict(rotary_dim=16, scaling="other"),
    dict(rotary_dim=16, factor=0.5), dict(rotary_dim=2, scaling="base", factor=2.0),
    dict(rotary_dim=16, scaling="ramp", slow_turns=3.0, fast_turns=3.0)])
def test_frequency_refusals(kw):
    with pytest.raises(ValueError):
        rope_frequencies(**kw)


# ------------------------------------------------------------- window with first tokens

def _dense(B=2, Hq=4, Hkv=2, Sq=37, Sk=50, d=16, seed=3):
    g = np.random.default_rng(seed)
    # bf16 values, so that the C oracle reads the same numbers
    as_bf16 = lambda x: torch.tensor(x, dtype=torch.float32).to(torch.bfloat16)  # noqa: E731
    return (as_bf16(g.standard_normal((B, Hq, Sq, d))), as_bf16(g.standard_normal((B, Hkv, Sk, d))),
            as_bf16(g.standard_normal((B, Hkv, Sk, d))))


def test_window_rule_by_enumeration():
    seen = S.window_visible([-1, 0, 4, 9], 12, 3, 2)
    assert [np.flatnonzero(r).tolist() for r in seen] == \
        [[], [0], [0, 1, 2, 3, 4], [0, 1, 7, 8, 9]]
    assert S.window_visible([5], 12, 0, 0)[0].tolist() == [True] * 6 + [False] * 6
    assert S.window_visible([9], 12, 1, 0)[0].nonzero()[0].tolist() == [9]


@pytest.mark.parametrize("window", [0, 1, 7, 64])
def test_without_first_tokens_it_is_the_window_oracle(window):
    import oracle
    q, k, v = _dense()
    lens = torch.tensor([50, 20], dtype=torch.int32)
    o, lse = S.window_fwd(q, k, v, 0.3, window, 0, lens)
    ro, rl = oracle.attn_fwd(q, k, v, True, 0.3, k_lens=lens, window=window)
    np.testing.assert_allclose(o, ro, rtol=0, atol=1e-12)
    np.testing.assert_allclose(lse, rl, rtol=0, atol=1e-12)


def test_enough_first_tokens_are_plain_causal_attention():
    import oracle
    q, k, v = _dense()
    o, lse = S.window_fwd(q, k, v, 0.3, 4, 50)
    ro, rl = oracle.attn_fwd(q, k, v, True, 0.3)
    np.testing.assert_allclose(o, ro, rtol=0, atol=1e-12)
    np.testing.assert_allclose(lse, rl, rtol=0, atol=1e-12)


def test_window_gradients_match_differences():
    q, k, v = (S.f64(x) for x in _dense(1, 2, 1, 9, 12, 4))
    g = np.random.default_rng(4)
    do = g.standard_normal(q.shape)
    lens = [11]
    grads = S.window_grads(q, k, v, do, 0.5, 3, 2, lens)
    for which, (x, grad) in enumerate(zip((q, k, v), grads)):
        for _ in range(25):
            at = tuple(int(g.integers(n)) for n in x.shape)
            args = [q, k, v]
            vals = []
            for h in (1e-5, -1e-5):
                y = x.copy()
                y[at] += h
                args[which] = y
                vals.append((S.window_fwd(*args, 0.5, 3, 2, lens)[0] * do).sum())
            assert abs((vals[0] - vals[1]) / 2e-5 - grad[at]) < 1e-7


def test_paged_and_single_token_forms_gather_the_dense_one():
    q, k, v = (S.f64(x) for x in _dense(1, 4, 2, 5, 40, 8))
    table = [[2, 0, 1, 3, 4]]
    kc, vc = np.zeros((5, 8, 2, 8)), np.zeros((5, 8, 2, 8))
    for t in range(40):
        kc[table[0][t // 8], t % 8], vc[table[0][t // 8], t % 8] = k[0, :, t], v[0, :, t]
    o, lse = S.window_fwd(q, k, v, 0.4, 6, 3)
    po, pl = S.paged_window(q[0].transpose(1, 0, 2), kc, vc, table, [0, 5], [40], 0.4, 6, 3)
    np.testing.assert_allclose(po.transpose(1, 0, 2), o[0], atol=1e-13)
    np.testing.assert_allclose(pl, lse[0], atol=1e-13)
    do, dl = S.paged_window(q[0, :, -1][None], kc, vc, table, None, [40], 0.4, 6, 3)
    np.testing.assert_allclose(do[0], o[0, :, -1], atol=1e-13)
    np.testing.assert_allclose(dl[0], lse[0, :, -1], atol=1e-13)
