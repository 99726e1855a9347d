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
