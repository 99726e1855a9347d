"""CPU oracle for rotary positions and the append to a paged cache -- TEST INFRASTRUCTURE ONLY.

Plain float64 numpy, from the definitions:

* ``rotate``: pair i of a head row (elements (i, i + n) in the half layout,
  (2i, 2i + 1) in the interleaved one, n = len(inv_freq)) at position p turns by
  t = p * inv_freq[i] and is scaled by m; the elements behind the 2n first pass.
* ``append_paged``: token i of a sequence with len_q new tokens and seq_len keys
  in all is key t = seq_len - len_q + i; its rotated K and its V go to row
  t mod page_size of page block_table[b][t div page_size].
* ``to_e4m3``: the nearest E4M3 value (ties to even), saturating at 448.

Pinned in ``tests/test_oracle_serving_pins.py``.
"""
from __future__ import annotations

import numpy as np


def f64(x) -> np.ndarray:
    """Torch tensor (any float dtype) or array -> float64 numpy."""
    if hasattr(x, "detach"):
        x = x.detach().cpu().double().numpy()
    return np.asarray(x, dtype=np.float64)


def rotate(x, positions, inv_freq, interleaved: bool = False, mscale: float = 1.0) -> np.ndarray:
    """x [..., S, d] turned row by row at positions [S] (or [..., S], broadcast)."""
    x = f64(x)
    freq = f64(inv_freq)
    n = freq.shape[0]
    t = f64(positions)[..., None] * freq
    c, s = np.cos(t) * mscale, np.sin(t) * mscale
    out = x.copy()
    ia, ib = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else \
        (slice(0, n), slice(n, 2 * n))
    a, b = x[..., ia], x[..., ib]
    out[..., ia] = a * c - b * s
    out[..., ib] = a * s + b * c
    return out


def pair_weight(x, n: int, interleaved: bool = False) -> np.ndarray:
    """|a| + |b| of the pair that each element belongs to (0 behind the rotated ones): what
    the rounding errors of its rotation scale with."""
    x = np.abs(f64(x))
    w = np.zeros_like(x)
    ia, ib = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else \
        (slice(0, n), slice(n, 2 * n))
    w[..., ia] = w[..., ib] = x[..., ia] + x[..., ib]
    return w


def to_e4m3(x) -> np.ndarray:
    """Nearest E4M3 value of each element of x, as float64."""
    x = np.clip(f64(x), -448.0, 448.0)
    e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -20)))
    step = np.exp2(np.maximum(e, -6.0) - 3.0)
    return np.clip(np.rint(x / step) * step, -448.0, 448.0)


def append_places(block_table, seq_lens, cu_seqlens, page_size: int):
    """[(token, sequence, key number, page, row)] of every new token; cu_seqlens None: one
    token per sequence, none for a sequence of length 0."""
    places = []
    lens = [int(n) for n in seq_lens]
    for b, n in enumerate(lens):
        if cu_seqlens is None:
            tokens = [b] if n > 0 else []
        else:
            tokens = list(range(int(cu_seqlens[b]), int(cu_seqlens[b + 1])))
        for i, tok in enumerate(tokens):
            key = n - len(tokens) + i
            places.append((tok, b, key, int(block_table[b][key // page_size]), key % page_size))
    return places


def append_paged(q, k, v, k_cache, v_cache, block_table, seq_lens, cu_seqlens, inv_freq,
                 interleaved=False, mscale=1.0, positions=None, k_scale=None, v_scale=None):
    """(q_out or None, k_cache, v_cache, places) in float64: the caches (bf16 values, or the
    values of E4M3 codes when scales are given) with the new tokens written.  Rows of q_out
    that no sequence owns stay NaN."""
    kc, vc = f64(k_cache).copy(), f64(v_cache).copy()
    page_size = kc.shape[1]
    places = append_places(block_table, seq_lens, cu_seqlens, page_size)
    q_out = None if q is None else np.full(tuple(q.shape), np.nan)
    for tok, _, key, page, row in places:
        pos = np.array([key if positions is None else int(positions[tok])])

        def turn(x):
            x = f64(x[tok])[:, None, :]
            if inv_freq is None:
                return x[:, 0]
            return rotate(x, pos, inv_freq, interleaved, mscale)[:, 0]

        if q is not None:
            q_out[tok] = turn(q)
        new_k, new_v = turn(k), f64(v[tok])
        if k_scale is not None:
            ks, vs = f64(k_scale[page])[:, None], f64(v_scale[page])[:, None]
            new_k = to_e4m3(np.where(ks != 0, new_k / np.where(ks != 0, ks, 1.0), 0.0))
            new_v = to_e4m3(np.where(vs != 0, new_v / np.where(vs != 0, vs, 1.0), 0.0))
        kc[page, row], vc[page, row] = new_k, new_v
    return q_out, kc, vc, places
