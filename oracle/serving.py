"""CPU oracle for rotary positions and the append to a paged cache -- TEST INFRASTRUCTURE ONLY.

Plain float64 numpy, from the definitions:

* ``rotate``: pair i of a head row (elements (i, i + n) in the half layout,
  (2i, 2i + 1) in the interleaved one, n = len(inv_freq)) at position p turns by
  t = p * inv_freq[i] and is scaled by m; the elements behind the 2n first pass.
* ``append_paged``: token i of a sequence with len_q new tokens and seq_len keys
  in all is key t = seq_len - len_q + i; its rotated K and its V go to row
  t mod page_size of page block_table[b][t div page_size].
* ``window_rows``: a query row at key position p sees key j iff j <= p and (j > p -
  window or j < sinks), window 0 meaning none; softmax attention over the keys
  seen, zero output and -inf LSE where there is none.  ``window_grads``: the
  gradients of sum(dO * O) by the formulas dV = P^T dO, dS = P (dO V^T - D),
  dQ = scale dS K, dK = scale dS^T Q.  The batch, ragged, paged and single-token
  forms below only gather rows for these two.
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


def window_visible(p, n_keys: int, window: int, sinks: int) -> np.ndarray:
    """[len(p), n_keys] bool: key j seen from position p."""
    p = np.asarray(p, dtype=np.int64)[:, None]
    j = np.arange(n_keys, dtype=np.int64)[None, :]
    seen = j <= p
    if window > 0:
        seen &= (j > p - window) | (j < sinks)
    return seen


def window_rows(q, k, v, p, scale, window, sinks):
    """(o [n, d], lse [n], weights [n, m]) of query rows q at positions p over keys k, v [m, d]."""
    q, k, v = f64(q), f64(k), f64(v)
    s = scale * (q @ k.T) if k.shape[0] else np.zeros((q.shape[0], 0))
    seen = window_visible(p, k.shape[0], window, sinks)
    s = np.where(seen, s, -np.inf)
    m = s.max(axis=1, initial=-np.inf)
    base = np.where(np.isneginf(m), 0.0, m)[:, None]
    e = np.exp(s - base)
    total = e.sum(axis=1)
    w = e / np.where(total > 0, total, 1.0)[:, None]
    with np.errstate(divide="ignore"):
        lse = base[:, 0] + np.log(total)
    return w @ v, lse, w


def rows_bound(q, k, v, w, o, scale):
    """How far bf16 output rows may be from o = w v when the kernel rounds weights to bf16
    and the row once on output, element by element.

    The weights the values meet carry a relative error |e_j| <= u = 2^-8 (half a bf16 step)
    plus that of an fp32 exponent: 2^-20 (1 + S), S the row's largest |scale| sum_i |q_i k_ji|
    log2 e, which bounds every score's magnitude and, times a few 2^-24, its rounding errors.
    They are normalised by their own sum, so that the row is sum w_j (1 + e_j) v_j /
    sum w_j (1 + e_j), and differs from o by at most (u + ..) / (1 - u) sum w_j |v_j - o| <=
    (u + ..)(1 + 2u) (sum w_j |v_j| + |o|).  The output's rounding adds u of the value."""
    u = 2.0 ** -8
    s = 1.45 * abs(scale) * (np.abs(q) @ np.abs(k).T).max(axis=1, initial=0.0)[:, None]
    mass = w @ np.abs(v)
    return (u + 2.0 ** -20 * (1.0 + s)) * (1.0 + 2.0 * u) * (mass + np.abs(o)) * (1.0 + u) + \
        u * np.abs(o)


def window_fwd(q, k, v, scale, window, sinks, k_lens=None, bound=False):
    """Dense batch: q [B,Hq,Sq,d], k/v [B,Hkv,Sk,d] -> (o, lse) float64, and with ``bound``
    the tolerance of each element of o (``rows_bound``)."""
    q, k, v = f64(q), f64(k), f64(v)
    B, Hq, Sq, _ = q.shape
    Hkv, Sk = k.shape[1], k.shape[2]
    o, lse, tol = np.zeros_like(q), np.zeros(q.shape[:3]), np.zeros_like(q)
    for b in range(B):
        n = Sk if k_lens is None else int(k_lens[b])
        p = np.arange(Sq) + n - Sq
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            row = (q[b, h], k[b, kv, :n], v[b, kv, :n])
            o[b, h], lse[b, h], w = window_rows(*row, p, scale, window, sinks)
            if bound:
                tol[b, h] = rows_bound(*row, w, o[b, h], scale)
    return (o, lse, tol) if bound else (o, lse)


def window_grads(q, k, v, do, scale, window, sinks, k_lens=None):
    """(dq, dk, dv) of sum(do * window_fwd(q, k, v)), float64."""
    q, k, v, do = f64(q), f64(k), f64(v), f64(do)
    B, Hq, Sq, _ = q.shape
    Hkv, Sk = k.shape[1], k.shape[2]
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for b in range(B):
        n = Sk if k_lens is None else int(k_lens[b])
        p = np.arange(Sq) + n - Sq
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            o, _, w = window_rows(q[b, h], k[b, kv, :n], v[b, kv, :n], p, scale, window, sinks)
            delta = (do[b, h] * o).sum(axis=1, keepdims=True)
            ds = w * (do[b, h] @ v[b, kv, :n].T - delta)
            dv[b, kv, :n] += w.T @ do[b, h]
            dq[b, h] = scale * (ds @ k[b, kv, :n])
            dk[b, kv, :n] += scale * (ds.T @ q[b, h])
    return dq, dk, dv


def gather_pages(cache, block_table, n: int) -> np.ndarray:
    """The first n keys (or values) [n, Hkv, d] of a sequence, by its block-table row."""
    page_size = cache.shape[1]
    return np.stack([cache[int(block_table[t // page_size]), t % page_size] for t in range(n)]) \
        if n else np.zeros((0,) + cache.shape[2:])


def paged_window(q, k_cache, v_cache, block_table, cu_seqlens_q, seq_lens_k, scale, window, sinks,
                 bound=False):
    """Packed queries [total_q, Hq, d], the last ones of their sequences, over paged K/V ->
    (o, lse [Hq, total_q]) (and ``rows_bound`` with ``bound``); rows of no sequence stay NaN.
    cu_seqlens_q None: one query per sequence (decode), lse [total_q, Hq]."""
    q, kc, vc = f64(q), f64(k_cache), f64(v_cache)
    total, Hq, _ = q.shape
    Hkv = kc.shape[2]
    o, lse, tol = np.full(q.shape, np.nan), np.full((Hq, total), np.nan), np.zeros(q.shape)
    for b, n in enumerate(int(x) for x in seq_lens_k):
        a, z = (b, b + 1) if cu_seqlens_q is None else (int(cu_seqlens_q[b]), int(cu_seqlens_q[b + 1]))
        k, v = gather_pages(kc, block_table[b], n), gather_pages(vc, block_table[b], n)
        p = np.arange(z - a) + n - (z - a)
        for h in range(Hq):
            kv = h // (Hq // Hkv)
            row = (q[a:z, h], k[:, kv], v[:, kv])
            o[a:z, h], lse[h, a:z], w = window_rows(*row, p, scale, window, sinks)
            if bound:
                tol[a:z, h] = rows_bound(*row, w, o[a:z, h], scale)
    lse = lse.T if cu_seqlens_q is None else lse
    return (o, lse, tol) if bound else (o, lse)
