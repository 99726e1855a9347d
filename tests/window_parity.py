"""The bar of the window-with-first-tokens tests: every element of O within the oracle's own
bound (``oracle.serving.rows_bound``: the weights' and the output's bf16 rounding), the relative
RMS and the LSE within tests/parity.py's, no NaN, and the same rows empty (zeros, -inf).

tests/parity.py's largest absolute error (1e-2) is meant for rows that average many keys: a row
that sees a single value of 4 is off by 1.6e-2 when that value is rounded to bf16."""
import numpy as np

from parity import LSE_MAX_ABS, O_REL_RMS, to_f64


def check_rows(o, lse, ref, what=""):
    ro, rl, tol = ref
    o, lse = to_f64(o), to_f64(lse)
    assert o.shape == ro.shape and lse.shape == rl.shape, what
    assert np.isfinite(o).all() and not np.isnan(lse).any(), f"{what}: not finite"
    off = np.abs(o - ro) - tol
    assert (off <= 0).all(), f"{what}: {int((off > 0).sum())} of {off.size} elements off, by up to {off.max():.3e}"
    empty = np.isneginf(rl)
    assert np.array_equal(empty, np.isneginf(lse)), f"{what}: other rows are empty"
    assert not np.abs(lse[~empty] - rl[~empty]).max(initial=0.0) > LSE_MAX_ABS, f"{what}: LSE"
    norm = np.linalg.norm(ro)
    assert np.linalg.norm(o - ro) <= O_REL_RMS * norm, f"{what}: rel RMS"
