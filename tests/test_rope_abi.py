"""Host-side checks of the rotary and append entry points (CPU; nothing is launched)."""
import ctypes

import pytest
import torch

from exact_softmax_attention_fwd_b200 import _binding as B
from exact_softmax_attention_fwd_b200 import build as build_mod

FAKE = 0x100000  # 16-byte aligned, never dereferenced: every call below fails validation


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load_library()


def _rope(lib, fn="attn_rope", q=FAKE, k=FAKE, qo=FAKE, ko=FAKE, freq=FAKE, pos=None, ps=0, B_=2,
          Hq=4, Hkv=2, S=5, d=128, rot=128, inter=0, m=1.0, strides=None):
    s = None if strides is None else (ctypes.c_longlong * 12)(*strides)
    return getattr(lib, fn)(q, k, qo, ko, freq, pos, ps, B_, Hq, Hkv, S, d, rot, inter, m, s, None)


def _strides(B_=2, Hq=4, Hkv=2, S=5, d=128):
    one = lambda h: [h * S * d, S * d, d]  # noqa: E731
    return one(Hq) + one(Hkv) + one(Hq) + one(Hkv)


def _with(i, value):
    s = _strides()
    s[i] = value
    return s


@pytest.mark.parametrize("fn", ["attn_rope", "attn_rope_bwd"])
@pytest.mark.parametrize("kw,status", [
    (dict(q=None), B.ATTN_ERR_INVALID_ARG),
    (dict(qo=None), B.ATTN_ERR_INVALID_ARG),
    (dict(k=None), B.ATTN_ERR_INVALID_ARG),
    (dict(ko=None), B.ATTN_ERR_INVALID_ARG),
    (dict(freq=None), B.ATTN_ERR_INVALID_ARG),
    (dict(B_=0), B.ATTN_ERR_INVALID_ARG),
    (dict(Hq=0), B.ATTN_ERR_INVALID_ARG),
    (dict(Hkv=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(S=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(B_=1 << 12, S=1 << 20), B.ATTN_ERR_INVALID_ARG),
    (dict(inter=2), B.ATTN_ERR_INVALID_ARG),
    (dict(m=float("nan")), B.ATTN_ERR_INVALID_ARG),
    (dict(pos=FAKE, ps=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(d=96, rot=96), B.ATTN_ERR_UNSUPPORTED),
    (dict(rot=0), B.ATTN_ERR_UNSUPPORTED),
    (dict(rot=24), B.ATTN_ERR_UNSUPPORTED),
    (dict(rot=144), B.ATTN_ERR_UNSUPPORTED),
    (dict(q=FAKE + 8), B.ATTN_ERR_ALIGNMENT),
    (dict(ko=FAKE + 2), B.ATTN_ERR_ALIGNMENT),
    (dict(freq=FAKE + 4), B.ATTN_ERR_ALIGNMENT),
    (dict(pos=FAKE + 2), B.ATTN_ERR_ALIGNMENT),
    (dict(strides=_with(0, -8)), B.ATTN_ERR_INVALID_ARG),
    (dict(strides=_with(2, 1 << 45)), B.ATTN_ERR_INVALID_ARG),
    (dict(strides=_with(1, 132)), B.ATTN_ERR_ALIGNMENT),
    (dict(strides=_with(8, 0)), B.ATTN_ERR_INVALID_ARG),      # output rows on one another
    (dict(strides=_with(8, 64)), B.ATTN_ERR_INVALID_ARG),
    (dict(strides=_with(9, 128)), B.ATTN_ERR_INVALID_ARG),
])
def test_rope_validation(lib, fn, kw, status):
    assert _rope(lib, fn, **kw) == status


@pytest.mark.parametrize("fn", ["attn_rope", "attn_rope_bwd"])
@pytest.mark.parametrize("side", [0, 1])
def test_rope_in_place_with_other_strides_is_refused(lib, fn, side):
    """Q (or K) turned into its own memory in another order of heads and rows."""
    S, d, H = 5, 128, (4, 2)[side]
    s = _strides()
    s[6 + 3 * side:9 + 3 * side] = [H * S * d, d, H * d]
    kw = dict(q=FAKE, qo=FAKE, k=2 * FAKE, ko=3 * FAKE) if side == 0 else \
        dict(q=FAKE, qo=3 * FAKE, k=2 * FAKE, ko=2 * FAKE)
    assert _rope(lib, fn, strides=s, **kw) == B.ATTN_ERR_INVALID_ARG


def test_append_in_place_of_strided_queries_is_refused(lib):
    for s in ([1024, 128, 256, 128, 256, 128], [512, 256, 256, 128, 256, 128]):
        assert _append(lib, q=FAKE, qo=FAKE, strides=s) == B.ATTN_ERR_INVALID_ARG


def test_rope_of_no_rows_launches_nothing(lib):
    assert _rope(lib, S=0, q=None, k=None, qo=None, ko=None) == B.ATTN_OK


def _append(lib, fp8=False, q=FAKE, k=FAKE, v=FAKE, qo=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE,
            tbl=FAKE, cu=FAKE, lens=FAKE, pos=None, freq=FAKE, ps=16, B_=2, Hq=4, Hkv=2, total=9,
            maxp=4, npages=8, d=128, rot=64, inter=0, m=1.0, strides=None):
    s = None if strides is None else (ctypes.c_longlong * 6)(*strides)
    scales = (ks, vs) if fp8 else ()
    fn = lib.attn_append_paged_fp8 if fp8 else lib.attn_append_paged
    return fn(q, k, v, qo, kc, vc, *scales, tbl, cu, lens, pos, freq, ps, B_, Hq, Hkv, total, maxp,
              npages, d, rot, inter, m, s, None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(k=None), B.ATTN_ERR_INVALID_ARG),
    (dict(v=None), B.ATTN_ERR_INVALID_ARG),
    (dict(q=None), B.ATTN_ERR_INVALID_ARG),
    (dict(Hq=0), B.ATTN_ERR_INVALID_ARG),
    (dict(qo=None), B.ATTN_ERR_INVALID_ARG),
    (dict(kc=None), B.ATTN_ERR_INVALID_ARG),
    (dict(tbl=None), B.ATTN_ERR_INVALID_ARG),
    (dict(lens=None), B.ATTN_ERR_INVALID_ARG),
    (dict(cu=None), B.ATTN_ERR_INVALID_ARG),      # 9 tokens, 2 sequences
    (dict(B_=0), B.ATTN_ERR_INVALID_ARG),
    (dict(Hkv=0), B.ATTN_ERR_INVALID_ARG),
    (dict(total=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(total=1 << 31), B.ATTN_ERR_INVALID_ARG),
    (dict(maxp=0), B.ATTN_ERR_INVALID_ARG),
    (dict(npages=1 << 28), B.ATTN_ERR_INVALID_ARG),
    (dict(inter=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(m=float("inf")), B.ATTN_ERR_INVALID_ARG),
    (dict(d=256), B.ATTN_ERR_UNSUPPORTED),
    (dict(ps=24), B.ATTN_ERR_UNSUPPORTED),
    (dict(ps=512), B.ATTN_ERR_UNSUPPORTED),
    (dict(rot=8), B.ATTN_ERR_UNSUPPORTED),
    (dict(k=FAKE + 8), B.ATTN_ERR_ALIGNMENT),
    (dict(vc=FAKE + 8), B.ATTN_ERR_ALIGNMENT),
    (dict(tbl=FAKE + 2), B.ATTN_ERR_ALIGNMENT),
    (dict(freq=FAKE + 4), B.ATTN_ERR_ALIGNMENT),
    (dict(strides=[512, 128, 256, 128, 256, -128]), B.ATTN_ERR_INVALID_ARG),
    (dict(strides=[512, 128, 260, 128, 256, 128]), B.ATTN_ERR_ALIGNMENT),
])
def test_append_validation(lib, fp8, kw, status):
    assert _append(lib, fp8, **kw) == status


def test_append_fp8_scales(lib):
    assert _append(lib, True, ks=None) == B.ATTN_ERR_INVALID_ARG
    assert _append(lib, True, vs=FAKE + 2) == B.ATTN_ERR_ALIGNMENT


def test_append_of_no_tokens_launches_nothing(lib):
    assert _append(lib, total=0, q=None, k=None, v=None, qo=None) == B.ATTN_OK


def test_binding_refuses_host_tensors():
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    f = torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="CUDA"):
        B.attn_rope(x, None, f)
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    c = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        B.attn_append_paged(k, k, c, c, torch.zeros(2, 2, dtype=torch.int32),
                            torch.ones(2, dtype=torch.int32))


def test_counts_are_clamped_to_a_c_int():
    assert B._tokens(5) == 5 and B._tokens(2 ** 31 - 1) == 2 ** 31 - 1
    assert B._tokens(2 ** 31) == 2 ** 31 - 1 and B._tokens(2 ** 40 + 7) == 2 ** 31 - 1
    assert B._tokens(-3) == -1 and B._tokens(-2 ** 40) == -1
