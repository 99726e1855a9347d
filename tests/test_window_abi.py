"""Host-side checks of the window-with-first-tokens entry points (CPU; nothing is launched)."""
import pytest

from exact_softmax_attention_fwd_b200 import _binding as B
from exact_softmax_attention_fwd_b200 import build as build_mod

FAKE = 0x100000  # 16-byte aligned, never dereferenced: every call below fails validation


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.load_library()


def _fwd(lib, q=FAKE, k=FAKE, o=FAKE, Hq=4, Hkv=2, Sq=100, Sk=100, d=128, scale=0.1, window=16,
         sinks=4):
    return lib.attn_fwd_window_sinks(q, k, FAKE, o, None, 1, Hq, Hkv, Sq, Sk, d, scale, None, window,
                                     sinks, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), B.ATTN_ERR_INVALID_ARG), (dict(o=None), B.ATTN_ERR_INVALID_ARG),
    (dict(Hq=3), B.ATTN_ERR_INVALID_ARG), (dict(Sq=0), B.ATTN_ERR_INVALID_ARG),
    (dict(window=-1), B.ATTN_ERR_INVALID_ARG), (dict(sinks=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(scale=float("inf")), B.ATTN_ERR_INVALID_ARG), (dict(d=96), B.ATTN_ERR_UNSUPPORTED),
    (dict(k=FAKE + 8), B.ATTN_ERR_ALIGNMENT)])
def test_forward_validation(lib, kw, status):
    assert _fwd(lib, **kw) == status


def _bwd(lib, q=FAKE, lse=FAKE, dk=FAKE, Hq=4, Hkv=2, Sq=2000, Sk=2000, d=128, window=16, sinks=4,
         ws=FAKE, ws_bytes=None):
    if ws_bytes is None:
        ws_bytes = lib.attn_bwd_window_sinks_workspace_size(1, Hq, Hkv, Sq, Sk, d, window, sinks)
    return lib.attn_bwd_window_sinks(q, FAKE, FAKE, FAKE, lse, FAKE, FAKE, dk, FAKE, 1, Hq, Hkv, Sq,
                                     Sk, d, 0.1, None, window, sinks, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), B.ATTN_ERR_INVALID_ARG), (dict(lse=None), B.ATTN_ERR_INVALID_ARG),
    (dict(dk=None), B.ATTN_ERR_INVALID_ARG), (dict(ws=None), B.ATTN_ERR_INVALID_ARG),
    (dict(window=-1, ws_bytes=0), B.ATTN_ERR_INVALID_ARG),
    (dict(sinks=-1, ws_bytes=0), B.ATTN_ERR_INVALID_ARG),
    (dict(d=80, ws_bytes=1 << 30), B.ATTN_ERR_UNSUPPORTED),
    (dict(ws=FAKE + 8), B.ATTN_ERR_ALIGNMENT),
    (dict(ws_bytes=8 * 4 * 2048), B.ATTN_ERR_WORKSPACE)])   # the statistics alone
def test_backward_validation(lib, kw, status):
    assert _bwd(lib, **kw) == status


def test_backward_workspace(lib):
    size = lib.attn_bwd_window_sinks_workspace_size
    base = lib.attn_bwd_workspace_size(2, 8, 4096)
    assert size(2, 8, 2, 4096, 4096, 128, 0, 4) == base       # no window
    assert size(2, 8, 2, 4096, 4096, 128, 256, 0) == base     # no first tokens
    assert size(2, 8, 2, 4096, 4096, 128, 4096, 4) == base    # the window reaches every row
    far = size(2, 8, 2, 4096, 4096, 128, 256, 4) - base
    row = 4 * 4 * 2 * 128 * 4   # 4 (sequence, KV head) pairs, 4 tokens, dK and dV, fp32
    assert far > row and far % row == 0
    # many first tokens: bounded by four units an SM, not by their number; none when the key
    # tiles alone are as many
    stats = lib.attn_bwd_workspace_size(1, 8, 32768)
    assert size(1, 8, 8, 32768, 32768, 128, 128, 8192) == stats
    for sinks in (128, 1000, 4000):
        assert 0 < size(1, 8, 8, 32768, 32768, 128, 128, sinks) - stats <= 900 * 128 * 2 * 128 * 4
    assert size(0, 8, 2, 4096, 4096, 128, 256, 4) == 0
    assert size(1, 8, 3, 4096, 4096, 128, 256, 4) == 0
    assert size(1, 8, 2, 4096, 4096, 96, 256, 4) == 0


def _paged(lib, q=FAKE, kc=FAKE, tbl=FAKE, page=16, B_=2, total=50, maxq=30, d=128, window=16,
           sinks=4, ws=FAKE, ws_bytes=None):
    if ws_bytes is None:
        ws_bytes = lib.attn_fwd_paged_window_workspace_size(B_, 4, 2, total, maxq) if B_ > 0 else 0
    return lib.attn_fwd_paged_window(q, kc, FAKE, tbl, FAKE, FAKE, page, B_, 4, 2, total, maxq, 8, 20,
                                     d, 0.1, window, sinks, FAKE, None, ws, ws_bytes, None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), B.ATTN_ERR_INVALID_ARG), (dict(tbl=None), B.ATTN_ERR_INVALID_ARG),
    (dict(B_=0), B.ATTN_ERR_INVALID_ARG), (dict(window=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(sinks=-3), B.ATTN_ERR_INVALID_ARG), (dict(maxq=0), B.ATTN_ERR_INVALID_ARG),
    (dict(page=48), B.ATTN_ERR_UNSUPPORTED), (dict(d=32), B.ATTN_ERR_UNSUPPORTED),
    (dict(kc=FAKE + 8), B.ATTN_ERR_ALIGNMENT), (dict(ws=None), B.ATTN_ERR_WORKSPACE),
    (dict(ws_bytes=8), B.ATTN_ERR_WORKSPACE)])
def test_paged_validation(lib, kw, status):
    assert _paged(lib, **kw) == status


def test_paged_workspace(lib):
    size = lib.attn_fwd_paged_window_workspace_size
    # the unit list: a 16-byte header and 8 bytes for each possible unit of 256 rows
    assert size(3, 4, 4, 1000, 512) == 16 + 8 * (1000 // 256 + 4)
    assert size(3, 8, 2, 1000, 512) == 16 + 8 * (4000 // 256 + 4)     # a group's heads as rows
    assert size(3, 6, 2, 1000, 512) == 16 + 8 * (1000 // 256 + 4)     # groups of 3: not
    for bad in ((0, 4, 2, 10, 10), (1, 4, 3, 10, 10), (1, 4, 2, -1, 10), (1, 4, 2, 10, 0)):
        assert size(*bad) == 0


def test_paged_without_tokens_launches_nothing(lib):
    assert _paged(lib, total=0) == B.ATTN_OK


def _decode(lib, fp8=False, q=FAKE, kc=FAKE, ks=FAKE, vs=FAKE, tbl=FAKE, lens=FAKE, page=16, B_=2,
            Hq=4, Hkv=2, d=128, maxp=8, npages=20, scale=0.1, window=16, sinks=4, o=FAKE, lse=None):
    fn = lib.attn_decode_paged_window_fp8 if fp8 else lib.attn_decode_paged_window
    return fn(q, kc, FAKE, *((ks, vs) if fp8 else ()), tbl, lens, page, B_, Hq, Hkv, d, maxp, npages,
              scale, window, sinks, o, lse, None)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("kw,status", [
    (dict(q=None), B.ATTN_ERR_INVALID_ARG), (dict(tbl=None), B.ATTN_ERR_INVALID_ARG),
    (dict(o=None), B.ATTN_ERR_INVALID_ARG), (dict(B_=0), B.ATTN_ERR_INVALID_ARG),
    (dict(Hq=5), B.ATTN_ERR_INVALID_ARG), (dict(window=-1), B.ATTN_ERR_INVALID_ARG),
    (dict(sinks=-1), B.ATTN_ERR_INVALID_ARG), (dict(scale=float("nan")), B.ATTN_ERR_INVALID_ARG),
    (dict(maxp=1 << 27), B.ATTN_ERR_INVALID_ARG), (dict(npages=1 << 28), B.ATTN_ERR_INVALID_ARG),
    (dict(page=8), B.ATTN_ERR_UNSUPPORTED), (dict(page=272), B.ATTN_ERR_UNSUPPORTED),
    (dict(d=96), B.ATTN_ERR_UNSUPPORTED), (dict(Hq=18), B.ATTN_ERR_UNSUPPORTED),
    (dict(kc=FAKE + 8), B.ATTN_ERR_ALIGNMENT), (dict(lens=FAKE + 1), B.ATTN_ERR_ALIGNMENT),
    (dict(lse=FAKE + 2), B.ATTN_ERR_ALIGNMENT)])
def test_decode_validation(lib, fp8, kw, status):
    assert _decode(lib, fp8, **kw) == status


def test_decode_fp8_scales(lib):
    assert _decode(lib, True, vs=None) == B.ATTN_ERR_INVALID_ARG
    assert _decode(lib, True, ks=FAKE + 2) == B.ATTN_ERR_ALIGNMENT
