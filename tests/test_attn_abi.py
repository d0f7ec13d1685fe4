"""Refusals of the windowed-attention and 8-bit-cache calls at the C boundary, without a GPU: only
argument combinations that fail validation are passed, so nothing is launched and no pointer
is dereferenced. Every accepted-looking call below has a misaligned output as a second guard."""
import pytest

from sparse_dynamic_routing_b200 import _binding as bnd
from sparse_dynamic_routing_b200 import build

FAKE, NULL = 0x1000, None


@pytest.fixture(scope="module")
def lib():
    build.build()
    return bnd.load_library()


def forward(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, dtype=bnd.GM_BF16, lens=NULL, B=1, n=8, hq=4, hkv=2, d=64, window=3, sinks=1,
             scale=0.1, o=FAKE + 8, lse=NULL, stream=NULL)
    a.update(kw)
    return lib.gm_window_attention_forward(*a.values())


def backward(lib, **kw):
    a = dict(q=FAKE, k=FAKE, v=FAKE, o=FAKE, dout=FAKE, lse=FAKE, dtype=bnd.GM_BF16, lens=NULL, B=1, n=8, hq=4, hkv=2,
             d=64, window=3, sinks=1, scale=0.1, dq=FAKE + 8, dk=FAKE, dv=FAKE, ws=FAKE, size=1 << 20, stream=NULL)
    a.update(kw)
    return lib.gm_window_attention_backward(*a.values())


COMMON = [(dict(B=-1), bnd.GM_ERR_INVALID_ARG), (dict(n=-1), bnd.GM_ERR_INVALID_ARG),
          (dict(hq=0), bnd.GM_ERR_INVALID_ARG), (dict(hkv=0), bnd.GM_ERR_INVALID_ARG),
          (dict(hq=3), bnd.GM_ERR_INVALID_ARG), (dict(window=0), bnd.GM_ERR_INVALID_ARG),
          (dict(sinks=-1), bnd.GM_ERR_INVALID_ARG), (dict(scale=float("nan")), bnd.GM_ERR_INVALID_ARG),
          (dict(scale=float("inf")), bnd.GM_ERR_INVALID_ARG), (dict(dtype=5), bnd.GM_ERR_INVALID_ARG),
          (dict(d=96), bnd.GM_ERR_UNSUPPORTED), (dict(d=256), bnd.GM_ERR_UNSUPPORTED),
          (dict(n=1 << 30), bnd.GM_ERR_UNSUPPORTED), (dict(B=1 << 16, n=1 << 16), bnd.GM_ERR_UNSUPPORTED),
          (dict(B=0), bnd.GM_OK), (dict(n=0), bnd.GM_OK)]


@pytest.mark.parametrize("kw,status", COMMON)
def test_window(lib, kw, status):
    assert forward(lib, **kw) == status
    assert backward(lib, **kw) == status


def test_window_pointers(lib):
    assert forward(lib) == bnd.GM_ERR_INVALID_ARG  # misaligned o
    for x in ("q", "k", "v", "o"):
        assert forward(lib, **{x: NULL}) == bnd.GM_ERR_INVALID_ARG
    assert backward(lib) == bnd.GM_ERR_INVALID_ARG  # misaligned dq
    for x in ("q", "k", "v", "o", "dout", "lse", "dk", "dv", "ws"):
        assert backward(lib, **{x: NULL}) == bnd.GM_ERR_INVALID_ARG
    size = lib.gm_window_attention_backward_workspace_size
    need = size(bnd.GM_BF16, 1, 8, 4, 2, 64, 3, 1)
    assert need >= 8 * 4 * 4
    assert backward(lib, dq=FAKE, size=need - 1) == bnd.GM_ERR_INVALID_ARG
    assert size(bnd.GM_BF16, 0, 8, 4, 2, 64, 3, 1) == 0 and size(bnd.GM_BF16, 1, 8, 4, 3, 64, 3, 1) == 0
    assert size(bnd.GM_F32, 1, 8, 4, 2, 64, 3, 1) >= 8 * 4 * 4
    # a few keys that every query of a long sequence sees: their steps are shared out
    assert size(bnd.GM_BF16, 1, 32768, 16, 8, 128, 512, 4) > size(bnd.GM_BF16, 1, 32768, 16, 8, 128, 512, 0)


CACHE = dict(kq=FAKE, vq=FAKE, ks=FAKE, vs=FAKE, pages=4, page=16, table=FAKE, maxp=2, lens=FAKE)


def append(lib, **kw):
    a = dict(k=FAKE + 8, v=FAKE, dtype=bnd.GM_BF16, B=1, t=1, hkv=2, d=64, **CACHE, new=NULL, stream=NULL)
    a.update(kw)
    return lib.gm_kv8_append(*a.values())


def attention(lib, **kw):
    a = dict(q=FAKE, dtype=bnd.GM_BF16, B=1, t=1, hq=4, hkv=2, d=64, **CACHE, ql=NULL, window=3, sinks=0, scale=0.1,
             o=FAKE + 8, lse=NULL, ws=NULL, size=0, stream=NULL)
    a.update(kw)
    return lib.gm_kv8_attention_forward(*a.values())


def sea(lib, **kw):
    a = dict(q=FAKE, dtype=bnd.GM_BF16, idx=FAKE, w=FAKE, s=4, B=1, t=1, hq=4, hkv=2, d=64, **CACHE, ql=NULL, scale=0.1,
             o=FAKE + 8, lse=NULL, stream=NULL)
    a.update(kw)
    return lib.gm_kv8_sea_forward(*a.values())


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), bnd.GM_ERR_INVALID_ARG), (dict(t=-1), bnd.GM_ERR_INVALID_ARG), (dict(hkv=0), bnd.GM_ERR_INVALID_ARG),
    (dict(dtype=9), bnd.GM_ERR_INVALID_ARG), (dict(pages=-1), bnd.GM_ERR_INVALID_ARG),
    (dict(maxp=-1), bnd.GM_ERR_INVALID_ARG), (dict(page=0), bnd.GM_ERR_INVALID_ARG),
    (dict(page=24), bnd.GM_ERR_UNSUPPORTED), (dict(page=256), bnd.GM_ERR_UNSUPPORTED),
    (dict(d=32), bnd.GM_ERR_UNSUPPORTED), (dict(maxp=1 << 30), bnd.GM_ERR_UNSUPPORTED),
    (dict(lens=NULL), bnd.GM_ERR_INVALID_ARG), (dict(table=NULL), bnd.GM_ERR_INVALID_ARG),
    (dict(kq=NULL), bnd.GM_ERR_INVALID_ARG), (dict(vs=NULL), bnd.GM_ERR_INVALID_ARG),
    (dict(kq=FAKE + 4), bnd.GM_ERR_INVALID_ARG), (dict(), bnd.GM_ERR_INVALID_ARG),
    (dict(B=0), bnd.GM_OK), (dict(t=0), bnd.GM_OK)])
def test_cache(lib, kw, status):
    for f in (append, attention, sea):
        assert f(lib, **kw) == status, f.__name__


def test_cache_own_arguments(lib):
    for f in (attention, sea):
        for kw in (dict(hq=3), dict(scale=float("nan")), dict(q=NULL), dict(o=NULL), dict(q=FAKE + 2)):
            assert f(lib, **kw) == bnd.GM_ERR_INVALID_ARG
    for kw in (dict(window=0), dict(sinks=-1)):
        assert attention(lib, **kw) == bnd.GM_ERR_INVALID_ARG
    for kw in (dict(s=0), dict(s=33), dict(idx=NULL), dict(w=NULL)):
        assert sea(lib, **kw) == bnd.GM_ERR_INVALID_ARG
    assert append(lib, k=NULL) == bnd.GM_ERR_INVALID_ARG
    assert append(lib, k=FAKE, v=FAKE + 2) == bnd.GM_ERR_INVALID_ARG


def test_cache_workspace(lib):
    size = lib.gm_kv8_attention_workspace_size
    assert size(512, 1, 16, 8, 128, 64, 4, 1 << 30, 0) == 0  # many rows of few keys: nothing to join
    need = size(1, 1, 16, 8, 128, 64, 1024, 1 << 30, 0)
    assert need > 0
    a = dict(maxp=1024, page=64, d=128, hq=16, hkv=8, window=1 << 30, o=FAKE)
    for kw in (dict(ws=NULL, size=need), dict(ws=FAKE, size=need - 1), dict(ws=FAKE + 4, size=need)):
        assert attention(lib, **a, **kw) == bnd.GM_ERR_INVALID_ARG
    assert size(0, 1, 16, 8, 128, 64, 4, 1, 0) == 0 and size(1, 1, 3, 2, 128, 64, 4, 1, 0) == 0
