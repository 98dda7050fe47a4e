"""The entry points around cached attention reject bad arguments on the host, before anything is launched."""
from __future__ import annotations

import ctypes

import pytest
import torch

import exact_tiled_attention_fa_gb300 as fa
from exact_tiled_attention_fa_gb300 import build as fa_build

P = ctypes.c_void_p(0x10000000)  # never dereferenced: each call below is rejected first
V = ctypes.c_void_p(0x12000000)
NULL = ctypes.c_void_p(0)
ODD = ctypes.c_void_p(0x10000008)
INVALID, UNSUPPORTED, WORKSPACE = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED, fa.FA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    return fa.library()


def caller(f, names, values):
    def call(**kw):
        assert not set(kw) - set(names), kw
        return f(*[kw.get(n, v) for n, v in zip(names, values)])
    return call


COMMON = [("B", 2), ("N", 5), ("Hq", 4), ("Hkv", 2), ("d", 64), ("rot", 64), ("max_pos", 100), ("interleaved", 0)]


def fwd(lib):
    spec = [(n, P) for n in ("q", "k", "v", "wq", "wk", "cos", "sin", "pos", "qo", "ko", "vo")]
    spec += [("qs", 512), ("ks", 512), ("vs", 512)] + COMMON + [("expand", 0), ("eps", 1e-6), ("wdt", 0), ("stream", NULL)]
    return caller(lib.fa_qk_norm_rope, [n for n, _ in spec], [v for _, v in spec])


def bwd(lib):
    spec = [(n, P) for n in ("dq", "dk", "dv", "q", "k", "wq", "wk", "cos", "sin", "pos", "gq", "gk", "gv", "gwq", "gwk", "ws")]
    spec += [("ws_bytes", 1 << 30)] + [(n, 512) for n in ("qs", "ks", "gqs", "gks", "gvs")] + COMMON
    spec += [("expand", 0), ("eps", 1e-6), ("wdt", 0), ("gdt", 0), ("odt", 0), ("stream", NULL)]
    return caller(lib.fa_qk_norm_rope_bwd, [n for n, _ in spec], [v for _, v in spec])


def append(lib):
    spec = [(n, P) for n in ("q", "k", "v", "wq", "wk", "cos", "sin", "lens", "par", "cnt", "qo", "ko")] + [("vo", V)]
    spec += [("qs", 512), ("ks", 512), ("vs", 512), ("B", 2), ("N", 5), ("Hq", 4), ("Hkv", 2), ("Nk", 64), ("d", 64), ("rot", 64),
             ("max_pos", 100), ("interleaved", 0), ("eps", 1e-6), ("wdt", 0), ("stream", NULL)]
    return caller(lib.fa_qk_norm_rope_append, [n for n, _ in spec], [v for _, v in spec])


def tree(lib):
    spec = [(n, P) for n in ("q", "k", "v", "lens", "par", "cnt", "o", "lse", "ws")]
    spec += [("ws_bytes", 1 << 40), ("B", 2), ("Hq", 4), ("Hkv", 2), ("T", 8), ("Nk", 64), ("d", 64), ("dv", 64), ("scale", 0.1),
             ("odt", 0), ("stream", NULL)]
    return caller(lib.fa_decode_tree, [n for n, _ in spec], [v for _, v in spec])


def compact(lib):
    spec = [("k", P), ("v", V), ("lens", ctypes.c_void_p(0x20000000)), ("acc", P), ("cnt", P), ("out", ctypes.c_void_p(0x30000000))]
    spec += [("L", 1), ("B", 2), ("Hkv", 2), ("Nk", 64), ("d", 64), ("dv", 64), ("T", 8), ("stream", NULL)]
    return caller(lib.fa_cache_compact, [n for n, _ in spec], [v for _, v in spec])


@pytest.mark.parametrize("make", [fwd, bwd, append])
def test_norm_calls_share_their_refusals(lib, make):
    call = make(lib)
    for kw in (dict(q=NULL), dict(k=NULL), dict(wq=NULL), dict(wk=NULL), dict(cos=NULL), dict(sin=NULL), dict(q=ODD), dict(k=ODD),
               dict(cos=ODD), dict(sin=ODD), dict(wq=ctypes.c_void_p(0x10000002)), dict(B=0), dict(N=-1), dict(Hq=0), dict(Hkv=0),
               dict(Hq=3), dict(d=0), dict(rot=0), dict(rot=80), dict(max_pos=0), dict(interleaved=2), dict(eps=-1.0),
               dict(eps=float("nan")), dict(eps=float("inf")), dict(wdt=2), dict(qs=248), dict(ks=120), dict(qs=516),
               dict(qs=-512), dict(B=1 << 16, N=1 << 15)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(d=48, rot=48), dict(d=96, rot=96), dict(rot=24), dict(rot=8)):
        assert call(**kw) == UNSUPPORTED, kw


def test_norm_forward_refusals(lib):
    call = fwd(lib)
    for kw in (dict(qo=NULL), dict(ko=NULL), dict(v=NULL), dict(vo=NULL), dict(v=ODD), dict(qo=ODD), dict(vs=120), dict(expand=2),
               dict(pos=ctypes.c_void_p(0x10000002))):
        assert call(**kw) == INVALID, kw


def test_norm_backward_refusals(lib):
    call = bwd(lib)
    for kw in (dict(dq=NULL), dict(dk=NULL), dict(dv=NULL), dict(gv=NULL), dict(gq=NULL), dict(gwq=NULL), dict(gwk=NULL),
               dict(ws=NULL), dict(ws=ctypes.c_void_p(0x10000010)), dict(gq=ODD), dict(dk=ODD), dict(gdt=3), dict(odt=-1),
               dict(gqs=248), dict(gks=124), dict(gvs=8), dict(expand=-1)):
        assert call(**kw) == INVALID, kw
    need = lib.fa_qk_norm_rope_bwd_workspace_size(64)
    assert need == 8192 * 64 and lib.fa_qk_norm_rope_bwd_workspace_size(0) == 0
    assert call(ws_bytes=need - 1) == WORKSPACE


def test_append_refusals(lib):
    call = append(lib)
    for kw in (dict(v=NULL), dict(lens=NULL), dict(qo=NULL), dict(ko=NULL), dict(vo=NULL), dict(Nk=0), dict(ko=ODD),
               dict(par=ctypes.c_void_p(0x10000002)), dict(vs=64), dict(vo=P), dict(vo=ctypes.c_void_p(0x10007ff0))):
        assert call(**kw) == INVALID, kw
    assert call(N=129) == UNSUPPORTED


def test_tree_refusals(lib):
    call = tree(lib)
    for kw in (dict(q=NULL), dict(k=NULL), dict(v=NULL), dict(lens=NULL), dict(o=NULL), dict(ws=NULL), dict(q=ODD), dict(o=ODD),
               dict(ws=ctypes.c_void_p(0x10000080)), dict(cnt=ctypes.c_void_p(0x10000001)), dict(B=0), dict(T=0), dict(Hkv=3),
               dict(Nk=0), dict(scale=0.0), dict(scale=float("inf")), dict(odt=2),
               dict(Hq=1 << 16, Hkv=2, T=128), dict(B=1 << 15, Hkv=1 << 16, Hq=1 << 16), dict(Nk=0x7fffffff)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(T=129), dict(d=96, dv=96), dict(dv=128)):
        assert call(**kw) == UNSUPPORTED, kw
    size = lib.fa_decode_tree_workspace_size
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    assert size(8, 2, 5, 128, 152) == up(4 * 152 * 20 * 512) + up(4 * 152 * 20 * 4) + up(32 * 152)
    assert size(8, 2, 100, 64, 152) == up(2 * 152 * 256 * 256) + up(2 * 152 * 256 * 4) + up(16 * 152)
    assert size(3, 2, 5, 64, 152) == 0 and size(4, 2, 0, 64, 152) == 0 and size(4, 2, 1, 64, 0) == 0


def test_compact_refusals(lib):
    call = compact(lib)
    for kw in (dict(k=NULL), dict(v=NULL), dict(lens=NULL), dict(acc=NULL), dict(cnt=NULL), dict(k=ODD), dict(L=0), dict(B=0),
               dict(T=0), dict(Nk=0), dict(out=ctypes.c_void_p(0x20000000)), dict(out=ctypes.c_void_p(0x20000004)),
               dict(out=ctypes.c_void_p(0x1ffffffc)), dict(out=P), dict(acc=ctypes.c_void_p(0x2fffffe0)), dict(v=P),
               dict(v=ctypes.c_void_p(0x10007ff0)), dict(L=1 << 15, B=1 << 15, Hkv=4)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(T=129), dict(d=96, dv=96), dict(dv=32)):
        assert call(**kw) == UNSUPPORTED, kw


def test_binding_refuses_host_tensors_and_wrong_layouts(lib):
    q = torch.zeros((1, 2, 4, 64), dtype=torch.bfloat16)
    w, t = torch.ones(64), torch.ones((9, 32))
    with pytest.raises(ValueError, match="CUDA"):
        fa.qk_norm_rope(q, q, q, w, w, t, t)
    with pytest.raises(ValueError, match="bfloat16"):
        fa.qk_norm_rope(q.float(), q, q, w, w, t, t)
    with pytest.raises(TypeError):
        fa.decode_tree(None, q, q, w)
    with pytest.raises(ValueError, match="CUDA"):
        fa.cache_compact(q, q, w, w, w)
