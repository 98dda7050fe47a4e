"""The entry points of attention under score rules reject bad arguments on the host, before anything is launched."""
from __future__ import annotations

import ctypes

import pytest
import torch

import exact_tiled_attention_fa_gb300 as fa
from exact_tiled_attention_fa_gb300 import build as fa_build

P = ctypes.c_void_p(0x10000000)  # never dereferenced: each call below is rejected first
NULL = ctypes.c_void_p(0)
ODD = ctypes.c_void_p(0x10000008)
ODD4 = ctypes.c_void_p(0x10000002)
INVALID, UNSUPPORTED, WORKSPACE = fa.FA_ERR_INVALID_ARG, fa.FA_ERR_UNSUPPORTED, fa.FA_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    fa_build.build()
    return fa.library()


def caller(f, spec):
    names = [n for n, _ in spec]

    def call(**kw):
        assert not set(kw) - set(names), kw
        return f(*[kw.get(n, v) for n, v in spec])
    return call


SIZES = [("B", 2), ("Hq", 4), ("Hkv", 2), ("N", 300), ("Nk", 300), ("d", 64), ("dv", 64), ("causal", 1), ("scale", 0.125), ("cap", 0.0)]


def fwd(lib):
    return caller(lib.fa_fwd_rules, [(n, P) for n in ("q", "k", "v", "slopes", "docs", "prefix", "o", "lse", "ws")] +
                  [("ws_bytes", 1 << 40)] + SIZES + [("odt", 0), ("stream", NULL)])


def bwd(lib):
    return caller(lib.fa_bwd_rules, [(n, P) for n in ("q", "k", "v", "o", "lse", "do", "slopes", "docs", "prefix", "dq", "dk", "dvg", "ws")] +
                  [("ws_bytes", 1 << 40)] + SIZES + [("odt", 0), ("gdt", 0), ("stream", NULL)])


@pytest.mark.parametrize("make", [fwd, bwd])
def test_shared_refusals(lib, make):
    call = make(lib)
    for kw in (dict(q=NULL), dict(k=NULL), dict(v=NULL), dict(o=NULL), dict(q=ODD), dict(k=ODD), dict(v=ODD), dict(o=ODD), dict(lse=ODD4),
               dict(slopes=ODD4), dict(docs=ODD4), dict(prefix=ODD4), dict(ws=NULL), dict(ws=ctypes.c_void_p(0x10000080)), dict(B=0),
               dict(Hq=0), dict(Hkv=0), dict(Hkv=3), dict(N=0), dict(Nk=-1), dict(d=0), dict(dv=0), dict(causal=2), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(cap=-1.0), dict(cap=float("nan")),
               dict(cap=float("inf")), dict(scale=1e-30, cap=1e30), dict(scale=1e30, cap=1e-30), dict(cap=3.4e38), dict(odt=2),
               dict(B=1 << 15, Hq=1 << 15, Hkv=1), dict(N=0x7fffff80), dict(Nk=0x7fffff80), dict(Nk=0x7fff8000), dict(B=1 << 12, Hq=1 << 12, N=1 << 14)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(d=96, dv=96), dict(d=48, dv=48), dict(dv=128)):
        assert call(**kw) == UNSUPPORTED, kw


def test_backward_refusals(lib):
    call = bwd(lib)
    for kw in (dict(lse=NULL), dict(do=NULL), dict(dq=NULL), dict(dk=NULL), dict(dvg=NULL), dict(do=ODD), dict(dq=ODD), dict(dk=ODD),
               dict(dvg=ODD), dict(gdt=3)):
        assert call(**kw) == INVALID, kw


def test_workspace_sizes(lib):
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    size = lib.fa_fwd_rules_workspace_size
    assert size(3, 1000) == 256 + up(3 * 1000 * 8) + up(3 * 8 * 8)
    assert size(0, 5) == 0 and size(5, 0) == 0
    assert fwd(lib)(ws_bytes=size(2, 300) - 1) == WORKSPACE
    size = lib.fa_bwd_rules_workspace_size
    # one head: no parts
    assert size(2, 4, 4, 300, 500, 64, 152) == lib.fa_bwd_workspace_size(2, 4, 300, 64) + 256 + up(2 * 500 * 8) + up(2 * 4 * 8)
    # 8 query heads to one key/value head and few items: sums of 8 parts
    assert size(1, 8, 1, 300, 300, 64, 152) == (lib.fa_bwd_workspace_size(1, 8, 300, 64) + 256 + up(300 * 8) + up(3 * 8) +
                                                2 * up(8 * 300 * 64 * 4))
    for bad in ((0, 4, 2, 9, 9, 64, 152), (1, 4, 3, 9, 9, 64, 152), (1, 4, 2, 9, 9, 64, 0), (1, 4, 2, 0, 9, 64, 152)):
        assert size(*bad) == 0


def test_binding_refuses_host_tensors_and_wrong_layouts(lib):
    q = torch.zeros((1, 2, 4, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        fa.fwd_rules(q, q, q)
    with pytest.raises(ValueError, match="bfloat16"):
        fa.fwd_rules(q.float(), q, q)
    with pytest.raises(TypeError):
        fa.bwd_rules(None, q, q, q, q, q)


@pytest.mark.gpu
def test_binding_refusals_on_the_device(lib):
    q = torch.zeros((2, 4, 30, 64), dtype=torch.bfloat16, device="cuda")
    k = torch.zeros((2, 2, 40, 64), dtype=torch.bfloat16, device="cuda")
    docs = torch.zeros((2, 40), dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="documents"):
        fa.fwd_rules(q, k, k, documents=docs.long())
    with pytest.raises(ValueError, match="documents"):
        fa.fwd_rules(q, k, k, documents=docs[:, :39].contiguous())
    with pytest.raises(ValueError, match="slopes"):
        fa.fwd_rules(q, k, k, slopes=torch.ones(2, device="cuda"))
    with pytest.raises(ValueError, match="prefix_lens"):
        fa.fwd_rules(q, k, k, prefix_lens=torch.zeros(2, device="cuda"))
    with pytest.raises(ValueError, match="contiguous"):
        fa.fwd_rules(q, k.transpose(2, 3).contiguous().transpose(2, 3), k)
    with pytest.raises(ValueError, match="v must be"):
        fa.fwd_rules(q, k, k[:, :, :39].contiguous())
    with pytest.raises(fa.FaError):
        fa.fwd_rules(q, k[:, :1].repeat(1, 3, 1, 1), k[:, :1].repeat(1, 3, 1, 1))  # 3 heads do not divide 4
    with pytest.raises(fa.FaError):
        fa.fwd_rules(q, k, k, softcap=-1.0)
    o, lse = fa.fwd_rules(q, k, k)
    with pytest.raises(ValueError, match="lse"):
        fa.bwd_rules(q, k, k, o, lse[:, :2].contiguous(), q)
    with pytest.raises(fa.FaError) as e:
        fa.bwd_rules(q, k, k, o, lse, q, workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))
    assert e.value.status == WORKSPACE
    with pytest.raises(ValueError, match="grads"):
        fa.bwd_rules(q, k, k, o, lse, q, grads=(torch.empty_like(q), None, None))


def decode(lib):
    return caller(lib.fa_decode_prefix, [(n, P) for n in ("q", "kp", "vp", "plen", "k", "v", "lens", "slopes", "o", "lse", "ws")] +
                  [("ws_bytes", 1 << 40), ("B", 2), ("Hq", 4), ("Hkv", 2), ("P_max", 300), ("Nk", 64), ("d", 64), ("dv", 64),
                   ("scale", 0.125), ("cap", 0.0), ("odt", 0), ("stream", NULL)])


def test_decode_prefix_refusals(lib):
    call = decode(lib)
    for kw in (dict(q=NULL), dict(k=NULL), dict(v=NULL), dict(lens=NULL), dict(o=NULL), dict(ws=NULL), dict(kp=NULL), dict(vp=NULL),
               dict(kp=NULL, vp=NULL), dict(kp=NULL, vp=NULL, P_max=0), dict(P_max=0), dict(P_max=-1), dict(q=ODD), dict(kp=ODD),
               dict(vp=ODD), dict(k=ODD), dict(v=ODD), dict(o=ODD), dict(lse=ODD4), dict(plen=ODD4), dict(lens=ODD4), dict(slopes=ODD4),
               dict(ws=ctypes.c_void_p(0x10000080)), dict(B=0), dict(Hq=0), dict(Hkv=3), dict(Hkv=0), dict(Nk=0), dict(d=0), dict(dv=0),
               dict(scale=0.0), dict(cap=-1.0), dict(cap=float("nan")), dict(odt=2), dict(P_max=0x40000000), dict(Nk=0x40000000),
               dict(B=1 << 16, Hq=1 << 16, Hkv=1 << 15), dict(B=1 << 12, Hq=1 << 10, Hkv=1 << 10, Nk=1 << 25)):
        assert call(**kw) == INVALID, kw
    for kw in (dict(d=96, dv=96), dict(dv=32), dict(Hq=258, Hkv=2)):
        assert call(**kw) == UNSUPPORTED, kw


def test_decode_prefix_workspace_size(lib):
    up = lambda x: (x + 255) // 256 * 256  # noqa: E731
    size = lib.fa_decode_prefix_workspace_size
    # 16 sequences of 4 rows: one tile of 64
    own = 4 * 152 * 64
    assert size(16, 32, 8, 128, 152) == (up(own * 512) + up(own * 4) + up(2 * 16 * 32 * 512) + up(2 * 16 * 32 * 4) + up((8 + 128) * 16))
    # 64 sequences of 4 rows: two tiles of 128
    own = 4 * 152 * 128
    assert size(64, 32, 8, 64, 152) == (up(own * 256) + up(own * 4) + up(2 * 64 * 32 * 256) + up(2 * 64 * 32 * 4) + up((16 + 512) * 16))
    assert size(0, 4, 2, 64, 152) == 0 and size(1, 3, 2, 64, 152) == 0 and size(1, 4, 2, 64, 0) == 0 and size(1, 258, 2, 64, 152) == 0


@pytest.mark.gpu
def test_decode_prefix_binding_refusals(lib):
    z = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    q, kp, k = z(2, 4, 1, 64), z(2, 30, 64), z(2, 2, 40, 64)
    n = torch.ones(2, dtype=torch.int32, device="cuda")
    fa.decode_prefix(q, kp, kp, k, k, n)
    with pytest.raises(ValueError, match="q must be"):
        fa.decode_prefix(z(2, 4, 2, 64), kp, kp, k, k, n)
    with pytest.raises(ValueError, match="v_prefix"):
        fa.decode_prefix(q, kp, kp[:, :29].contiguous(), k, k, n)
    with pytest.raises(ValueError, match="go with"):
        fa.decode_prefix(q, None, kp, k, k, n)
    with pytest.raises(ValueError, match="go with"):
        fa.decode_prefix(q, None, None, k, k, n, prefix_len=n[:1])
    with pytest.raises(ValueError, match="prefix_len"):
        fa.decode_prefix(q, kp, kp, k, k, n, prefix_len=n)
    with pytest.raises(ValueError, match="seqlens"):
        fa.decode_prefix(q, kp, kp, k, k, n.long())
    with pytest.raises(fa.FaError) as e:
        fa.decode_prefix(q, kp, kp, k, k, n, workspace=torch.empty(1024, dtype=torch.uint8, device="cuda"))
    assert e.value.status == WORKSPACE
