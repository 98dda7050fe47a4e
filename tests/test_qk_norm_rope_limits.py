"""Norm and rotation at the ends of their ranges: eps = 0."""
from __future__ import annotations

import pytest
import torch

from tests.test_qk_norm_rope import BF16, DEV, SHAPES, dev, fa, make
from tests.tree_reference import F64, check_close, norm_rope_bwd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,N,Hq,Hkv,d,rot", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("expand,g_dtype", [(False, BF16), (True, BF16), (False, torch.float32), (True, torch.float32)])
@pytest.mark.parametrize("eps", [0.0, 1e-46])
def test_backward_without_eps(B, N, Hq, Hkv, d, rot, interleaved, expand, g_dtype, eps):
    """eps = 0, and one that is 0 in fp32, with head counts that leave lanes without a row: their zeros have no
    norm, and must not reach the weights' gradients."""
    q, k, v, w, cos, sin, pos = make(B, N, Hq, Hkv, d, rot, True, N + d + 2)
    rep = Hq // Hkv if expand else 1
    g = torch.Generator().manual_seed(8)
    dq, dk, dv = (torch.randn((B, h, N, d), generator=g).to(g_dtype) for h in (Hq, Hkv * rep, Hkv * rep))
    got = fa().qk_norm_rope_bwd(dq.to(DEV), dk.to(DEV), dv.to(DEV), *dev(q, k), w[0].to(DEV), w[1].to(DEV), cos.to(DEV), sin.to(DEV),
                                positions=pos.to(DEV), eps=eps, interleaved=interleaved, expand=expand, out_dtype=g_dtype)
    c, s = cos.to(F64)[pos.long()], sin.to(F64)[pos.long()]
    kind = " bf16" if g_dtype == BF16 else " fp32"
    shared = lambda t: t.to(F64).unflatten(1, (Hkv, rep)).sum(2).transpose(1, 2)  # noqa: E731
    for t, tw, x, wt, gr, name in ((got[0], got[3], q, w[0], dq.to(F64).transpose(1, 2), "q"),
                                   (got[1], got[4], k, w[1], shared(dk), "k")):
        dx, dw, bx, bw = norm_rope_bwd(gr, x.to(F64), wt.to(F64), c, s, 0.0, interleaved)
        check_close(t, dx, bx, name + kind)
        check_close(tw, dw, bw, name + " weight fp32")
    assert fa().get_device_error() == 0
