"""Norm and rotation at the ends of their ranges: eps = 0, rows whose sum of squares overflows."""
from __future__ import annotations

import pytest
import torch

from tests.test_qk_norm_rope import BF16, DEV, SHAPES, dev, fa, make
from tests.tree_reference import F64, check_close, norm_rope, norm_rope_bound, norm_rope_bwd

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


HUGE = torch.finfo(BF16).max


def overflowing(d, seed):
    """q, k, v and the others of two sequences of 9 tokens with rows of the largest values among them, weights that
    overflow with those; which rows [B, N, heads] of q and of k they are."""
    q, k, v, w, cos, sin, pos = make(2, 9, 3, 3, d, d, False, seed, torch.float32)
    sign = torch.where(torch.arange(d) % 2 == 0, 1.0, -1.0).to(BF16)
    q[0, 0, 0], q[0, 1, 1], k[1, 8, 2] = HUGE, HUGE * sign, -HUGE
    q[0, 2, 2, 5], k[0, 3, 0, d - 1], k[1, 0, 1] = HUGE, -HUGE, 2.0 ** 64  # one element of a row; 2^128 already overflows
    w = [t.abs().clamp_min(0.5) * 2 for t in w]
    return q, k, v, w, cos, sin, pos, [(x.to(F64).square().sum(-1) >= 2.0 ** 127) for x in (q, k)]


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("form", ["prompt", "append"])
def test_overflowing_rows_are_zero(d, interleaved, form):
    """A row whose sum of squares is past fp32 is written as 0, also where the row times its weights is past fp32
    itself; the others are right."""
    q, k, v, w, cos, sin, pos, big = overflowing(d, d)
    rest = (*dev(q, k, v), w[0].to(DEV), w[1].to(DEV), cos.to(DEV), sin.to(DEV))
    if form == "prompt":
        got = fa().qk_norm_rope(*rest, positions=pos.to(DEV), interleaved=interleaved)[:2]
    else:
        kc, vc = (torch.zeros((2, 3, 9, d), dtype=BF16, device=DEV) for _ in range(2))
        pos = torch.arange(9).repeat(2, 1)
        got = fa().qk_norm_rope_append(*rest, kc, vc, torch.zeros(2, dtype=torch.int32, device=DEV), interleaved=interleaved), kc
    c, s = cos.to(F64)[pos.long()], sin.to(F64)[pos.long()]
    assert big[0].sum() == 3 and big[1].sum() == 3
    for t, x, wt, b in ((got[0], q, w[0], big[0]), (got[1], k, w[1], big[1])):
        x = torch.where(b[..., None], 0.0, x.to(F64))
        a = (x, wt.to(F64), c, s, 1e-6, interleaved)
        assert torch.all(t.cpu().transpose(1, 2)[b] == 0)
        check_close(t, norm_rope(*a).transpose(1, 2), norm_rope_bound(*a).transpose(1, 2), "beside large rows bf16")


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("copies", [1, 2])
@pytest.mark.parametrize("g_dtype", [BF16, torch.float32])
def test_overflowing_rows_have_no_gradient(d, copies, g_dtype):
    """Such a row is 0 whatever it holds: its gradient is 0 and it adds nothing to the weights'."""
    q, k, v, w, cos, sin, pos, big = overflowing(d, d + 1)
    if copies > 1:
        q = torch.cat((q, q.flip(2)), 2)
        big[0] = torch.cat((big[0], big[0].flip(2)), 2)
    g = torch.Generator().manual_seed(4)
    dq, dk, dv = (torch.randn((2, 3 * copies, 9, d), generator=g).to(g_dtype) for _ in range(3))
    got = fa().qk_norm_rope_bwd(dq.to(DEV), dk.to(DEV), dv.to(DEV), *dev(q, k), w[0].to(DEV), w[1].to(DEV), cos.to(DEV), sin.to(DEV),
                                positions=pos.to(DEV), expand=True, out_dtype=g_dtype)
    c, s = cos.to(F64)[pos.long()], sin.to(F64)[pos.long()]
    kind = " bf16" if g_dtype == BF16 else " fp32"
    shared = lambda t: t.to(F64).unflatten(1, (3, copies)).sum(2).transpose(1, 2)  # noqa: E731
    for t, tw, x, wt, gr, b in ((got[0], got[3], q, w[0], dq.to(F64).transpose(1, 2), big[0]),
                                (got[1], got[4], k, w[1], shared(dk), big[1])):
        gr, x = torch.where(b[..., None], 0.0, gr), torch.where(b[..., None], 1.0, x.to(F64))
        dx, dw, bx, bw = norm_rope_bwd(gr, x, wt.to(F64), c, s, 1e-6, False)
        assert torch.all(t.cpu()[b] == 0)
        check_close(t, dx, bx, "beside large rows" + kind)
        check_close(tw, dw, bw, "weights beside large rows fp32")
