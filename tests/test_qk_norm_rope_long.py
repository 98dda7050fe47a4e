"""Norm and rotation of many tokens: a warp walks several steps of a token (forward), several tokens (gradient), and
offsets pass 32 bits.  The plain fp64 forms run on the GPU."""
from __future__ import annotations

import pytest
import torch

from tests.test_qk_norm_rope import BF16, DEV, fa, tables
from tests.tree_reference import F64, HALF_BF16, HALF_F32, norm_rope, norm_rope_bound, norm_rope_bwd, paths, random_parents

pytestmark = pytest.mark.gpu


def inputs(B, N, Hq, Hkv, d, rot, seed, extra=50):
    """One projection's q, k, v on the GPU, weights, tables, positions."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn((B, N, Hq + 2 * Hkv, d), generator=g, device=DEV).to(BF16)
    w = [(1 + 0.3 * torch.randn(d, generator=g, device=DEV)).to(BF16) for _ in range(2)]
    cos, sin = (t.to(DEV) for t in tables(N + extra, rot))
    pos = torch.randint(0, N + extra, (B, N), generator=g, device=DEV).to(torch.int32)
    return x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:], w, cos, sin, pos


def close(a, ref, bound, half, what):
    a = a.to(F64)
    assert not a.isnan().any(), what
    over = (a - ref).abs() - bound - half * (ref.abs() + bound)
    assert float(over.max()) <= 0, f"{what}: exceeds its bound by {float(over.max()):.3e}"


def check_forward(got, q, k, v, w, c, s, rep, interleaved):
    for t, x, wt, r, name in ((got[0], q, w[0], 1, "q"), (got[1], k, w[1], rep, "k")):
        a = (x.to(F64), wt.to(F64), c, s, 1e-6, interleaved)
        y, b = (z.transpose(1, 2).repeat_interleave(r, 1) for z in (norm_rope(*a), norm_rope_bound(*a)))
        close(t, y, b, HALF_BF16, name)
    if v is not None:
        assert torch.equal(got[2], v.transpose(1, 2).repeat_interleave(rep, 1))


# tokens such that a warp has all of a token's steps, or a third or so of them
@pytest.mark.parametrize("B,N", [(3, 3333), (1, 2111)])
@pytest.mark.parametrize("Hq,Hkv,d,rot", [(25, 5, 64, 64), (9, 3, 128, 96), (40, 8, 32, 32), (3, 1, 128, 128), (44, 44, 64, 16)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("expand,values", [(False, True), (True, True), (False, False)])
def test_forward_of_many_tokens(B, N, Hq, Hkv, d, rot, interleaved, expand, values):
    q, k, v, w, cos, sin, pos = inputs(B, N, Hq, Hkv, d, rot, N + d)
    got = fa().qk_norm_rope(q, k, v if values else None, *w, cos, sin, positions=pos, interleaved=interleaved, expand=expand)
    assert values or got[2] is None
    c, s = cos.to(F64)[pos.long()], sin.to(F64)[pos.long()]
    check_forward(got, q, k, v if values else None, w, c, s, Hq // Hkv if expand else 1, interleaved)
    assert fa().get_device_error() == 0


@pytest.mark.parametrize("B,T,Hq,Hkv,d,tree", [(64, 64, 32, 8, 128, True), (200, 64, 9, 3, 64, True), (130, 100, 20, 20, 32, False),
                                               (64, 64, 32, 8, 128, False)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_append_of_many_tokens(B, T, Hq, Hkv, d, tree, interleaved):
    q, k, v, w, cos, sin, _ = inputs(B, T, Hq, Hkv, d, d, B, extra=200)
    Nk = T + 130
    g = torch.Generator().manual_seed(T)
    lens = torch.randint(0, 131, (B,), generator=g).to(torch.int32)
    cnt = torch.randint(0, T + 1, (B,), generator=g).to(torch.int32) if tree else torch.full((B,), T, dtype=torch.int32)
    par = random_parents(B, T, T) if tree else None
    kc, vc = (torch.full((B, Hkv, Nk, d), 7.0, dtype=BF16, device=DEV) for _ in range(2))
    qo = fa().qk_norm_rope_append(q, k, v, *w, cos, sin, kc, vc, lens.to(DEV), parents=par.to(DEV) if tree else None,
                                  n_nodes=cnt.to(DEV) if tree else None, interleaved=interleaved)
    assert fa().get_device_error() == 0
    pos = torch.zeros((B, T), dtype=torch.long)
    for b in range(B):
        n = int(cnt[b])
        pos[b, :n] = torch.tensor([int(lens[b]) + len(p) - 1 for p in paths(par[b] if tree else None, n)], dtype=torch.long)
    live = (torch.arange(T) < cnt[:, None]).to(DEV)
    c, s = cos.to(F64)[pos.to(DEV)], sin.to(F64)[pos.to(DEV)]
    bi, t = live.nonzero(as_tuple=True)
    row = lens.to(DEV).long()[bi] + t
    for out, x, wt in ((qo.transpose(1, 2)[bi, t], q, w[0]), (kc[bi, :, row], k, w[1])):
        a = (x.to(F64), wt.to(F64), c, s, 1e-6, interleaved)
        close(out, norm_rope(*a)[bi, t], norm_rope_bound(*a)[bi, t], HALF_BF16, "append")
    assert torch.equal(vc[bi, :, row], v[bi, t]) and torch.all(qo.transpose(1, 2)[~live] == 0)
    rest = torch.ones((B, Nk), dtype=torch.bool, device=DEV)
    rest[bi, row] = False
    assert torch.all(kc.transpose(1, 2)[rest] == 7) and torch.all(vc.transpose(1, 2)[rest] == 7)


@pytest.mark.parametrize("Hq,Hkv,d,rot", [(8, 2, 128, 128), (5, 5, 128, 64), (12, 3, 64, 64), (16, 16, 64, 32), (10, 2, 32, 32),
                                          (24, 24, 32, 16), (1, 1, 64, 64)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("expand,g_dtype,out_dtype,values", [(False, BF16, BF16, True), (True, torch.float32, torch.float32, True),
                                                             (True, BF16, BF16, False), (False, torch.float32, BF16, False)])
def test_gradient_of_many_tokens(Hq, Hkv, d, rot, interleaved, expand, g_dtype, out_dtype, values):
    """6999 tokens: every warp of two CTAs an SM has two or three, each in a new place of every ring; no values.

    A weight's gradient is a sum of chains: a lane's rows (at most 3 tokens x 24 heads), 4 levels of lanes, 8 warps, 10
    partial rows in a slice and 32 slices: far below 2^8 fp32 additions, as the plain form's bound assumes."""
    B, N = 3, 2333
    q, k, _, w, cos, sin, pos = inputs(B, N, Hq, Hkv, d, rot, d + Hq)
    rep = Hq // Hkv if expand else 1
    g = torch.Generator(device=DEV).manual_seed(7)
    dq, dk, dv = (torch.randn((B, h, N, d), generator=g, device=DEV).to(g_dtype) for h in (Hq, Hkv * rep, Hkv * rep))
    got = fa().qk_norm_rope_bwd(dq, dk, dv if values else None, q, k, *w, cos, sin, positions=pos, interleaved=interleaved,
                                expand=expand, out_dtype=out_dtype)
    half = HALF_BF16 if out_dtype == BF16 else HALF_F32
    c, s = cos.to(F64)[pos.long()], sin.to(F64)[pos.long()]
    shared = lambda t: t.to(F64).unflatten(1, (Hkv, rep)).sum(2).transpose(1, 2)  # noqa: E731
    for t, tw, x, wt, gr, name in ((got[0], got[3], q, w[0], dq.to(F64).transpose(1, 2), "q"),
                                   (got[1], got[4], k, w[1], shared(dk), "k")):
        dx, dw, bx, bw = norm_rope_bwd(gr, x.to(F64), wt.to(F64), c, s, 1e-6, interleaved)
        close(t, dx, bx, half, name)
        close(tw, dw, bw, HALF_F32, name + " weight")
    if values:
        close(got[2], shared(dv), rep * HALF_F32 * shared(dv.abs()), half, "v")
    else:
        assert got[2] is None
    assert fa().get_device_error() == 0


def test_offsets_past_32_bits():
    """More than 2^31 elements of queries and of their gradients: the last tokens and heads are those of a call on
    them alone, and the others, spot by spot, too."""
    B, N, Hq, Hkv, d = 2, (1 << 16) + 24, 134, 2, 128
    q, k, v, w, cos, sin, pos = inputs(B, N, Hq, Hkv, d, d, 1, extra=0)
    assert q.numel() > 1 << 31
    out = fa().qk_norm_rope(q, k, v, *w, cos, sin, positions=pos)
    grads = fa().qk_norm_rope_bwd(*out, q, k, *w, cos, sin, positions=pos)
    total = [torch.zeros(d, dtype=F64, device=DEV) for _ in range(2)]
    size = [torch.zeros(d, dtype=F64, device=DEV) for _ in range(2)]
    step = 4096
    for b in range(B):
        for at in range(0, N, step):
            some = slice(at, min(N, at + step))
            part = [t[b:b + 1, some] for t in (q, k, v)]
            p = pos[b:b + 1, some].contiguous()
            o = fa().qk_norm_rope(*part, *w, cos, sin, positions=p)
            assert all(torch.equal(x, y[b:b + 1, :, some]) for x, y in zip(o, out))
            gr = fa().qk_norm_rope_bwd(*o, *part[:2], *w, cos, sin, positions=p)
            assert all(torch.equal(x, y[b:b + 1, some]) for x, y in zip(gr[:3], grads[:3]))
            for i in range(2):
                total[i] += gr[3 + i].to(F64)
                size[i] += gr[3 + i].to(F64).abs()
    # each term of a weight's gradient is h x^, h = x^ w here: all of one sign, so the sum of the parts' sizes is
    # that of the terms' but for the rotation's rounding.  A lane's chain: ceil(131120 / 2432) = 54 tokens x 67 steps,
    # then some 60 additions; the same in the parts.
    for i in range(2):
        assert float(((grads[3 + i].to(F64) - total[i]).abs() - 2 * (54 * 67 + 60) * HALF_F32 * size[i]).max()) <= 0
    assert fa().get_device_error() == 0
