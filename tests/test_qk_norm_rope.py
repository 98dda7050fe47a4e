"""fa_qk_norm_rope, its gradient and its cache form against the plain fp64 forms."""
from __future__ import annotations

import pytest
import torch

from tests.tree_reference import (F64, check_close, norm_rope, norm_rope_bound, norm_rope_bwd, paths,
                                  random_parents)

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16 = torch.bfloat16


def fa():
    import exact_tiled_attention_fa_gb300 as m
    return m


def tables(max_pos, rot):
    a = torch.arange(max_pos, dtype=F64)[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, dtype=F64) / rot)
    return a.cos().float(), a.sin().float()


def make(B, N, Hq, Hkv, d, rot, packed, seed, w_dtype=BF16, extra=8):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((B, N, Hq + 2 * Hkv, d), generator=g).to(BF16)
    q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
    if not packed:
        q, k, v = (t.contiguous() for t in (q, k, v))
    w = [(1 + 0.3 * torch.randn(d, generator=g)).to(w_dtype) for _ in range(2)]
    cos, sin = tables(N + extra, rot)
    pos = torch.randint(0, N + extra, (B, N), generator=g).to(torch.int32)
    return q, k, v, w, cos, sin, pos


def dev(*ts):
    """On the GPU with strides kept (slices of one projection stay slices)."""
    out, base = [], {}
    for t in ts:
        if t is None or t._base is None:
            out.append(None if t is None else t.to(DEV))
            continue
        b = base.setdefault(id(t._base), t._base.to(DEV))
        out.append(b.as_strided(t.shape, t.stride(), t.storage_offset()))
    return out


SHAPES = [(1, 1, 1, 1, 32, 32), (2, 7, 5, 5, 64, 64), (3, 33, 6, 2, 128, 128), (1, 130, 16, 4, 128, 96), (2, 9, 7, 1, 32, 16),
          (2, 50, 12, 3, 64, 48), (40, 3, 3, 3, 128, 16)]


@pytest.mark.parametrize("B,N,Hq,Hkv,d,rot", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("expand,packed,w_dtype", [(False, False, BF16), (True, True, torch.float32)])
def test_forward(B, N, Hq, Hkv, d, rot, interleaved, expand, packed, w_dtype):
    q, k, v, w, cos, sin, pos = make(B, N, Hq, Hkv, d, rot, packed, N + d, w_dtype)
    gq, gk, gv = dev(q, k, v)
    for p in (pos, None):
        got = fa().qk_norm_rope(gq, gk, gv, w[0].to(DEV), w[1].to(DEV), cos.to(DEV), sin.to(DEV),
                                positions=None if p is None else p.to(DEV), interleaved=interleaved, expand=expand)
        at = (p if p is not None else torch.arange(N).repeat(B, 1)).long()
        c, s = cos.to(F64)[at], sin.to(F64)[at]
        rep = Hq // Hkv if expand else 1
        for t, x, wt, r, name in ((got[0], q, w[0], 1, "q"), (got[1], k, w[1], rep, "k")):
            a = (x.to(F64), wt.to(F64), c, s, 1e-6, interleaved)
            y, b = (z.transpose(1, 2).repeat_interleave(r, 1) for z in (norm_rope(*a), norm_rope_bound(*a)))
            assert t.shape == y.shape and t.is_contiguous()
            check_close(t, y, b, name + " bf16")
        assert torch.equal(got[2].cpu(), v.transpose(1, 2).repeat_interleave(rep, 1))
    assert fa().get_device_error() == 0


def test_forward_extremes():
    """Zero rows (eps alone), rows of the largest and the smallest values, no values to carry, eps = 0."""
    q, k, _, w, cos, sin, _ = make(1, 6, 2, 2, 64, 64, False, 1)
    q[0, 0], q[0, 1], q[0, 2], k[0, 3] = 0, 1e18, 1e-18, 1e-30
    got = fa().qk_norm_rope(*dev(q, k), None, w[0].to(DEV), w[1].to(DEV), cos.to(DEV), sin.to(DEV))
    assert got[2] is None
    c, s = cos[:6].to(F64)[None], sin[:6].to(F64)[None]
    for t, x, wt in ((got[0], q, w[0]), (got[1], k, w[1])):
        a = (x.to(F64), wt.to(F64), c, s, 1e-6, False)
        check_close(t, norm_rope(*a).transpose(1, 2), norm_rope_bound(*a).transpose(1, 2), "extremes bf16")
    q[0, 0], q[0, 2], k[0, 3] = 1, 1e-3, 1e-4
    got = fa().qk_norm_rope(*dev(q, k), None, w[0].to(DEV), w[1].to(DEV), cos.to(DEV), sin.to(DEV), eps=0.0)
    a = (q.to(F64), w[0].to(F64), c, s, 0.0, False)
    check_close(got[0], norm_rope(*a).transpose(1, 2), norm_rope_bound(*a).transpose(1, 2), "eps 0 bf16")


@pytest.mark.parametrize("B,N,Hq,Hkv,d,rot", SHAPES)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("expand,packed,g_dtype,out_dtype", [(False, False, BF16, BF16), (True, True, torch.float32, torch.float32),
                                                             (True, False, BF16, torch.float32)])
def test_backward(B, N, Hq, Hkv, d, rot, interleaved, expand, packed, g_dtype, out_dtype):
    q, k, v, w, cos, sin, pos = make(B, N, Hq, Hkv, d, rot, packed, N + d + 1)
    rep = Hq // Hkv if expand else 1
    g = torch.Generator().manual_seed(7)
    dq, dk, dv = (torch.randn((B, h, N, d), generator=g).to(g_dtype) for h in (Hq, Hkv * rep, Hkv * rep))
    gq, gk = dev(q, k)
    grads = None
    if packed:  # into slices of one buffer, as the projection's gradient wants them
        buf = torch.full((B, N, Hq + 2 * Hkv, d), float("nan"), dtype=out_dtype, device=DEV)
        grads = (buf[:, :, :Hq], buf[:, :, Hq:Hq + Hkv], buf[:, :, Hq + Hkv:])
    args = (dq.to(DEV), dk.to(DEV), dv.to(DEV), gq, gk, w[0].to(DEV), w[1].to(DEV), cos.to(DEV), sin.to(DEV))
    kw = dict(positions=pos.to(DEV), interleaved=interleaved, expand=expand, out_dtype=out_dtype, grads=grads)
    got = fa().qk_norm_rope_bwd(*args, **kw)
    again = [t.clone() for t in got]
    got = fa().qk_norm_rope_bwd(*args, **kw)
    assert all(torch.equal(a, b) for a, b in zip(got, again))
    c, s = cos.to(F64)[pos.long()], sin.to(F64)[pos.long()]
    kind = " bf16" if out_dtype == BF16 else " fp32"
    shared = lambda t: t.to(F64).unflatten(1, (Hkv, rep)).sum(2).transpose(1, 2)  # noqa: E731
    for t, tw, x, wt, gr, name in ((got[0], got[3], q, w[0], dq.to(F64).transpose(1, 2), "q"),
                                   (got[1], got[4], k, w[1], shared(dk), "k")):
        dx, dw, bx, bw = norm_rope_bwd(gr, x.to(F64), wt.to(F64), c, s, 1e-6, interleaved)
        check_close(t, dx, bx, name + kind)
        check_close(tw, dw, bw, name + " weight fp32")
    # the sum over rep fp32 additions of the copies
    check_close(got[2], shared(dv), rep * 2.0 ** -24 * shared(dv.abs()), "v" + kind)
    assert fa().get_device_error() == 0


def test_backward_against_differences():
    """The slope along a direction, from the fp64 definition at two points, equals the gradients' share in it.

    With step h the difference is off by h^2 times a third derivative of order one per element; the fp32
    gradients by 2^-14 of their magnitudes (two of the bounds above)."""
    B, N, Hq, Hkv, d, rot = 2, 9, 4, 2, 64, 32
    q, k, v, w, cos, sin, pos = make(B, N, Hq, Hkv, d, rot, False, 3, torch.float32)
    g = torch.Generator().manual_seed(11)
    dq, dk, dv = (torch.randn((B, Hq, N, d), generator=g) for _ in range(3))
    got = [t.cpu().to(F64) for t in fa().qk_norm_rope_bwd(
        dq.to(DEV), dk.to(DEV), dv.to(DEV), q.to(DEV), k.to(DEV), w[0].to(DEV), w[1].to(DEV), cos.to(DEV), sin.to(DEV),
        positions=pos.to(DEV), expand=True, out_dtype=torch.float32)]
    c, s = cos.to(F64)[pos.long()], sin.to(F64)[pos.long()]
    x = [t.to(F64) for t in (q, k, v, w[0], w[1])]

    def loss(y):
        oq = norm_rope(y[0], y[3], c, s, 1e-6, False).transpose(1, 2)
        ok = norm_rope(y[1], y[4], c, s, 1e-6, False).transpose(1, 2).repeat_interleave(2, 1)
        ov = y[2].transpose(1, 2).repeat_interleave(2, 1)
        return (oq * dq).sum() + (ok * dk).sum() + (ov * dv).sum()

    h = 1e-4
    for i in range(5):
        u = torch.randn(x[i].shape, generator=g).to(F64)
        slope = (loss([t + h * u if j == i else t for j, t in enumerate(x)])
                 - loss([t - h * u if j == i else t for j, t in enumerate(x)])) / (2 * h)
        mine = (got[i] * u).sum()
        assert abs(float(mine - slope)) <= 2.0 ** -14 * float((got[i] * u).abs().sum()) + 100 * h * h * u.numel()


@pytest.mark.parametrize("B,T,Hq,Hkv,d,rot", [(3, 1, 4, 4, 64, 64), (4, 9, 6, 2, 128, 128), (2, 128, 8, 1, 32, 16), (1, 40, 2, 2, 128, 32),
                                              (200, 2, 3, 1, 64, 48)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tree", [False, True])
def test_append(B, T, Hq, Hkv, d, rot, interleaved, tree):
    q, k, v, w, cos, sin, _ = make(B, T, Hq, Hkv, d, rot, True, T + d, extra=200)
    Nk = 150 + T
    g = torch.Generator().manual_seed(T)
    lens = torch.randint(0, 150, (B,), generator=g).to(torch.int32)
    lens[0] = 150  # the last row of the cache is written
    cnt = torch.randint(0, T + 1, (B,), generator=g).to(torch.int32) if tree else None
    par = random_parents(B, T, T) if tree else None
    if tree:
        cnt[0] = T
    kc, vc = (torch.randn((B, Hkv, Nk, d), generator=g).to(BF16).to(DEV) for _ in range(2))
    kc0, vc0 = kc.cpu(), vc.cpu()
    qo = fa().qk_norm_rope_append(*dev(q, k, v), w[0].to(DEV), w[1].to(DEV), cos.to(DEV), sin.to(DEV), kc, vc, lens.to(DEV),
                                  parents=par.to(DEV) if tree else None, n_nodes=cnt.to(DEV) if tree else None,
                                  interleaved=interleaved)
    kc, vc, qo = kc.cpu(), vc.cpu(), qo.cpu()
    assert fa().get_device_error() == 0
    for b in range(B):
        at, n = int(lens[b]), int(cnt[b]) if tree else T
        assert torch.all(qo[b, :, n:] == 0)
        assert torch.equal(kc[b, :, :at], kc0[b, :, :at]) and torch.equal(kc[b, :, at + n:], kc0[b, :, at + n:])
        assert torch.equal(vc[b, :, :at], vc0[b, :, :at]) and torch.equal(vc[b, :, at + n:], vc0[b, :, at + n:])
        if n == 0:
            continue
        pos = torch.tensor([[at + len(p) - 1 for p in paths(par[b] if tree else None, n)]])
        c, s = cos.to(F64)[pos], sin.to(F64)[pos]
        for t, x, wt in ((qo[b, :, :n], q, w[0]), (kc[b, :, at:at + n], k, w[1])):
            a = (x[b:b + 1, :n].to(F64), wt.to(F64), c, s, 1e-6, interleaved)
            check_close(t, norm_rope(*a)[0].transpose(0, 1), norm_rope_bound(*a)[0].transpose(0, 1), "append bf16")
        assert torch.equal(vc[b, :, at:at + n], v[b, :n].transpose(0, 1))


def test_append_records_bad_lengths():
    """A length out of range, a tree that does not fit, a bad parent and a position past the tables are
    recorded; nothing outside the cache rows of the sequence is written."""
    B, T, H, d = 4, 6, 2, 64
    q, k, v, w, cos, sin, _ = make(B, T, H, H, d, 64, False, 2, extra=300)
    kc = torch.zeros((B + 2, H, 50, d), dtype=BF16, device=DEV)
    vc = torch.zeros_like(kc)
    args = (*dev(q, k, v), w[0].to(DEV), w[1].to(DEV), cos.to(DEV), sin.to(DEV), kc[1:-1], vc[1:-1])
    fa().qk_norm_rope_append(*args, torch.tensor([-3, 48, 99, 44], dtype=torch.int32, device=DEV))
    assert fa().get_device_error() == fa().FA_ERR_INVALID_ARG and fa().get_device_error() == 0
    used = (vc != 0).any(-1).any(1).cpu()  # [B + 2, rows]
    want = torch.zeros((B + 2, 50), dtype=torch.bool)
    want[1, :6] = want[2, 48:] = want[4, 44:] = True
    assert torch.equal(used, want)
    ok = torch.zeros(B, dtype=torch.int32, device=DEV)
    par = torch.tensor([[-1, 1, 0, 2, 3, 9]] * B, dtype=torch.int32, device=DEV)
    fa().qk_norm_rope_append(*args, ok, parents=par)
    assert fa().get_device_error() == fa().FA_ERR_INVALID_ARG
    fa().qk_norm_rope_append(*args[:5], cos[:2].to(DEV), sin[:2].to(DEV), *args[7:], ok)
    assert fa().get_device_error() == fa().FA_ERR_INVALID_ARG
    pos = torch.full((B, T), -1, dtype=torch.int32, device=DEV)
    fa().qk_norm_rope(*args[:7], positions=pos)
    assert fa().get_device_error() == fa().FA_ERR_INVALID_ARG and fa().get_device_error() == 0


def test_graph_and_streams():
    q, k, v, w, cos, sin, pos = make(2, 40, 8, 2, 128, 128, False, 4)
    x = dev(q, k, v)
    rest = (w[0].to(DEV), w[1].to(DEV), cos.to(DEV), sin.to(DEV))
    outs = [torch.empty((2, h, 40, 128), dtype=BF16, device=DEV) for h in (8, 2, 2)]
    ws = torch.empty(fa().qk_norm_rope_bwd_workspace_size(128), dtype=torch.uint8, device=DEV)
    fa().qk_norm_rope_bwd(*outs, *x[:2], *rest)  # first-use set-up
    fa().qk_norm_rope(*x, *rest)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa().qk_norm_rope(*x, *rest, q_out=outs[0], k_out=outs[1], v_out=outs[2])
        grads = fa().qk_norm_rope_bwd(*outs, *x[:2], *rest, workspace=ws)
    for t in x:
        t.copy_(torch.randn(t.shape, device=DEV))
    for _ in range(2):
        g.replay()
    want = fa().qk_norm_rope(*x, *rest)
    back = fa().qk_norm_rope_bwd(*want, *x[:2], *rest)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((*outs, *grads), (*want, *back)))
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(4):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(fa().qk_norm_rope_bwd(*want, *x[:2], *rest))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for t in got for a, b in zip(t, back))


@pytest.mark.parametrize("B,T,Hq,Hkv,d", [(64, 64, 32, 8, 128), (200, 40, 9, 3, 64), (3, 9, 5, 5, 32)])
def test_append_uses_nothing_of_absent_nodes(B, T, Hq, Hkv, d):
    """Rows, parents and values of nodes past n_nodes may hold anything; the others come out as they do alone, from
    one warp to a few heads up to one warp to a token."""
    q, k, v, w, cos, sin, _ = make(B, T, Hq, Hkv, d, d, True, B + T, extra=200)
    g = torch.Generator().manual_seed(B)
    cnt = torch.randint(0, T + 1, (B,), generator=g).to(torch.int32)
    lens = torch.randint(0, 100, (B,), generator=g).to(torch.int32)
    par = random_parents(B, T, T)
    rest = (w[0].to(DEV), w[1].to(DEV), cos.to(DEV), sin.to(DEV))
    out = []
    for fill in (0.0, float("nan")):
        gone = torch.arange(T) >= cnt[:, None]
        q._base[gone] = fill
        par[gone] = 0 if fill == 0.0 else 1 << 30
        kc, vc = (torch.zeros((B, Hkv, 100 + T, d), dtype=BF16, device=DEV) for _ in range(2))
        qo = fa().qk_norm_rope_append(*dev(q, k, v), *rest, kc, vc, lens.to(DEV), parents=par.to(DEV), n_nodes=cnt.to(DEV))
        out.append((qo, kc, vc))
    assert all(torch.equal(a, b) for a, b in zip(*out)) and fa().get_device_error() == 0
    assert torch.all(out[0][0].cpu().transpose(1, 2)[gone] == 0)
