"""fa_cache_compact against indexing, and a verification step of the operators around a cache together."""
from __future__ import annotations

import math

import pytest
import torch

from tests.tree_reference import check_tree, random_parents, tree_attention

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF16 = torch.bfloat16


def fa():
    import exact_tiled_attention_fa_gb300 as m
    return m


def expected(c, lens, acc, cnt):
    c = c.clone()
    for b in range(lens.numel()):
        at, n = int(lens[b]), int(cnt[b])
        c[:, b, :, at:at + n] = c[:, b, :, [at + int(a) for a in acc[b, :n]]].clone()
    return c


@pytest.mark.parametrize("L,B,H,Nk,d,T", [(1, 1, 1, 1, 32, 1), (1, 3, 2, 140, 128, 128), (4, 5, 3, 77, 64, 16), (2, 300, 1, 20, 32, 7),
                                          (3, 2, 8, 200, 128, 60)])
@pytest.mark.parametrize("order", ["path", "any", "same"])
def test_rows_move(L, B, H, Nk, d, T, order):
    """Increasing nodes, any order, and one node named every time; counts from none to all."""
    g = torch.Generator().manual_seed(B + T)
    k, v = (torch.randn((L, B, H, Nk, d), generator=g).to(BF16) for _ in range(2))
    lens = torch.randint(0, Nk - T + 1, (B,), generator=g).to(torch.int32)
    cnt = torch.randint(0, T + 1, (B,), generator=g).to(torch.int32)
    lens[0], cnt[0] = Nk - T, T
    perm = torch.stack([torch.randperm(T, generator=g) for _ in range(B)])
    acc = {"path": perm, "any": perm, "same": perm[:, :1].expand(B, T)}[order].clone()
    if order == "path":
        for b in range(B):
            acc[b, :int(cnt[b])] = acc[b, :int(cnt[b])].sort()[0]
    acc = acc.to(torch.int32)
    gk, gv = k.to(DEV), v.to(DEV)
    if L == 1:
        gk, gv = gk[0], gv[0]
    out = fa().cache_compact(gk, gv, lens.to(DEV), acc.to(DEV), cnt.to(DEV))
    assert fa().get_device_error() == 0
    assert torch.equal(out.cpu(), lens + cnt)
    assert torch.equal(gk.cpu().view(k.shape), expected(k, lens, acc, cnt))
    assert torch.equal(gv.cpu().view(v.shape), expected(v, lens, acc, cnt))


def test_bad_values_are_recorded():
    """Nodes out of range stay where they are, lengths and counts are clamped, nothing else is touched."""
    g = torch.Generator().manual_seed(0)
    k = torch.randn((1, 6, 2, 30, 32), generator=g).to(BF16)
    lens = torch.tensor([-2, 40, 28, 5, 5, 5], dtype=torch.int32)
    acc = torch.tensor([[1, 0, 3, 2]] * 6, dtype=torch.int32)
    acc[3] = torch.tensor([2, -1, 4, 1])
    cnt = torch.tensor([1, 2, 4, 3, 9, -1], dtype=torch.int32)
    gk, gv = k[0].to(DEV), k[0].to(DEV)
    out = fa().cache_compact(gk, gv, lens.to(DEV), acc.to(DEV), cnt.to(DEV))
    assert fa().get_device_error() == fa().FA_ERR_INVALID_ARG and fa().get_device_error() == 0
    assert out.tolist() == [1, 30, 30, 8, 9, 5]
    want = k[0].clone()
    want[0, :, 0] = k[0, 0, :, 1]                       # length 0
    want[2, :, 28], want[2, :, 29] = k[0, 2, :, 29], k[0, 2, :, 28]  # two rows left in the cache
    want[3, :, 5] = k[0, 3, :, 7]                       # nodes -1 and 4 of 4 are not moved
    want[4, :, 5:9] = k[0, 4, :, [6, 5, 8, 7]]          # 4 of 4
    assert torch.equal(gk.cpu(), want) and torch.equal(gv.cpu(), want)


def test_lengths_in_place_are_refused():
    k = torch.zeros((2, 1, 8, 32), dtype=BF16, device=DEV)
    n = torch.zeros(4, dtype=torch.int32, device=DEV)
    acc = torch.zeros((2, 3), dtype=torch.int32, device=DEV)
    for out in (n[:2], n[1:3]):
        with pytest.raises(fa().FaError, match="invalid"):
            fa().cache_compact(k, k.clone(), n[:2], acc, n[2:], seqlens_out=out)
    fa().cache_compact(k, k.clone(), n[:2], acc, n[2:], seqlens_out=torch.empty(2, dtype=torch.int32, device=DEV))


def test_graph():
    k, v = (torch.randn((2, 3, 2, 40, 64), device=DEV).to(BF16) for _ in range(2))
    lens = torch.tensor([3, 0, 30], dtype=torch.int32, device=DEV)
    acc = torch.tensor([[0, 2, 4, 0, 0]] * 3, dtype=torch.int32, device=DEV)
    cnt = torch.tensor([3, 2, 1], dtype=torch.int32, device=DEV)
    out = torch.empty_like(lens)
    fa().cache_compact(k.clone(), v.clone(), lens, acc, cnt)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa().cache_compact(k, v, lens, acc, cnt, seqlens_out=out)
    acc.copy_(torch.tensor([[1, 3, 4, 0, 0], [2, 3, 0, 0, 0], [4, 0, 0, 0, 0]]))
    k0, v0 = k.cpu(), v.cpu()
    g.replay()
    torch.cuda.synchronize()
    args = (lens.cpu(), acc.cpu(), cnt.cpu())
    assert torch.equal(k.cpu(), expected(k0, *args)) and torch.equal(v.cpu(), expected(v0, *args))
    assert torch.equal(out, lens + cnt)


def test_verification_steps_together():
    """Prefill by the forward, then two rounds of: append a tree, attend, keep a path, drop the rest.  At the end
    the cache holds exactly what appending the kept tokens one after another would have put there, and a plain
    grouped decode over it agrees with the tree's own rows."""
    B, Hq, Hkv, d, T, N, Nk = 3, 8, 2, 128, 10, 37, 80
    g = torch.Generator().manual_seed(1)
    mk = lambda *s: torch.randn(s, generator=g).to(BF16).to(DEV)  # noqa: E731
    wq, wk = mk(d), mk(d)
    a = torch.arange(200, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    cos, sin = a.cos().float().to(DEV), a.sin().float().to(DEV)
    rest = (wq, wk, cos, sin)
    x = mk(B, N, Hq + 2 * Hkv, d)
    parts = lambda t: (t[:, :, :Hq], t[:, :, Hq:Hq + Hkv], t[:, :, Hq + Hkv:])  # noqa: E731
    q, k, v = fa().qk_norm_rope(*parts(x), *rest, expand=True)
    o, _ = fa().fwd(q, k, v, causal=True)
    _, k1, v1 = fa().qk_norm_rope(*parts(x), *rest)
    kc, vc = (torch.full((B, Hkv, Nk, d), float("nan"), dtype=BF16, device=DEV) for _ in range(2))
    kc[:, :, :N], vc[:, :, :N] = k1, v1
    line_k, line_v = kc.clone(), vc.clone()  # the same sequence token by token
    # the last prompt token again, as a chain of one over the others: the forward's last row
    lens = torch.full((B,), N - 1, dtype=torch.int32, device=DEV)
    q1 = fa().qk_norm_rope_append(*(t[:, -1:].contiguous() for t in parts(x)), *rest, kc, vc, lens)
    o1, _ = fa().decode_tree(q1, kc, vc, lens)
    assert torch.equal(kc[:, :, :N], line_k[:, :, :N]) and torch.equal(q1[:, :, 0], q[:, :, -1])
    # both within 2^-8 (weights) + 2^-8 (output) of the exact value: |O| <= max |v| row-wise mean
    assert float((o1[:, :, 0] - o[:, :, -1]).abs().max()) <= 4 * 2.0 ** -8 * float(v.abs().max())
    lens += 1
    for step in range(2):
        par = random_parents(B, T, step)
        cnt = torch.tensor([T, 1, 6], dtype=torch.int32)
        y = mk(B, T, Hq + 2 * Hkv, d)
        qt = fa().qk_norm_rope_append(*parts(y), *rest, kc, vc, lens, parents=par.to(DEV), n_nodes=cnt.to(DEV))
        ot, lt = fa().decode_tree(qt, kc, vc, lens, parents=par.to(DEV), n_nodes=cnt.to(DEV), out_dtype=torch.float32)
        check_tree(ot, lt, tree_attention(qt.cpu(), kc.cpu(), vc.cpu(), lens.cpu(), par, cnt, 1 / math.sqrt(d)), f"step {step}")
        acc = torch.zeros((B, T), dtype=torch.int32)
        kept = torch.zeros(B, dtype=torch.int32)
        for b in range(B):
            path, t = [], int(cnt[b]) - 1
            while t >= 0:
                path.append(t)
                t = int(par[b, t])
            acc[b, :len(path)], kept[b] = torch.tensor(path[::-1]), len(path)
        new = fa().cache_compact(kc, vc, lens, acc.to(DEV), kept.to(DEV))
        for b in range(B):  # the kept tokens one by one
            for i in range(int(kept[b])):
                tok = [t[b:b + 1, int(acc[b, i]):int(acc[b, i]) + 1].contiguous() for t in parts(y)]
                fa().qk_norm_rope_append(*tok, *rest, line_k[b:b + 1], line_v[b:b + 1], (lens[b:b + 1] + i).contiguous())
            n = int(new[b])
            assert torch.equal(kc[b, :, :n], line_k[b, :, :n]) and torch.equal(vc[b, :, :n], line_v[b, :, :n])
            leaf = qt[b:b + 1, :, int(acc[b, int(kept[b]) - 1])][:, :, None].contiguous()
            og, lg = fa().decode_splitkv_gqa(leaf, kc[b:b + 1], vc[b:b + 1], new[b:b + 1].contiguous(), out_dtype=torch.float32)
            check_tree(og, lg, tree_attention(leaf.cpu(), kc[b:b + 1].cpu(), vc[b:b + 1].cpu(), [n - 1], None, None,
                                              1 / math.sqrt(d)), "leaf")
        lens = new
    assert fa().get_device_error() == 0


def test_rows_past_32_bit_offsets():
    """A cache of more than 2^31 elements: the last rows are appended, attended to and moved.  Every key but the
    appended ones is 0 (score 0, weight 1), every value 0; the appended keys are long enough to carry most of
    the weight."""
    Hq, d, T, Nk = 2, 128, 4, (1 << 24) + 40
    g = torch.Generator().manual_seed(3)
    kc, vc = (torch.zeros((1, 1, Nk, d), dtype=BF16, device=DEV) for _ in range(2))
    at = Nk - 9
    lens = torch.tensor([at], dtype=torch.int32, device=DEV)
    x = torch.randn((1, T, Hq + 2, d), generator=g).to(BF16)
    par = torch.tensor([[-1, 0, 0, 2]], dtype=torch.int32, device=DEV)
    ones = torch.full((d,), 1.5, dtype=torch.float32, device=DEV)
    cos, sin = torch.ones((Nk, 8), device=DEV), torch.zeros((Nk, 8), device=DEV)
    gx = x.to(DEV)
    q = fa().qk_norm_rope_append(gx[:, :, :Hq], gx[:, :, Hq:Hq + 1], gx[:, :, Hq + 1:], ones, ones, cos, sin, kc, vc, lens, parents=par)
    assert int((kc != 0).any(-1).sum()) == T and int((vc != 0).any(-1).sum()) == T
    k, v = kc[0, 0, at:at + T].double().cpu(), vc[0, 0, at:at + T].double().cpu()
    assert torch.equal(v, x[0, :, Hq + 1].double())
    scale = 2.0
    o, lse = fa().decode_tree(q, kc, vc, lens, parents=par, scale=scale, out_dtype=torch.float32)
    see = torch.tensor([[1, 0, 0, 0], [1, 1, 0, 0], [1, 0, 1, 0], [1, 0, 1, 1]], dtype=torch.bool)
    s = torch.where(see, q[0].double().cpu() @ k.T * scale, -math.inf)
    L = torch.logsumexp(torch.cat((s, torch.full((Hq, T, 1), math.log(at), dtype=torch.float64)), -1), -1)
    O = torch.exp(s - L[..., None]) @ v
    # scores: 4 d 2^-24 of |q||k| scale; weights 2^-8 more; 2^17 tiles' sums of equal terms are exact in fp32 (weights
    # of 1 in up to 2^24 of them, split over the shares), then at most 2^9 additions of the parts
    e = 4 * d * 2.0 ** -24 * float((q[0].double().cpu().abs() @ k.abs().T).max()) * scale
    bound = (torch.exp(s - L[..., None]) @ v.abs()) * (2.0 ** -8 + 2 * e + 2.0 ** -14)
    assert float(((o[0].double().cpu() - O).abs() - bound).max()) <= 0
    assert float((lse[0].double().cpu() - L).abs().max()) <= e + 2.0 ** -14
    keep = torch.tensor([[0, 2, 3, 0]], dtype=torch.int32, device=DEV)
    n = fa().cache_compact(kc, vc, lens, keep, torch.tensor([3], dtype=torch.int32, device=DEV))
    assert n.tolist() == [at + 3] and torch.equal(kc[0, 0, at:at + 4].double().cpu(), k[[0, 2, 3, 3]])
    assert torch.equal(vc[0, 0, at:at + 4].double().cpu(), v[[0, 2, 3, 3]])
    assert fa().get_device_error() == 0


def test_training_step_together():
    """qk_norm_rope -> fwd -> bwd -> qk_norm_rope_bwd with shared heads: the gradients of the packed projection
    against fp64 differentiation of the whole.  bwd's gradients carry bf16 operands (P, dS and dO rounded: three
    relative 2^-8 on sums of N terms, and its own bf16 outputs): 2^-5 of the gradients' root mean square."""
    B, N, Hq, Hkv, d = 2, 130, 4, 2, 64
    g = torch.Generator().manual_seed(5)
    x = torch.randn((B, N, Hq + 2 * Hkv, d), generator=g).to(BF16)
    w = [(1 + 0.2 * torch.randn(d, generator=g)).to(BF16) for _ in range(2)]
    a = torch.arange(N, dtype=torch.float64)[:, None] * 10000.0 ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    cos, sin = a.cos().float(), a.sin().float()
    do = torch.randn((B, Hq, N, d), generator=g).to(BF16)
    gx = x.to(DEV)
    parts = lambda t: (t[:, :, :Hq], t[:, :, Hq:Hq + Hkv], t[:, :, Hq + Hkv:])  # noqa: E731
    rest = (w[0].to(DEV), w[1].to(DEV), cos.to(DEV), sin.to(DEV))
    q, k, v = fa().qk_norm_rope(*parts(gx), *rest, expand=True)
    o, lse = fa().fwd(q, k, v, causal=True)
    dq, dk, dv = fa().bwd(q, k, v, o, lse, do.to(DEV), causal=True)
    buf = torch.empty_like(gx)
    *_, gwq, gwk = fa().qk_norm_rope_bwd(dq, dk, dv, *parts(gx)[:2], *rest, expand=True, grads=parts(buf))
    from tests.tree_reference import norm_rope
    X = x.double().requires_grad_()
    W = [t.double().requires_grad_() for t in w]
    c, s = cos.double()[None].expand(B, -1, -1), sin.double()[None].expand(B, -1, -1)
    Q, K, V = parts(X)
    Q = norm_rope(Q, W[0], c, s, 1e-6, False).transpose(1, 2)
    K = norm_rope(K, W[1], c, s, 1e-6, False).transpose(1, 2).repeat_interleave(2, 1)
    V = V.transpose(1, 2).repeat_interleave(2, 1)
    S = (Q @ K.transpose(2, 3) / 8).masked_fill(torch.ones(N, N, dtype=torch.bool).triu(1), -math.inf)
    (torch.softmax(S, -1) @ V * do.double()).sum().backward()
    for mine, ref in ((buf, X.grad), (gwq, W[0].grad), (gwk, W[1].grad)):
        err = (mine.double().cpu() - ref)
        assert float(err.norm() / ref.norm()) <= 2.0 ** -5
