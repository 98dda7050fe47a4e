"""Plain fp64 forms of the operators around cached attention, for the tests.

Each returns, beside its values, a bound on what the kernels may be off by, worked out from the
roundings they make (half a step: bf16 2^-8, fp32 2^-24, relative to the value).
"""
from __future__ import annotations

import math

import torch

F64 = torch.float64
HALF_BF16 = 2.0 ** -8
HALF_F32 = 2.0 ** -24


def random_parents(B, T, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.floor(torch.rand((B, T), generator=g) * (torch.arange(T) + 1)) - 1).to(torch.int32)


def paths(parents, n):
    """Each of the first n nodes' path from the root, the node last."""
    out = []
    for t in range(n):
        p = int(parents[t]) if parents is not None else t - 1
        out.append((out[p] if p >= 0 else []) + [t])
    return out


def tree_attention(q, k_cache, v_cache, lens, parents, n_nodes, scale):
    """O, LSE (fp64) and the bounds of |O - O*| before the output's own rounding and of |LSE - LSE*|.

    A weight p of the kernel differs from the exact one by its score's error e (fp32 accumulation of d
    products: at most d 2^-24 sum |q_i k_i|, taken four times over for the tensor core's own order and
    truncation), the exponential's (2^-21) and, in the product alone, its rounding to bf16 (2^-8).  So
    |dO| <= sum p |v| (2^-8 + 2 e + 2^-20) and |dLSE| <= e + 2^-20 (1 + |LSE|).
    """
    B, Hq, T, d = q.shape
    Hkv = k_cache.shape[1]
    R = Hq // Hkv
    O, dO = torch.zeros((B, Hq, T, d), dtype=F64), torch.zeros((B, Hq, T, d), dtype=F64)
    L, dL = torch.full((B, Hq, T), -math.inf, dtype=F64), torch.zeros((B, Hq, T), dtype=F64)
    for b in range(B):
        at, n = int(lens[b]), int(n_nodes[b]) if n_nodes is not None else T
        see = torch.zeros((n, at + n), dtype=torch.bool)
        see[:, :at] = True
        for t, path in enumerate(paths(parents[b] if parents is not None else None, n)):
            see[t, [at + p for p in path]] = True
        if n == 0:
            continue
        k = k_cache[b, :, :at + n].to(F64).repeat_interleave(R, 0)
        v = v_cache[b, :, :at + n].to(F64).repeat_interleave(R, 0)
        x = q[b, :, :n].to(F64)
        s = torch.where(see, x @ k.transpose(1, 2) * scale, -math.inf)
        mag = torch.where(see, x.abs() @ k.abs().transpose(1, 2) * scale, 0.0).amax(-1)
        e = 4 * d * HALF_F32 * mag
        p = torch.softmax(s, -1)
        O[b, :, :n] = p @ torch.where(see.any(0)[None, :, None], v, 0.0)
        dO[b, :, :n] = (p @ v.abs()) * (HALF_BF16 + 2 * e + 2.0 ** -20)[..., None]
        L[b, :, :n] = torch.logsumexp(s, -1)
        dL[b, :, :n] = e + 2.0 ** -20 * (1 + L[b, :, :n].abs())
    return O, L, dO, dL


def check_tree(o, lse, ref, what=""):
    O, L, dO, dL = ref
    a = o.double().cpu()
    bound = dO + (HALF_BF16 * (O.abs() + dO) if o.dtype == torch.bfloat16 else HALF_F32 * O.abs())
    over = (a - O).abs() - bound
    assert not a.isnan().any(), f"{what}: NaN in O"
    assert float(over.max()) <= 0, f"{what}: O exceeds its bound by {float(over.max()):.3e}"
    if lse is not None:
        x = lse.double().cpu()
        assert torch.equal(torch.isneginf(x), torch.isneginf(L)), f"{what}: empty rows disagree"
        f = torch.isfinite(L)
        if f.any():
            over = (x - L).abs()[f] - dL[f]
            assert float(over.max()) <= 0, f"{what}: LSE exceeds its bound by {float(over.max()):.3e}"


def rotate(y, cos, sin, interleaved):
    """y [..., d] rotated by angles with cos, sin [..., rot/2]."""
    rot = 2 * cos.shape[-1]
    y = y.clone()
    ia = torch.arange(0, rot, 2) if interleaved else torch.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    a, b = y[..., ia], y[..., ib]
    y[..., ia] = a * cos - b * sin
    y[..., ib] = a * sin + b * cos
    return y


def norm_rope(x, w, cos, sin, eps, interleaved):
    """x [B, n, H, d], cos and sin [B, n, rot/2], all fp64: the normed and rotated rows."""
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w
    return rotate(y, cos[:, :, None], sin[:, :, None], interleaved)


def norm_rope_bound(x, w, cos, sin, eps, interleaved):
    """|error| of a row before its rounding: the fp32 sum of d <= 128 squares is off by at most 2^-17
    of itself, r by half of that; everything else is a handful of 2^-24: 2^-17 (|a c| + |b s|)."""
    y = x.abs() / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.abs()
    c, s = cos.abs()[:, :, None], sin.abs()[:, :, None]
    return 2.0 ** -17 * torch.maximum(rotate(y, c, -s, interleaved).abs(), rotate(y, c, s, interleaved).abs())


def norm_rope_bwd(g, x, w, cos, sin, eps, interleaved):
    """Gradients (dx, dw) for g [B, n, H, d] and their bounds before dx's rounding.  Each term of dx
    carries the errors above twice (r, and the second row sum): 2^-15 of the terms' magnitudes; dw is a
    sum of such terms, added in chains of at most 2^8 fp32 additions: 2^-15 of the magnitudes again."""
    h = rotate(g, cos[:, :, None], -sin[:, :, None], interleaved)
    c, s = cos.abs()[:, :, None], sin.abs()[:, :, None]
    hm = torch.maximum(rotate(g.abs(), c, -s, interleaved).abs(), rotate(g.abs(), c, s, interleaved).abs())
    r = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    xh = x * r
    z = w * h
    dx = r * (z - xh * (xh * z).mean(-1, keepdim=True))
    zm = w.abs() * hm
    bx = 2.0 ** -15 * r * (zm + xh.abs() * (xh.abs() * zm).mean(-1, keepdim=True))
    return dx, (h * xh).sum((0, 1, 2)), bx, 2.0 ** -15 * (hm * xh.abs()).sum((0, 1, 2))


def check_close(a, ref, bound, what=""):
    a = a.double().cpu()
    half = HALF_BF16 if what.endswith("bf16") else HALF_F32
    over = (a - ref).abs() - bound - half * (ref.abs() + bound)
    assert not a.isnan().any(), f"{what}: NaN"
    assert float(over.max()) <= 0, f"{what}: exceeds its bound by {float(over.max()):.3e}"
