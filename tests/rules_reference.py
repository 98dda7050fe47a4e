"""Plain fp64 forms of attention under score rules, for the tests, with bounds on what the kernels may be off by.

Bounds (half a step: bf16 2^-8, fp32 2^-24, relative to the value).  A score is off by e: the fp32 sum of d
products by at most d 2^-24 sum |q_c k_c| (taken four times over for the tensor core's own order and truncation);
the cap by 2^-21 of the cap (tanh is off by 3e-7 at most); everything that is then done to it in fp32 by 2^-21
of the magnitudes that meet there, |s| and the bias.  A weight is off by its score's error, the weighted mean
E of the row's (that of its log-sum-exp), the exponential's 2^-21 and, in the products alone, its rounding to bf16:
  |dO| <= sum_j p_j |v_j| (2^-8 + e_j + E + 2^-20),  |dLSE| <= E + 2^-20 (1 + |LSE|).
The gradients: the products take P and dX in bf16 (2^-8 each, of M = |A| |B|), and D's error goes with P |dO| (P |V|);
the bound is twice 2^-8 of M, as for the backward without rules, widened by the weights' errors, plus 1e-4 for fp32
sums; the cap's slope 1 - t^2 is off by 2^-21, 2^-13 of it times 2^-8.
"""
from __future__ import annotations

import math

import torch

F64 = torch.float64
HALF_BF16 = 2.0 ** -8
HALF_F32 = 2.0 ** -24


def runs(ids):
    """Documents of a sequence: (first, end) of each run of equal numbers >= 0."""
    out, a = [], 0
    ids = [int(x) for x in ids]
    for j in range(1, len(ids) + 1):
        if j == len(ids) or ids[j] != ids[a]:
            if ids[a] >= 0:
                out.append((a, j))
            a = j
    return out


def visible(N, Nk, causal, ids=None, prefix=0):
    """[N, Nk] truth for one sequence."""
    pos = torch.arange(Nk - N, Nk)[:, None]
    key = torch.arange(Nk)[None, :]
    see = torch.ones((N, Nk), dtype=torch.bool)
    if causal:
        see = (key <= pos) | (key < prefix)
    if ids is not None:
        same = torch.zeros((N, Nk), dtype=torch.bool)
        for a, e in runs(ids):
            same |= (pos >= a) & (pos < e) & (key >= a) & (key < e)
        see = see & same
    return see


class Rules:
    def __init__(self, causal=False, scale=None, softcap=0.0, slopes=None, documents=None, prefix_lens=None):
        self.causal, self.scale, self.cap = causal, scale, softcap
        self.slopes, self.docs, self.prefix = slopes, documents, prefix_lens

    def kwargs(self, dev):
        to = lambda t: None if t is None else t.to(dev)  # noqa: E731
        return dict(causal=self.causal, scale=self.scale, softcap=self.cap, slopes=to(self.slopes), documents=to(self.docs),
                    prefix_lens=to(self.prefix))


def scores(q, k, rules, slope, N, Nk):
    """s, tanh (or 0), error bound of s for one head, fp64."""
    d = q.shape[-1]
    scale = rules.scale if rules.scale is not None else 1 / math.sqrt(d)
    x = q @ k.T * scale
    e = 4 * d * HALF_F32 * (q.abs() @ k.abs().T) * scale
    t = torch.zeros_like(x)
    s = x
    if rules.cap:
        t = torch.tanh(x / rules.cap)
        s = rules.cap * t
        e = e + 2.0 ** -21 * rules.cap
    e = e + 2.0 ** -21 * s.abs()
    if slope is not None:
        dist = (torch.arange(Nk - N, Nk)[:, None] - torch.arange(Nk)[None, :]).abs().to(F64)
        s = s - float(slope) * dist
        e = e + 2.0 ** -21 * abs(float(slope)) * dist
    return s, t, e


def attention(q, k, v, rules, do=None):
    """dict of O, L and bounds dO, dL; with `do` the gradients (dq, dk, dv) and their bounds too.  CPU, fp64."""
    B, Hq, N, d = q.shape
    Hkv, Nk = k.shape[1:3]
    R = Hq // Hkv
    scale = rules.scale if rules.scale is not None else 1 / math.sqrt(d)
    r = dict(O=torch.zeros((B, Hq, N, d), dtype=F64), dO=torch.zeros((B, Hq, N, d), dtype=F64),
             L=torch.full((B, Hq, N), -math.inf, dtype=F64), dL=torch.zeros((B, Hq, N), dtype=F64))
    if do is not None:
        for n, like in (("dq", q), ("dk", k), ("dv", v)):
            r[n] = torch.zeros(like.shape, dtype=F64)
            r["b" + n] = torch.zeros(like.shape, dtype=F64)
    for b in range(B):
        see = visible(N, Nk, rules.causal, rules.docs[b] if rules.docs is not None else None,
                      max(0, min(Nk, int(rules.prefix[b]))) if rules.prefix is not None else 0)
        empty = ~see.any(-1, keepdim=True)
        for h in range(Hq):
            Q, K, V = q[b, h].to(F64), k[b, h // R].to(F64), v[b, h // R].to(F64)
            s, t, e = scores(Q, K, rules, rules.slopes[h] if rules.slopes is not None else None, N, Nk)
            s = torch.where(see, s, -math.inf)
            e = torch.where(see, e, 0.0)
            P = torch.softmax(torch.where(empty, 0.0, s), -1).masked_fill(~see, 0.0)
            E = (P * e).sum(-1, keepdim=True)
            r["O"][b, h] = P @ V
            r["dO"][b, h] = (P * (HALF_BF16 + e + E + 2.0 ** -20)) @ V.abs()
            r["L"][b, h] = torch.logsumexp(s, -1)
            r["dL"][b, h] = torch.where(empty[:, 0], 0.0, E[:, 0] + 2.0 ** -20 * (1 + r["L"][b, h].abs()))
            if do is None:
                continue
            G = do[b, h].to(F64)
            D = (G * r["O"][b, h]).sum(-1, keepdim=True)
            dS = P * (G @ V.T - D)
            f = 1 - t * t
            dX = dS * f * scale
            w = 2 * HALF_BF16 + 4 * (e + E)  # of each weight
            A = w * (dS.abs() + P * (G.abs() * (P @ V.abs())).sum(-1, keepdim=True)) * (f + 2.0 ** -13) * scale
            r["dq"][b, h] = dX @ K
            r["bdq"][b, h] = A @ K.abs()
            r["dk"][b, h // R] += dX.T @ Q
            r["bdk"][b, h // R] += A.T @ Q.abs()
            r["dv"][b, h // R] += P.T @ G
            r["bdv"][b, h // R] += (w * P).T @ G.abs()
    if do is not None:
        for n in ("bdq", "bdk", "bdv"):
            r[n] += 1e-4
    return r


def check(a, ref, bound, what):
    x = a.double().cpu()
    assert not x.isnan().any(), f"{what}: NaN"
    half = HALF_BF16 if a.dtype == torch.bfloat16 else HALF_F32
    over = (x - ref).abs() - bound - half * (ref.abs() + bound)
    assert float(over.max()) <= 0, f"{what}: exceeds its bound by {float(over.max()):.3e}"


def check_forward(o, lse, r, what=""):
    check(o, r["O"], r["dO"], what + " O")
    if lse is not None:
        x, L = lse.double().cpu(), r["L"]
        assert torch.equal(torch.isneginf(x), torch.isneginf(L)), f"{what}: empty rows disagree"
        f = torch.isfinite(L)
        assert bool(torch.isfinite(x)[f].all()), f"{what}: LSE is not finite"
        if f.any():
            over = (x - L).abs()[f] - r["dL"][f]
            assert float(over.max()) <= 0, f"{what}: LSE exceeds its bound by {float(over.max()):.3e}"


def check_gradients(grads, r, what=""):
    for g, n in zip(grads, ("dq", "dk", "dv")):
        check(g, r[n], r["b" + n], f"{what} {n}")


def documents(B, Nk, lengths, pads=None, seed=0):
    """int32 [B, Nk]: documents of `lengths` (the last one to the end), each row's shifted, padding behind."""
    ids = torch.full((B, Nk), -1, dtype=torch.int32)
    for b in range(B):
        end = Nk - (pads[b] if pads is not None else 0)
        at, n, i = 0, 0, b
        while at < end:
            m = lengths[i % len(lengths)]
            ids[b, at:min(end, at + m)] = (n * 7 + seed) % 5 + 10 * (n % 2)  # neighbours differ, numbers come again
            at, n, i = at + m, n + 1, i + 1
    return ids
