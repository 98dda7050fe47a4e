"""Measured cases of attention under score rules (scores capped by a tanh, a bias that falls with the
distance, document and prefix masks, shared key/value heads), its training step, and decode attention for
a batch whose sequences share a long prefix.

``run`` computes each operator in its plain form (elementary torch operations in fp32, rounded once
at the end) or, with ``own`` set, through the package's entry points.
"""
import math

import torch

own = False

DEV = "cuda"
BF16 = torch.bfloat16


# ----------------------------------------------------------------------------------------- cases
# mask: "full", "causal", "docs" (causal within packed documents, padding behind them), "docs_full"
# (documents, both directions) or "prefix" (causal, but a prefix of each sequence is seen by all)
def listed():
    return [
        # the GPT-2-medium-shaped prefill, several documents packed into each sequence
        dict(name="fwd_docs_b64_h16_d64", op="fwd", B=64, Hq=16, Hkv=16, N=1024, Nk=1024, d=64, mask="docs", docs=5, pad=60,
             cap=0.0, slopes=False),
        # ragged long causal prefill, capped scores, 4 query heads per key/value head: arithmetic counts
        dict(name="fwd_cap_n4097_d128", op="fwd", B=4, Hq=16, Hkv=4, N=4097, Nk=4097, d=128, mask="causal", docs=0, pad=0,
             cap=50.0, slopes=False),
        # one long packed sequence, capped scores
        dict(name="fwd_docs_cap_n16384_d128", op="fwd", B=1, Hq=32, Hkv=8, N=16384, Nk=16384, d=128, mask="docs", docs=9,
             pad=100, cap=30.0, slopes=False),
        # few queries behind cached keys, distance bias and a prefix mask: latency
        dict(name="fwd_bias_prefix_odd_d32", op="fwd", B=8, Hq=8, Hkv=2, N=77, Nk=513, d=32, mask="prefix", docs=0, pad=0,
             cap=0.0, slopes=True),
        # training step over packed documents
        dict(name="train_docs_b16_h16_d64", op="train", B=16, Hq=16, Hkv=16, N=1024, Nk=1024, d=64, mask="docs", docs=5, pad=60,
             cap=0.0, slopes=False),
        # training step with capped scores and shared key/value heads, ragged length
        dict(name="train_cap_n4097_d128", op="train", B=1, Hq=16, Hkv=4, N=4097, Nk=4097, d=128, mask="causal", docs=0, pad=0,
             cap=50.0, slopes=False),
        # training step with a distance bias and a prefix mask
        dict(name="train_bias_prefix_d64", op="train", B=4, Hq=12, Hkv=4, N=1500, Nk=1500, d=64, mask="prefix", docs=0, pad=0,
             cap=0.0, slopes=True),
        # a short odd batch: documents seen both ways, capped scores and a distance bias: latency
        dict(name="train_all_odd_d32", op="train", B=3, Hq=6, Hkv=2, N=77, Nk=77, d=32, mask="docs_full", docs=3, pad=9,
             cap=20.0, slopes=True),
        # two sequences behind a short prompt: latency
        dict(name="decode_b2_p512", op="decode", B=2, Hq=32, Hkv=8, d=128, P=512, Nk_max=256, lo=1, hi=200, cap=0.0,
             slopes=False),
        # a batch behind a long shared prompt: 64 query rows meet the prefix in each key/value head
        dict(name="decode_b16_p8192", op="decode", B=16, Hq=32, Hkv=8, d=128, P=8192, Nk_max=2048, lo=0, hi=2000, cap=0.0,
             slopes=False),
        # a large batch behind a very long prompt, capped scores: arithmetic counts in the prefix
        dict(name="decode_cap_b64_p32768", op="decode", B=64, Hq=32, Hkv=8, d=128, P=32768, Nk_max=2048, lo=0, hi=2000,
             cap=50.0, slopes=False),
        # odd sizes, distance bias
        dict(name="decode_bias_b37_d64", op="decode", B=37, Hq=15, Hkv=5, d=64, P=3001, Nk_max=1100, lo=0, hi=1001, cap=0.0,
             slopes=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["fwd", "train", "decode"])
    d = rng.choice([32, 64, 128])
    Hkv = rng.randint(1, 8)
    R = rng.choice([1, 2, 3, 4, 5, 8])
    cap = rng.choice([0.0, 0.0, 15.0, 30.0, 50.0])
    slopes = rng.random() < 0.4
    if op == "decode":
        P = _log(rng, 100, 32000)
        Nk_max = _log(rng, 16, 2000)
        B = _log(rng, 1, 64)
        return dict(op=op, B=B, Hq=Hkv * R, Hkv=Hkv, d=d, P=P, Nk_max=Nk_max, lo=0, hi=Nk_max, cap=cap, slopes=slopes)
    mask = rng.choice(["full", "causal", "docs", "docs_full", "prefix"])
    N = _log(rng, 1, 5000)
    Nk = N if mask in ("docs", "docs_full") or op == "train" or rng.random() < 0.5 else N + _log(rng, 1, 3000)
    most = 1 << (29 if op == "fwd" else 27)  # pairs of a query and a key, over all heads
    B = _log(rng, 1, 16)
    B = max(1, min(B, most // (Hkv * R * N * Nk)))
    while Hkv * R * N * Nk > most and R > 1:
        R -= 1
    while Hkv * R * N * Nk > most and Hkv > 1:
        Hkv -= 1
    return dict(op=op, B=B, Hq=Hkv * R, Hkv=Hkv, N=N, Nk=Nk, d=d, mask=mask, docs=rng.randint(1, 8) if "docs" in mask else 0,
                pad=rng.randint(0, N // 8) if "docs" in mask else 0, cap=cap, slopes=slopes)


# ---------------------------------------------------------------------------------------- inputs
def _pads(case):
    """Padding positions at the end of each sequence: evenly spaced over [0, pad]."""
    return torch.linspace(0, case["pad"], case["B"]).round().long().tolist()


def _doc_lengths(case, pad):
    """Lengths of a sequence's documents, in growing order: proportional to 1, 2, ..."""
    n = min(case["docs"], case["Nk"] - pad)
    total = case["Nk"] - pad
    cuts = [total * i * (i + 1) // (n * (n + 1)) for i in range(n + 1)]
    return [b - a for a, b in zip(cuts, cuts[1:])]


def _prefixes(case):
    """Prefix lengths: evenly spaced over [0, Nk / 2]."""
    return torch.linspace(0, case["Nk"] // 2, case["B"]).round().to(torch.int32)


def _ladder(case):
    """Lengths of the sequences' own keys: evenly spaced over [lo, hi]."""
    return torch.linspace(case["lo"], case["hi"], case["B"]).round().to(torch.int32)


def prepare(case, seed):
    g = torch.Generator().manual_seed(int(seed))  # small host-side draws
    gd = torch.Generator(device=DEV).manual_seed(int(seed))
    rand = lambda *s: torch.randn(s, generator=gd, device=DEV, dtype=torch.float32).to(BF16)  # noqa: E731
    s = {"case": case}
    B, Hq, Hkv, d = (case[n] for n in ("B", "Hq", "Hkv", "d"))
    # heads' slopes fall geometrically, as distance biases are trained with
    s["slopes"] = torch.exp2(-8.0 * torch.arange(1, Hq + 1, device=DEV) / Hq) if case["slopes"] else None
    gain = 3.0 if case["cap"] else 1.0  # scores that a cap is there for
    if case["op"] == "decode":
        s["q"] = (gain * rand(B, Hq, 1, d).float()).to(BF16)
        s["k_prefix"], s["v_prefix"] = rand(Hkv, case["P"], d), rand(Hkv, case["P"], d)
        s["k_cache"], s["v_cache"] = rand(B, Hkv, case["Nk_max"], d), rand(B, Hkv, case["Nk_max"], d)
        s["lens"] = _ladder(case)[torch.randperm(B, generator=g)].to(DEV)
        return s
    N, Nk = case["N"], case["Nk"]
    s["q"], s["k"], s["v"] = (gain * rand(B, Hq, N, d).float()).to(BF16), rand(B, Hkv, Nk, d), rand(B, Hkv, Nk, d)
    s["docs"] = s["prefix"] = None
    if "docs" in case["mask"]:
        ids = torch.full((B, Nk), -1, dtype=torch.int32)  # padding: no document
        for b, pad in enumerate(_pads(case)):
            lens = _doc_lengths(case, pad)
            lens = [lens[i] for i in torch.randperm(len(lens), generator=g).tolist()]
            ids[b, :Nk - pad] = torch.repeat_interleave(torch.arange(len(lens)), torch.tensor(lens)).to(torch.int32)
        s["docs"] = ids.to(DEV)
    elif case["mask"] == "prefix":
        s["prefix"] = _prefixes(case)[torch.randperm(B, generator=g)].to(DEV)
    if case["op"] == "train":
        s["do"] = rand(B, Hq, N, d)
    return s


# ------------------------------------------------------------------------------------ plain forms
def _seen(s, case, b):
    """[N, Nk] truth: query i of sequence b, at position Nk - N + i, sees key j."""
    N, Nk = case["N"], case["Nk"]
    pos = torch.arange(Nk - N, Nk, device=DEV)[:, None]
    key = torch.arange(Nk, device=DEV)[None, :]
    if case["mask"] in ("full", "docs_full"):
        see = torch.ones((N, Nk), dtype=torch.bool, device=DEV)
    else:
        see = key <= pos
    if s["prefix"] is not None:
        see = see | (key < s["prefix"][b])
    if s["docs"] is not None:
        ids = s["docs"][b]
        see = see & (ids[pos.clamp(min=0)] == ids[key]) & (ids[key] >= 0) & (pos >= 0)
    return see


def _scores(q, k, case, slopes, dist):
    """Scaled, capped and biased scores of q [h, n, d] and k [h, m, d], and tanh of the scaled ones (or None)."""
    x = (q @ k.transpose(-1, -2)).mul_(1.0 / math.sqrt(case["d"]))
    t = None
    if case["cap"]:
        t = x.div_(case["cap"]).tanh_()
        x = t * case["cap"]
    if slopes is not None:
        x = x - slopes[:, None, None] * dist
    return x, t


def _softmax(x):
    """Weights and log-sum-exp of scores; a row of -inf has weights 0."""
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = (x - m).exp_()
    l = p.sum(-1, keepdim=True)
    p /= torch.where(l > 0, l, 1.0)
    return p, (m + l.log()).squeeze(-1)


def _plain_rules(s, case):
    B, Hq, N, d = s["q"].shape
    Hkv, Nk = s["k"].shape[1:3]
    R = Hq // Hkv
    train = case["op"] == "train"
    o = torch.empty((B, Hq, N, d), dtype=BF16, device=DEV)
    lse = torch.empty((B, Hq, N), dtype=torch.float32, device=DEV)
    if train:
        dq, dk, dv = (torch.empty_like(s[n]) for n in ("q", "k", "v"))
    step = max(1, (1 << 28) // (R * N * Nk))  # key/value heads at a time
    dist = (torch.arange(Nk - N, Nk, device=DEV)[:, None] - torch.arange(Nk, device=DEV)[None, :]).abs().float()
    for b in range(B):
        see = _seen(s, case, b)
        for h in range(0, Hkv, step):
            e = min(h + step, Hkv)
            q = s["q"][b, h * R:e * R].float()
            k = s["k"][b, h:e].float().repeat_interleave(R, 0)
            v = s["v"][b, h:e].float().repeat_interleave(R, 0)
            x, t = _scores(q, k, case, s["slopes"][h * R:e * R] if s["slopes"] is not None else None, dist)
            p, l = _softmax(x.masked_fill(~see, -math.inf))
            y = p @ v
            o[b, h * R:e * R] = y.to(BF16)
            lse[b, h * R:e * R] = l
            if not train:
                continue
            do = s["do"][b, h * R:e * R].float()
            dx = p * (do @ v.transpose(-1, -2) - (do * y).sum(-1, keepdim=True))
            if t is not None:
                dx *= 1.0 - t * t  # the cap's derivative
            dx *= 1.0 / math.sqrt(d)
            dq[b, h * R:e * R] = (dx @ k).to(BF16)
            dk[b, h:e] = (dx.transpose(-1, -2) @ q).unflatten(0, (e - h, R)).sum(1).to(BF16)
            dv[b, h:e] = (p.transpose(-1, -2) @ do).unflatten(0, (e - h, R)).sum(1).to(BF16)
    return (o, lse, dq, dk, dv) if train else (o, lse)


def _plain_decode(s, case):
    B, Hq, _, d = s["q"].shape
    Hkv, P = s["k_prefix"].shape[:2]
    R, Nk = Hq // Hkv, case["Nk_max"]
    lens = s["lens"].long()
    q = s["q"].float().reshape(B, Hkv, R, d)
    # the prefix's scores as one product for each key/value head, over the rows of all sequences
    kp, vp = s["k_prefix"].float(), s["v_prefix"].float()
    xp = (q.transpose(0, 1).reshape(Hkv, B * R, d) @ kp.transpose(1, 2)).reshape(Hkv, B, R, P).transpose(0, 1)
    xs = q @ s["k_cache"].float().transpose(2, 3)
    x = torch.cat((xp, xs), -1).mul_(1.0 / math.sqrt(d))
    if case["cap"]:
        x = (x / case["cap"]).tanh_() * case["cap"]
    key = torch.arange(P + Nk, device=DEV)
    end = P + lens[:, None]  # the query sits at the last key
    if s["slopes"] is not None:
        x = x - s["slopes"].reshape(1, Hkv, R, 1) * (end - 1 - key)[:, None, None].float()
    p, lse = _softmax(x.masked_fill((key >= end)[:, None, None], -math.inf))
    o = (p[..., :P].transpose(0, 1).reshape(Hkv, B * R, P) @ vp).reshape(Hkv, B, R, d).transpose(0, 1)
    o = o + p[..., P:] @ s["v_cache"].float()
    return o.reshape(B, Hq, 1, d).to(BF16), lse.reshape(B, Hq, 1)


# ------------------------------------------------------------------------------------- own kernels
def _own(s, case):
    import exact_tiled_attention_fa_gb300 as fa
    if case["op"] == "decode":
        if "ws" not in s:
            size = fa.decode_prefix_workspace_size(case["B"], case["Hq"], case["Hkv"], case["d"], fa.num_sms())
            s["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV)
        return fa.decode_prefix(s["q"], s["k_prefix"], s["v_prefix"], s["k_cache"], s["v_cache"], s["lens"], softcap=case["cap"],
                                slopes=s["slopes"], workspace=s["ws"])
    rules = dict(causal=case["mask"] not in ("full", "docs_full"), softcap=case["cap"], slopes=s["slopes"],
                 documents=s["docs"], prefix_lens=s["prefix"])
    train = case["op"] == "train"
    if "ws" not in s:
        size = fa.fwd_rules_workspace_size(case["B"], case["N"])
        if train:
            size = max(size, fa.bwd_rules_workspace_size(*(case[n] for n in ("B", "Hq", "Hkv", "N", "Nk", "d")), fa.num_sms()))
        s["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV)
    o, lse = fa.fwd_rules(s["q"], s["k"], s["v"], workspace=s["ws"], **rules)
    if not train:
        return o, lse
    grads = fa.bwd_rules(s["q"], s["k"], s["v"], o, lse, s["do"], workspace=s["ws"], **rules)
    return (o, lse, *grads)


def run(state):
    case = state["case"]
    if own:
        return _own(state, case)
    return _plain_decode(state, case) if case["op"] == "decode" else _plain_rules(state, case)


# ------------------------------------------------------------------------------------------- work
def _pairs(case):
    """(query, key) pairs that see each other, over the batch, for one head."""
    B, N, Nk, mask = case["B"], case["N"], case["Nk"], case["mask"]
    if mask == "full":
        return B * N * Nk
    if "docs" in mask:
        lens = [n for pad in _pads(case) for n in _doc_lengths(case, pad)]
        return sum(n * (n + 1) // 2 if mask == "docs" else n * n for n in lens)
    causal = N * (N + 1) // 2 + N * (Nk - N)
    if mask == "causal":
        return B * causal
    total = 0
    for f in _prefixes(case).tolist():
        first = max(0, f - (Nk - N) - 1)  # queries that would see fewer than the f keys of the prefix
        hidden = sum(f - (Nk - N + i + 1) for i in range(min(first, N)))
        total += causal + hidden
    return total


def work(case):
    B, Hq, Hkv, d = (case[n] for n in ("B", "Hq", "Hkv", "d"))
    if case["op"] == "decode":
        keys = int(_ladder(case).sum())
        return {"bytes": (case["P"] + keys) * Hkv * d * 4 + B * Hq * (d * 4 + 4),
                "flops": 4.0 * d * Hq * (B * case["P"] + keys)}
    qn, kn = B * Hq * case["N"] * d, B * Hkv * case["Nk"] * d
    if case["op"] == "fwd":
        return {"bytes": qn * 4 + kn * 4 + B * Hq * case["N"] * 4, "flops": 4.0 * d * Hq * _pairs(case)}
    return {"bytes": qn * 8 + kn * 8 + B * Hq * case["N"] * 4, "flops": 14.0 * d * Hq * _pairs(case)}


# ------------------------------------------------------------------------------------------ exact
def _exact_mask(s, case, b):
    """What each query sees, document by document."""
    N, Nk = case["N"], case["Nk"]
    see = torch.zeros((N, Nk), dtype=torch.bool)
    runs = [(0, Nk)]
    if s["docs"] is not None:
        ids = s["docs"][b].tolist()
        runs, a = [], 0
        for j in range(1, Nk + 1):
            if j == Nk or ids[j] != ids[a]:
                if ids[a] >= 0:
                    runs.append((a, j))
                a = j
    pre = int(s["prefix"][b]) if s["prefix"] is not None else 0
    off = Nk - N
    for a, e in runs:
        rows = range(max(a - off, 0), e - off) if s["docs"] is not None else range(N)
        if case["mask"] in ("full", "docs_full"):
            see[rows.start:rows.stop, a:e] = True
            continue
        for i in rows:
            see[i, a:min(e, max(off + i + 1, pre))] = True
    return see.to(DEV)


def exact(case, seed):
    s = prepare(case, seed)
    B, Hq, Hkv, d = (case[n] for n in ("B", "Hq", "Hkv", "d"))
    R, cap = Hq // Hkv, case["cap"]

    def attend(q, k, v, see, slope, dist):
        x = torch.einsum("nd,md->nm", q, k) / d ** 0.5
        if cap:
            x = cap * (1.0 - 2.0 / (torch.exp(2.0 * x / cap) + 1.0))  # tanh by exponentials
        if slope is not None:
            x = x - slope.double() * dist
        x = torch.where(see, x, -math.inf)
        empty = ~see.any(-1, keepdim=True)
        lse = torch.logsumexp(x, -1)
        return torch.softmax(torch.where(empty, 0.0, x), -1).masked_fill(empty, 0.0) @ v, lse

    if case["op"] == "decode":
        o = torch.empty((B, Hq, 1, d), dtype=torch.float64, device=DEV)
        lse = torch.empty((B, Hq, 1), dtype=torch.float64, device=DEV)
        kp, vp = s["k_prefix"].double(), s["v_prefix"].double()
        for b, n in enumerate(s["lens"].tolist()):
            m = case["P"] + n
            dist = torch.arange(m - 1, -1, -1, dtype=torch.float64, device=DEV)[None]
            see = torch.ones((1, m), dtype=torch.bool, device=DEV)
            for g in range(Hkv):
                k = torch.cat((kp[g], s["k_cache"][b, g, :n].double()))
                v = torch.cat((vp[g], s["v_cache"][b, g, :n].double()))
                for h in range(g * R, (g + 1) * R):
                    o[b, h], lse[b, h] = attend(s["q"][b, h].double(), k, v, see,
                                                s["slopes"][h] if s["slopes"] is not None else None, dist)
        return o, lse
    train = case["op"] == "train"
    N, Nk = case["N"], case["Nk"]
    o = torch.empty((B, Hq, N, d), dtype=torch.float64, device=DEV)
    lse = torch.empty((B, Hq, N), dtype=torch.float64, device=DEV)
    if train:
        dq = torch.empty((B, Hq, N, d), dtype=torch.float64, device=DEV)
        dk, dv = (torch.zeros((B, Hkv, Nk, d), dtype=torch.float64, device=DEV) for _ in range(2))
    dist = (torch.arange(Nk - N, Nk, dtype=torch.float64, device=DEV)[:, None]
            - torch.arange(Nk, dtype=torch.float64, device=DEV)[None, :]).abs()
    for b in range(B):
        see = _exact_mask(s, case, b)
        for h in range(Hq):
            x = [s["q"][b, h].double(), s["k"][b, h // R].double(), s["v"][b, h // R].double()]
            if train:
                x = [t.requires_grad_() for t in x]
            y, l = attend(*x, see, s["slopes"][h] if s["slopes"] is not None else None, dist)
            o[b, h], lse[b, h] = y.detach(), l.detach()
            if train:
                grads = torch.autograd.grad(y, x, s["do"][b, h].double())
                dq[b, h] = grads[0]
                dk[b, h // R] += grads[1]
                dv[b, h // R] += grads[2]
    return (o, lse, dq, dk, dv) if train else (o, lse)
