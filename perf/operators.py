"""Measured cases of the operators around cached attention: query/key norm with rotation (and its
gradient), the same written into a key/value cache, decode attention for a tree of drafted tokens,
and the compaction of a cache onto the accepted path.

``run`` computes each operator in its plain form (elementary torch operations in fp32, rounded once
at the end) or, with ``own`` set, through the package's entry points.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BF16 = torch.bfloat16
EPS = 1e-6


# ----------------------------------------------------------------------------------------- cases
def listed():
    return [
        # training step of the GPT-2-medium-shaped prefill: the operands of the forward
        dict(name="norm_rope_b64_h16_d64", op="norm_rope", B=64, N=1024, Hq=16, Hkv=16, d=64, rot=64,
             interleaved=False, expand=False, packed=False, grad="bf16"),
        # a short ragged batch with shared key/value heads, partial rotation, other token positions
        dict(name="norm_rope_odd_d32", op="norm_rope", B=3, N=77, Hq=10, Hkv=2, d=32, rot=16,
             interleaved=True, expand=True, packed=True, grad="bf16"),
        # the gradient of the first, from bf16 gradients
        dict(name="norm_rope_bwd_b64_h16_d64", op="norm_rope_bwd", B=64, N=1024, Hq=16, Hkv=16, d=64, rot=64,
             interleaved=False, expand=False, packed=False, grad="bf16"),
        # long ragged sequence, 8 key/value heads under 32 query heads (gradients summed over each group), fp32 gradients
        dict(name="norm_rope_bwd_n4097_d128", op="norm_rope_bwd", B=2, N=4097, Hq=32, Hkv=8, d=128, rot=128,
             interleaved=False, expand=True, packed=True, grad="fp32"),
        # one new token for each of 16 sequences (the decode configuration): latency
        dict(name="append_b16_t1", op="append", B=16, T=1, Hq=32, Hkv=32, d=128, rot=128, interleaved=False,
             Nk_max=2048, lo=1, hi=2000, ragged=False),
        # verification step of a large batch, trees of different sizes
        dict(name="append_b64_t64_ragged", op="append", B=64, T=64, Hq=32, Hkv=8, d=128, rot=64, interleaved=True,
             Nk_max=1024, lo=0, hi=960, ragged=True),
        # one sequence, a small tree: latency
        dict(name="tree_b1_t8", op="tree", B=1, T=8, Hq=32, Hkv=8, d=128, Nk_max=2048, lo=2000, hi=2000, ragged=False),
        # the decode configuration's lengths, 4 query heads per key/value head, 16 drafted tokens: bandwidth
        dict(name="tree_b16_t16", op="tree", B=16, T=16, Hq=32, Hkv=8, d=128, Nk_max=32768, lo=1024, hi=32700, ragged=False),
        # the same with 64 drafted tokens: 256 rows for each key/value head, arithmetic counts
        dict(name="tree_b16_t64", op="tree", B=16, T=64, Hq=32, Hkv=8, d=128, Nk_max=32768, lo=1024, hi=32700, ragged=True),
        # odd sizes: 3 query heads per key/value head, 27 nodes at most, d = 64
        dict(name="tree_b5_t27_d64", op="tree", B=5, T=27, Hq=15, Hkv=5, d=64, Nk_max=9001, lo=0, hi=8970, ragged=True),
        # one layer of a small batch: latency
        dict(name="compact_b2_t8", op="compact", L=1, B=2, T=8, Hkv=8, d=128, Nk_max=1024),
        # every layer of a large batch in one call
        dict(name="compact_l16_b32_t64", op="compact", L=16, B=32, T=64, Hkv=8, d=128, Nk_max=256),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_bwd", "append", "tree", "tree", "compact"])
    d = rng.choice([32, 64, 128])
    Hkv = rng.randint(1, 16)
    R = rng.choice([1, 2, 3, 4, 5, 7, 8])
    if op in ("norm_rope", "norm_rope_bwd"):
        B = _log(rng, 1, 32)
        R = min(R, max(1, 32 // Hkv))
        N = _log(rng, 1, max(2, min(5000, (1 << 26) // (B * Hkv * (R + 2) * d))))
        return dict(op=op, B=B, N=N, Hq=Hkv * R, Hkv=Hkv, d=d, rot=16 * rng.randint(1, d // 16),
                    interleaved=rng.random() < 0.5, expand=rng.random() < 0.5, packed=rng.random() < 0.5,
                    grad=rng.choice(["bf16", "fp32"]))
    if op == "append":
        Nk_max = _log(rng, 200, 1100)
        return dict(op=op, B=_log(rng, 1, 48), T=_log(rng, 1, 64), Hq=Hkv * min(R, 4), Hkv=Hkv, d=d,
                    rot=16 * rng.randint(1, d // 16), interleaved=rng.random() < 0.5, Nk_max=Nk_max, lo=0,
                    hi=Nk_max - 64, ragged=rng.random() < 0.5)
    if op == "tree":
        Hkv = min(Hkv, 8)
        B = _log(rng, 1, 16)
        Nk_max = _log(rng, 200, 32000)
        T = _log(rng, 1, 128)
        R = max(1, min(R, 256 // T))
        return dict(op=op, B=B, T=T, Hq=Hkv * R, Hkv=Hkv, d=d, Nk_max=Nk_max, lo=0, hi=Nk_max - T,
                    ragged=rng.random() < 0.5)
    return dict(op=op, L=_log(rng, 1, 12), B=_log(rng, 1, 32), T=_log(rng, 1, 64), Hkv=min(Hkv, 8), d=d,
                Nk_max=_log(rng, 128, 300))


# ---------------------------------------------------------------------------------------- inputs
def _lengths(case, g, room):
    """Cached lengths: evenly spaced over [lo, hi], in the order the seed gives."""
    B = case["B"]
    hi = min(case["hi"], case["Nk_max"] - room)
    ladder = torch.linspace(min(case["lo"], hi), hi, B).round().to(torch.int32)
    return ladder[torch.randperm(B, generator=g)]


def _node_ladder(case):
    """Nodes in use: all T, or (ragged) evenly spaced over [1, T]."""
    B, T = case["B"], case["T"]
    return torch.linspace(1, T, B).round().to(torch.int32) if case["ragged"] else torch.full((B,), T, dtype=torch.int32)


def _tree(B, T, g):
    """Parents of a random recursive tree: node t hangs below a uniformly drawn earlier node, or below the
    last cached token (-1)."""
    u = torch.rand((B, T), generator=g)
    return (torch.floor(u * (torch.arange(T) + 1)) - 1).to(torch.int32)


def _tables(max_pos, rot):
    """cos and sin of position * 10000^(-2i/rot), computed in fp64 (far positions) and held in fp32."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(max_pos, dtype=torch.float64, device=DEV)[:, None] * inv
    return a.cos().float(), a.sin().float()


def prepare(case, seed):
    g = torch.Generator().manual_seed(int(seed))  # small host-side draws
    gd = torch.Generator(device=DEV).manual_seed(int(seed))
    rand = lambda *s: torch.randn(s, generator=gd, device=DEV, dtype=torch.float32).to(BF16)  # noqa: E731
    s = {"case": case}
    op = case["op"]
    if op in ("norm_rope", "norm_rope_bwd", "append"):
        B, Hq, Hkv, d, rot = (case[n] for n in ("B", "Hq", "Hkv", "d", "rot"))
        n = case["T"] if op == "append" else case["N"]
        if op == "append" or case["packed"]:  # slices of one projection's output
            x = rand(B, n, Hq + 2 * Hkv, d)
            s["q"], s["k"], s["v"] = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
        else:
            s["q"], s["k"], s["v"] = rand(B, n, Hq, d), rand(B, n, Hkv, d), rand(B, n, Hkv, d)
        s["wq"] = (1.0 + 0.2 * torch.randn(d, generator=gd, device=DEV)).to(BF16)
        s["wk"] = (1.0 + 0.2 * torch.randn(d, generator=gd, device=DEV)).to(BF16)
        if op == "append":
            s["lens"] = _lengths(case, g, n).to(DEV)
            s["n_nodes"] = _node_ladder(case)[torch.randperm(B, generator=g)].to(DEV)
            s["parents"] = _tree(B, n, g).to(DEV)
            s["k_cache"], s["v_cache"] = rand(B, Hkv, case["Nk_max"], d), rand(B, Hkv, case["Nk_max"], d)
            s["cos"], s["sin"] = _tables(case["Nk_max"], rot)
            return s
        s["cos"], s["sin"] = _tables(n + 256, rot)
        # packed sequences start anew at other positions: an offset for each batch row
        s["pos"] = (torch.arange(n)[None, :] + torch.randint(0, 256, (B, 1), generator=g)).to(torch.int32).to(DEV)
        if op == "norm_rope_bwd":
            gt = BF16 if case["grad"] == "bf16" else torch.float32
            Ho = Hq if case["expand"] else Hkv
            s["dq"], s["dk"], s["dv"] = (rand(B, h, n, d).to(gt) for h in (Hq, Ho, Ho))
        return s
    if op == "tree":
        B, T, Hq, Hkv, d, Nk_max = (case[n] for n in ("B", "T", "Hq", "Hkv", "d", "Nk_max"))
        s["q"], s["k_cache"], s["v_cache"] = rand(B, Hq, T, d), rand(B, Hkv, Nk_max, d), rand(B, Hkv, Nk_max, d)
        s["lens"] = _lengths(case, g, T).to(DEV)
        s["n_nodes"] = _node_ladder(case).to(DEV)
        s["parents"] = _tree(B, T, g).to(DEV)
        return s
    L, B, T, Hkv, d, Nk_max = (case[n] for n in ("L", "B", "T", "Hkv", "d", "Nk_max"))
    s["k_cache"], s["v_cache"] = rand(L, B, Hkv, Nk_max, d), rand(L, B, Hkv, Nk_max, d)
    s["lens"] = torch.randint(0, Nk_max - T + 1, (B,), generator=g).to(torch.int32).to(DEV)
    par = _tree(B, T, g).tolist()
    acc, cnt = np.zeros((B, T), dtype=np.int32), np.zeros(B, dtype=np.int32)
    for b, leaf in enumerate(torch.randint(0, T, (B,), generator=g).tolist()):
        path = []
        while leaf >= 0:  # the path from the root to a drawn node
            path.append(leaf)
            leaf = par[b][leaf]
        cnt[b] = len(path)
        acc[b, :len(path)] = path[::-1]
    s["accepted"], s["n_accepted"] = torch.from_numpy(acc).to(DEV), torch.from_numpy(cnt).to(DEV)
    return s


# ------------------------------------------------------------------------------------ plain forms
def _rotate(y, cos, sin, rot, interleaved):
    """Rotates the first rot dims of y [..., d] by the angles whose cosines and sines are given [..., rot/2]."""
    r, rest = y[..., :rot], y[..., rot:]
    if interleaved:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, a * sin + b * cos), dim=-1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat((a * cos - b * sin, a * sin + b * cos), dim=-1)
    return torch.cat((r, rest), dim=-1)


def _norm(x, w):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _angles(s, pos):
    """Table rows of the positions [B, n], with a head axis."""
    return s["cos"][pos.long()][:, :, None], s["sin"][pos.long()][:, :, None]


def _plain_norm_rope(s, case):
    cos, sin = _angles(s, s["pos"])
    rep = case["Hq"] // case["Hkv"] if case["expand"] else 1
    q = _rotate(_norm(s["q"], s["wq"]), cos, sin, case["rot"], case["interleaved"]).to(BF16).transpose(1, 2)
    k = _rotate(_norm(s["k"], s["wk"]), cos, sin, case["rot"], case["interleaved"]).to(BF16).transpose(1, 2)
    v = s["v"].transpose(1, 2)
    return q.contiguous(), k.repeat_interleave(rep, 1).contiguous(), v.repeat_interleave(rep, 1).contiguous()


def _plain_norm_rope_bwd(s, case):
    cos, sin = _angles(s, s["pos"])
    B, n, Hkv, d = s["k"].shape
    rep = case["Hq"] // case["Hkv"] if case["expand"] else 1
    gt = s["dq"].dtype

    def shared(g):  # sum over the query heads that a key/value head was written for
        return g.float().unflatten(1, (Hkv, rep)).sum(2)

    def one(x, w, g):
        g = _rotate(g.transpose(1, 2), cos, -sin, case["rot"], case["interleaved"])  # the rotation's transpose
        x = x.float()
        r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        xh, wg = x * r, g * w.float()
        dw = (g * xh).sum(2).sum(1).sum(0)
        return (r * (wg - xh * (wg * xh).mean(-1, keepdim=True))).to(gt), dw

    dxq, dwq = one(s["q"], s["wq"], s["dq"].float())
    dxk, dwk = one(s["k"], s["wk"], shared(s["dk"]))
    return dxq, dxk, shared(s["dv"]).transpose(1, 2).to(gt).contiguous(), dwq, dwk


def _ancestors(parents):
    """[B, T, T] truth: node j is node i or above it.  (I + A)^T with A[i, parent(i)] = 1 counts walks."""
    B, T = parents.shape
    a = (parents[..., None] == torch.arange(T, device=parents.device)).float()
    return torch.linalg.matrix_power(a + torch.eye(T, device=parents.device), T) > 0


def _plain_append(s, case):
    B, T, Hkv, d = s["k"].shape
    live = torch.arange(T, device=DEV) < s["n_nodes"][:, None]
    pos = s["lens"][:, None] + _ancestors(s["parents"]).sum(-1) - 1
    cos, sin = _angles(s, torch.where(live, pos, 0))
    q = _rotate(_norm(s["q"], s["wq"]), cos, sin, case["rot"], case["interleaved"])
    k = _rotate(_norm(s["k"], s["wk"]), cos, sin, case["rot"], case["interleaved"])
    b, t = live.nonzero(as_tuple=True)
    row = s["lens"][b].long() + t
    s["k_cache"][b, :, row] = k[b, t].to(BF16)
    s["v_cache"][b, :, row] = s["v"][b, t]
    q = torch.where(live[..., None, None], q, 0.0)
    return q.to(BF16).transpose(1, 2).contiguous(), s["k_cache"], s["v_cache"]


def _plain_tree(s, case):
    q, k, v, lens, n = s["q"], s["k_cache"], s["v_cache"], s["lens"], s["n_nodes"]
    B, Hq, T, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    j = torch.arange(Nk, device=DEV) - lens[:, None]  # node index of each cache row (negative: cached)
    node = (j >= 0) & (j < n[:, None])
    anc = _ancestors(s["parents"])
    vis = torch.gather(anc, 2, j.clamp(0, T - 1)[:, None, :].expand(B, T, Nk)) & node[:, None] | (j < 0)[:, None]
    vis &= (torch.arange(T, device=DEV) < n[:, None])[..., None]
    qs = q.float().unflatten(1, (Hkv, Hq // Hkv)).flatten(2, 3) * (1.0 / math.sqrt(d))
    sc = qs @ k.float().transpose(2, 3)
    sc = sc.unflatten(2, (Hq // Hkv, T)).masked_fill_(~vis[:, None, None], -math.inf).flatten(2, 3)
    m = sc.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = sc.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p @ v.float()) / torch.where(l > 0, l, 1.0)
    lse = (m + l.log()).squeeze(-1)
    return o.reshape(B, Hq, T, d).to(BF16), lse.reshape(B, Hq, T)


def _plain_compact(s, case):
    L, B, H, Nk, d = s["k_cache"].shape
    T = s["accepted"].shape[1]
    b, i = (torch.arange(T, device=DEV) < s["n_accepted"][:, None]).nonzero(as_tuple=True)
    src = s["lens"][b].long() + s["accepted"][b, i]
    dst = s["lens"][b].long() + i
    s["k_cache"][:, b, :, dst] = s["k_cache"][:, b, :, src]
    s["v_cache"][:, b, :, dst] = s["v_cache"][:, b, :, src]
    return s["k_cache"], s["v_cache"], s["lens"] + s["n_accepted"]


PLAIN = {"norm_rope": _plain_norm_rope, "norm_rope_bwd": _plain_norm_rope_bwd, "append": _plain_append,
         "tree": _plain_tree, "compact": _plain_compact}


# ------------------------------------------------------------------------------------- own kernels
def _own(s, case):
    import exact_tiled_attention_fa_gb300 as fa
    op = case["op"]
    if op == "norm_rope":
        return fa.qk_norm_rope(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["cos"], s["sin"], positions=s["pos"], eps=EPS,
                               interleaved=case["interleaved"], expand=case["expand"])
    if op == "norm_rope_bwd":
        if "ws" not in s:
            s["ws"] = torch.empty(fa.qk_norm_rope_bwd_workspace_size(case["d"]), dtype=torch.uint8, device=DEV)
        return fa.qk_norm_rope_bwd(s["dq"], s["dk"], s["dv"], s["q"], s["k"], s["wq"], s["wk"], s["cos"], s["sin"],
                                   positions=s["pos"], eps=EPS, interleaved=case["interleaved"], expand=case["expand"],
                                   out_dtype=s["dq"].dtype, workspace=s["ws"])
    if op == "append":
        q = fa.qk_norm_rope_append(s["q"], s["k"], s["v"], s["wq"], s["wk"], s["cos"], s["sin"], s["k_cache"], s["v_cache"],
                                   s["lens"], parents=s["parents"], n_nodes=s["n_nodes"], eps=EPS,
                                   interleaved=case["interleaved"])
        return q, s["k_cache"], s["v_cache"]
    if op == "tree":
        if "ws" not in s:
            size = fa.decode_tree_workspace_size(case["Hq"], case["Hkv"], case["T"], case["d"], fa.num_sms())
            s["ws"] = torch.empty(size, dtype=torch.uint8, device=DEV)
        return fa.decode_tree(s["q"], s["k_cache"], s["v_cache"], s["lens"], parents=s["parents"], n_nodes=s["n_nodes"],
                              workspace=s["ws"])
    n = fa.cache_compact(s["k_cache"], s["v_cache"], s["lens"], s["accepted"], s["n_accepted"])
    return s["k_cache"], s["v_cache"], n


def run(state):
    case = state["case"]
    return _own(state, case) if own else PLAIN[case["op"]](state, case)


# ------------------------------------------------------------------------------------------- work
def work(case):
    op = case["op"]
    if op in ("norm_rope", "norm_rope_bwd"):
        B, N, Hq, Hkv, d = (case[n] for n in ("B", "N", "Hq", "Hkv", "d"))
        tok, Ho = B * N, Hq if case["expand"] else Hkv
        tables = (N + 256) * case["rot"] * 4 + tok * 4
        if op == "norm_rope":
            return {"bytes": tok * d * 2 * (Hq + 2 * Hkv + Hq + 2 * Ho) + tables, "flops": tok * d * (Hq + Hkv) * 8}
        es = 2 if case["grad"] == "bf16" else 4
        return {"bytes": tok * d * ((Hq + 2 * Ho) * es + (Hq + Hkv) * 2 + (Hq + 2 * Hkv) * es) + tables,
                "flops": tok * d * ((Hq + Hkv) * 16 + (Ho - Hkv) * 2)}
    if op == "append":
        tok = int(_node_ladder(case).sum())
        heads = case["Hq"] + 2 * case["Hkv"]
        return {"bytes": tok * (heads * case["d"] * 4 + case["rot"] * 4), "flops": tok * case["d"] * heads * 8}
    if op == "tree":
        B, T, Hq, Hkv, d = (case[n] for n in ("B", "T", "Hq", "Hkv", "d"))
        hi = min(case["hi"], case["Nk_max"] - T)
        keys = int(torch.linspace(min(case["lo"], hi), hi, B).round().sum()) + int(_node_ladder(case).sum())
        return {"bytes": keys * Hkv * d * 4 + B * Hq * T * (d * 4 + 4), "flops": 4.0 * d * (Hq // Hkv) * T * Hkv * keys}
    # a path of a random recursive tree holds about the harmonic number of T nodes
    rows = case["B"] * max(1.0, math.log(case["T"]))
    return {"bytes": case["L"] * rows * case["Hkv"] * case["d"] * 2 * 4, "flops": 0}


# ------------------------------------------------------------------------------------------ exact
def _exact_fn(x, w, cos, sin, rot, interleaved):
    """Norm and rotation of x [B, n, H, d] in fp64, the rotation as a product of complex numbers."""
    y = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt() * w
    turn = torch.complex(cos, sin)[:, :, None]
    pairs = y[..., :rot].unflatten(-1, (rot // 2, 2) if interleaved else (2, rot // 2))
    pairs = pairs if interleaved else pairs.transpose(-1, -2)
    z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
    z = z if interleaved else z.transpose(-1, -2)
    return torch.cat((z.flatten(-2), y[..., rot:]), -1)


def _exact_paths(parents, n):
    """Each used node's path from the root (node last)."""
    paths = []
    for t in range(n):
        p = int(parents[t])
        paths.append((paths[p] if p >= 0 else []) + [t])
    return paths


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("norm_rope", "norm_rope_bwd"):
        cos, sin = s["cos"].double()[s["pos"].long()], s["sin"].double()[s["pos"].long()]
        x = [s[n].double().requires_grad_() for n in ("q", "k", "v", "wq", "wk")]
        rep = case["Hq"] // case["Hkv"] if case["expand"] else 1
        y = [_exact_fn(x[0], x[3], cos, sin, case["rot"], case["interleaved"]),
             _exact_fn(x[1], x[4], cos, sin, case["rot"], case["interleaved"]), x[2]]
        y = [y[0].permute(0, 2, 1, 3)] + [torch.stack([t] * rep, 3).flatten(2, 3).permute(0, 2, 1, 3) for t in y[1:]]
        if op == "norm_rope":
            return tuple(t.detach() for t in y)
        return torch.autograd.grad(y, x, [s[n].double() for n in ("dq", "dk", "dv")])
    if op == "append":
        B, T, Hq, d = s["q"].shape
        q = torch.zeros((B, T, Hq, d), dtype=torch.float64, device=DEV)
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        par, lens, cnt = s["parents"].tolist(), s["lens"].tolist(), s["n_nodes"].tolist()
        for b in range(B):
            n, at = cnt[b], lens[b]
            pos = torch.tensor([[at + len(p) - 1 for p in _exact_paths(par[b], n)]], device=DEV)
            cos, sin = s["cos"].double()[pos], s["sin"].double()[pos]
            q[b, :n] = _exact_fn(s["q"][b:b + 1, :n].double(), s["wq"].double(), cos, sin, case["rot"], case["interleaved"])[0]
            k = _exact_fn(s["k"][b:b + 1, :n].double(), s["wk"].double(), cos, sin, case["rot"], case["interleaved"])[0]
            kc[b, :, at:at + n] = k.permute(1, 0, 2)
            vc[b, :, at:at + n] = s["v"][b, :n].double().permute(1, 0, 2)
        return q.permute(0, 2, 1, 3), kc, vc
    if op == "tree":
        B, Hq, T, d = s["q"].shape
        R = Hq // case["Hkv"]
        o = torch.zeros((B, Hq, T, d), dtype=torch.float64, device=DEV)
        lse = torch.full((B, Hq, T), -math.inf, dtype=torch.float64, device=DEV)
        par, lens, cnt = s["parents"].tolist(), s["lens"].tolist(), s["n_nodes"].tolist()
        for b in range(B):
            at, n = lens[b], cnt[b]
            see = torch.zeros((n, at + n), dtype=torch.bool)
            see[:, :at] = True
            for t, path in enumerate(_exact_paths(par[b], n)):
                see[t, [at + p for p in path]] = True
            see = see.to(DEV)
            for h in range(Hq):
                k, v = (s[c][b, h // R, :at + n].double() for c in ("k_cache", "v_cache"))
                sc = torch.where(see, s["q"][b, h, :n].double() @ k.T / d ** 0.5, -math.inf)
                lse[b, h, :n] = torch.logsumexp(sc, -1)
                o[b, h, :n] = torch.softmax(sc, -1) @ v
        return o, lse
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    lens, acc, cnt = s["lens"].tolist(), s["accepted"].tolist(), s["n_accepted"].tolist()
    for b in range(case["B"]):
        for c in (kc, vc):
            kept = [c[:, b, :, lens[b] + t].clone() for t in acc[b][:cnt[b]]]
            for i, row in enumerate(kept):
                c[:, b, :, lens[b] + i] = row
    return kc, vc, s["lens"] + s["n_accepted"]
