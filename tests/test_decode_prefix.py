"""fa_decode_prefix against the plain fp64 form, at the sizes and lengths where it can go wrong."""
from __future__ import annotations

import math

import pytest
import torch

from tests.rules_reference import HALF_BF16, F64, Rules, check_forward, scores

BF16, F32 = torch.bfloat16, torch.float32
DEV = "cuda"
pytestmark = pytest.mark.gpu


def fa():
    import exact_tiled_attention_fa_gb300 as m
    return m


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


def slopes(Hq):
    return torch.exp2(-8.0 * torch.arange(1, Hq + 1) / Hq).float()


def inputs(B, Hq, Hkv, P_max, Nk_max, d, lens, P=None, seed=0, gain=1.0, fill=math.nan):
    """q, prefix, caches; rows behind the lengths hold `fill`."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g).to(BF16)  # noqa: E731
    q = (gain * torch.randn((B, Hq, 1, d), generator=g)).to(BF16)
    kp, vp, k, v = r(Hkv, P_max, d), r(Hkv, P_max, d), r(B, Hkv, Nk_max, d), r(B, Hkv, Nk_max, d)
    if P is not None:
        kp[:, P:], vp[:, P:] = fill, fill
    for b in range(B):
        k[b, :, int(lens[b]):], v[b, :, int(lens[b]):] = fill, fill
    return q, kp, vp, k, v


def reference(q, kp, vp, k, v, lens, P, rules):
    B, Hq, _, d = q.shape
    Hkv = k.shape[1]
    R = Hq // Hkv
    r = dict(O=torch.zeros((B, Hq, 1, d), dtype=F64), dO=torch.zeros((B, Hq, 1, d), dtype=F64),
             L=torch.full((B, Hq, 1), -math.inf, dtype=F64), dL=torch.zeros((B, Hq, 1), dtype=F64))
    for b in range(B):
        n = int(lens[b])
        if P + n == 0:
            continue
        for h in range(Hq):
            K = torch.cat((kp[h // R, :P], k[b, h // R, :n])).to(F64)
            V = torch.cat((vp[h // R, :P], v[b, h // R, :n])).to(F64)
            s, _, e = scores(q[b, h].to(F64), K, rules, rules.slopes[h] if rules.slopes is not None else None, 1, P + n)
            p = torch.softmax(s, -1)
            E = (p * e).sum(-1, keepdim=True)
            r["O"][b, h] = p @ V
            r["dO"][b, h] = (p * (HALF_BF16 + e + E + 2.0 ** -20)) @ V.abs()
            r["L"][b, h] = torch.logsumexp(s, -1)
            r["dL"][b, h] = E[:, 0] + 2.0 ** -20 * (1 + r["L"][b, h].abs())
    return r


def call(q, kp, vp, k, v, lens, plen=None, rules=Rules(), **kw):
    to = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    o, lse = fa().decode_prefix(to(q), to(kp), to(vp), to(k), to(v), to(lens), prefix_len=to(plen), scale=rules.scale,
                                softcap=rules.cap, slopes=to(rules.slopes), **kw)
    torch.cuda.synchronize()
    return o, lse


def check(B, Hq, Hkv, P_max, Nk_max, d, lens, P=None, rules=Rules(), seed=0, what="", dtypes=(F32,)):
    x = inputs(B, Hq, Hkv, P_max, Nk_max, d, lens, P, seed, 3.0 if rules.cap else 1.0)
    ref = reference(*x, lens, P_max if P is None else P, rules)
    for dt in dtypes:
        o, lse = call(*x, lens, None if P is None else i32(P), rules, out_dtype=dt)
        assert fa().get_device_error() == 0
        check_forward(o, lse, ref, what)
    return x, ref


RULES = {"none": lambda Hq: Rules(), "cap": lambda Hq: Rules(softcap=6.0), "bias": lambda Hq: Rules(slopes=slopes(Hq)),
         "both": lambda Hq: Rules(scale=0.3, softcap=20.0, slopes=slopes(Hq))}


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("name", list(RULES))
@pytest.mark.parametrize("R", [1, 3, 4, 8])
def test_groups_and_lengths(d, name, R):
    """Up to 128 rows meet the prefix (one launch for both sides); own lengths none, one, at and beside a tile's end."""
    lens = i32(0, 1, 127, 128, 129, 300, 64)
    check(7, 2 * R, 2, 500, 300, d, lens, rules=RULES[name](2 * R), seed=R, what=f"{d} {name} {R}", dtypes=(F32, BF16))


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("B,R", [(129, 1), (40, 4), (17, 8), (70, 5), (300, 2), (5, 100), (2, 128), (3, 65)])
def test_more_rows_than_a_tile(d, B, R):
    """The prefix in a launch of its own, one or two query tiles to a unit, the last ones partly or wholly without rows."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, 200, (B,), generator=g).to(torch.int32)
    lens[0] = 0
    rules = Rules(softcap=10.0, slopes=slopes(R)) if B % 2 else Rules()
    check(B, R, 1, 700, 200, d, lens, rules=rules, seed=R, what=f"{d} {B} {R}")


@pytest.mark.parametrize("name,P", [("none", 20011), ("both", 20011), ("bias", 9000)])
def test_long_prefix_for_several_query_tiles(name, P):
    """Query tiles that come to the same prefix later begin further on in it and go round; its last tile is cut."""
    lens = torch.arange(34, dtype=torch.int32) * 7 % 60
    check(34, 16, 2, P + 30, 60, 128, lens, P=P, rules=RULES[name](16), seed=P, what=f"{name} {P}")


@pytest.mark.parametrize("P,P_max", [(0, 64), (1, 64), (127, 300), (128, 128), (129, 300), (4000, 4001)])
@pytest.mark.parametrize("B", [3, 60])
def test_prefix_lengths(P, P_max, B):
    """A prefix of no, one and many tokens behind which anything may stand; sequences with nothing of their own."""
    lens = torch.arange(B, dtype=torch.int32) * 5 % 77
    x, ref = check(B, 8, 2, P_max, 77, 64, lens, P=P, rules=Rules(slopes=slopes(8)), seed=P, what=f"{P}/{P_max}")
    if P == 0:
        o, lse = call(*x, lens, i32(0))
        assert bool((o[0] == 0).all()) and bool(torch.isneginf(lse[0]).all())


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("B,Hkv,hi", [(1, 1, 1), (5, 2, 400), (200, 4, 300), (3, 1, 9000)])
def test_without_a_prefix(d, B, Hkv, hi):
    """None for the prefix: decode over the caches alone, units of one and of many shares."""
    g = torch.Generator().manual_seed(hi)
    lens = torch.randint(0, hi + 1, (B,), generator=g).to(torch.int32)
    lens[0] = hi
    Hq = 4 * Hkv
    q, _, _, k, v = inputs(B, Hq, Hkv, 1, hi, d, lens, seed=d)
    rules = Rules(softcap=15.0)
    none = torch.zeros((Hkv, 0, d), dtype=BF16)
    ref = reference(q, none, none, k, v, lens, 0, rules)
    o, lse = call(q, None, None, k, v, lens, rules=rules, out_dtype=F32)
    assert fa().get_device_error() == 0
    check_forward(o, lse, ref, f"{B} {Hkv} {hi}")
    o, lse = call(q, None, None, k, v, lens, rules=rules)
    check_forward(o, lse, ref, f"{B} {Hkv} {hi} bf16")


@pytest.mark.parametrize("B,Hkv,P,hi", [(330, 4, 200, 500), (64, 8, 3000, 1500), (16, 8, 20000, 100), (2, 8, 600, 100), (100, 1, 30000, 40)])
def test_shares_cross_units(B, Hkv, P, hi):
    """Many units on a CTA, units over many CTAs; the same from run to run."""
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, hi + 1, (B,), generator=g).to(torch.int32)
    x, _ = check(B, 2 * Hkv, Hkv, P, hi, 64, lens, seed=B, what=f"{B} {Hkv} {P}")
    o, lse = call(*x, lens, out_dtype=F32)
    for _ in range(3):
        o2, lse2 = call(*x, lens, out_dtype=F32)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_lengths_out_of_range_are_clamped_and_recorded():
    x = inputs(3, 4, 2, 200, 100, 64, i32(100, 0, 50), seed=3)
    for lens, plen, good, P in ((i32(101, -4, 50), None, i32(100, 0, 50), 200), (i32(100, 0, 50), i32(201), i32(100, 0, 50), 200),
                                (i32(100, 0, 50), i32(-1), i32(100, 0, 50), 0)):
        fa().get_device_error()
        o, lse = call(*x, lens, plen, out_dtype=F32)
        assert fa().get_device_error() == fa().FA_ERR_INVALID_ARG
        check_forward(o, lse, reference(*x, good, P, Rules()), "clamped")


def test_capped_scores_in_both_forms_of_tanh():
    lens = i32(130, 40, 0, 77)
    q, kp, vp, k, v = inputs(4, 8, 2, 300, 130, 128, lens, seed=4)
    q = (q.float() * torch.logspace(-3, 3, 4)[:, None, None, None]).to(BF16)
    for cap in (1e-3, 5.0, 1e4):
        rules = Rules(softcap=cap)
        o, lse = call(q, kp, vp, k, v, lens, rules=rules, out_dtype=F32)
        check_forward(o, lse, reference(q, kp, vp, k, v, lens, 300, rules), f"cap {cap}")


def test_rows_past_32_bit_offsets():
    """Caches of more than 2^31 elements: the last sequence's last head, against the same rows in a small cache."""
    B, Hq, Hkv, P, Nk, d = 3, 16, 8, 300, 1 << 20, 128
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB")
    lens = i32(5, Nk, 333)
    kc, vc = (torch.zeros((B, Hkv, Nk, d), dtype=BF16, device=DEV) for _ in range(2))
    g = torch.Generator().manual_seed(8)
    r = lambda *s: torch.randn(s, generator=g).to(BF16)  # noqa: E731
    q, kp, vp, k, v = r(B, Hq, 1, d), r(Hkv, P, d), r(Hkv, P, d), r(B, Hkv, 400, d), r(B, Hkv, 400, d)
    kc[:, :, :400], vc[:, :, :400] = k.to(DEV), v.to(DEV)
    o, lse = call(q, kp, vp, kc, vc, lens, out_dtype=F32)
    assert kc.numel() > 1 << 31 and fa().get_device_error() == 0
    short = i32(5, 333, 333)
    ref = reference(q, kp, vp, k, v, short, P, Rules())
    for b in (0, 2):
        check_forward(o[b:b + 1], lse[b:b + 1], {n: t[b:b + 1] for n, t in ref.items()}, f"{b}")
    # sequence 1: 400 keys, and zeros' weights e^0 behind them
    s = torch.einsum("hd,hkd->hk", q[1, :, 0].double(), torch.cat((kp, k[1]), 1).repeat_interleave(2, 0).double()) / d ** 0.5
    want = torch.logsumexp(torch.cat((s, torch.full((Hq, 1), math.log(Nk - 400.0))), 1).double(), 1)
    assert float((lse[1, :, 0].double().cpu() - want).abs().max()) < 1e-4


@pytest.mark.parametrize("B,R,P,Nk,d", [(3, 4, 1000, 300, 32), (3, 4, 1000, 300, 64), (80, 4, 600, 300, 64), (3, 4, 1000, 300, 128),
                                        (40, 8, 500, 300, 128)])
def test_wait_limit_is_reported_and_the_next_call_is_right(B, R, P, Nk, d):
    """With a limit of 1 ns waits run out in each form of the kernel: the status says so, every role ends, the merge
    follows no record that was not written, and the next call is right."""
    lens = torch.arange(B, dtype=torch.int32) % (Nk + 1)
    Hq, Hkv = 4 * R, 4
    x = inputs(B, Hq, Hkv, P, Nk, d, lens, seed=9)
    ws = torch.full((fa().decode_prefix_workspace_size(B, Hq, Hkv, d, fa().num_sms()),), 0x7F, dtype=torch.uint8, device=DEV)
    for junk in (0x7F, 0xFF, 0x01):
        ws.fill_(junk)
        fa().set_wait_timeout_ns(1)
        try:
            call(*x, lens, workspace=ws)
            status = fa().get_device_error()
        finally:
            fa().set_wait_timeout_ns(0)
        assert status == fa().FA_ERR_TIMEOUT
    o, lse = call(*x, lens, out_dtype=F32, workspace=ws)
    assert fa().get_device_error() == 0
    check_forward(o, lse, reference(*x, lens, P, Rules()), "after")


def test_outputs_and_workspace_given():
    B, Hq, Hkv, P, Nk, d = 50, 16, 4, 333, 90, 128
    lens = torch.arange(B, dtype=torch.int32) % 91
    x = [t.to(DEV) for t in inputs(B, Hq, Hkv, P, Nk, d, lens, seed=5)]
    n = lens.to(DEV)
    need = fa().decode_prefix_workspace_size(B, Hq, Hkv, d, fa().num_sms())
    for dt in (BF16, F32):
        for pre in (True, False):
            a = (x[0], x[1] if pre else None, x[2] if pre else None, x[3], x[4], n)
            ws = torch.full((need + 4096,), 0xAB, dtype=torch.uint8, device=DEV)
            out = torch.full((x[0].numel() + 512,), 7.0, dtype=dt, device=DEV)
            lse = torch.full((B * Hq + 64,), 7.0, device=DEV)
            r = fa().decode_prefix(*a, out=out[:x[0].numel()].view(x[0].shape), lse=lse[:B * Hq].view(B, Hq, 1), workspace=ws[:need])
            want = fa().decode_prefix(*a, out_dtype=dt)
            assert torch.equal(r[0], want[0]) and torch.equal(r[1], want[1])
            assert bool((ws[need:] == 0xAB).all()) and bool((out[x[0].numel():] == 7).all()) and bool((lse[B * Hq:] == 7).all())
            o, none = fa().decode_prefix(*a, out_dtype=dt, return_lse=False, workspace=ws[:need])
            assert none is None and torch.equal(o, want[0])


def test_captured_with_lengths_that_grow():
    """A captured step replayed while the lengths and the prefix's grow, on a stream of its own."""
    B, Hq, Hkv, P, Nk, d = 40, 16, 4, 600, 300, 64
    lens = torch.arange(B, dtype=torch.int32) * 3
    x = inputs(B, Hq, Hkv, P, Nk, d, i32(*[Nk] * B), seed=6)
    rules = Rules(softcap=30.0, slopes=slopes(Hq))
    y = [t.to(DEV) for t in x]
    n, plen, sl = lens.to(DEV), i32(100).to(DEV), rules.slopes.to(DEV)
    ws = torch.empty(fa().decode_prefix_workspace_size(B, Hq, Hkv, d, fa().num_sms()), dtype=torch.uint8, device=DEV)
    step = lambda: fa().decode_prefix(*y, n, prefix_len=plen, softcap=30.0, slopes=sl, out_dtype=F32, workspace=ws)  # noqa: E731
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
        st.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            o, lse = step()
        for i in range(3):
            graph.replay()
            st.synchronize()
            check_forward(o, lse, reference(*x, lens + 60 * i, 100 + 250 * i, rules), f"step {i}")
            n += 60
            plen += 250
    assert fa().get_device_error() == 0


def test_prompt_then_tokens():
    """As it is served: the prompt's keys made by qk_norm_rope, each new token appended behind it, decoded behind the shared
    prompt; what fwd_rules gives over the whole of each sequence's tokens."""
    B, Hq, Hkv, d, P, steps = 3, 8, 2, 64, 150, 4
    g = torch.Generator().manual_seed(7)
    w = torch.ones(d, device=DEV)
    ang = torch.arange(P + steps)[:, None] * 10000.0 ** (-torch.arange(d // 2) / (d // 2))
    cos, sin = ang.cos().float().to(DEV), ang.sin().float().to(DEV)
    split = lambda t: (t[:, :, :Hq], t[:, :, Hq:Hq + Hkv], t[:, :, Hq + Hkv:])  # noqa: E731
    prompt = torch.randn((1, P, Hq + 2 * Hkv, d), generator=g).to(BF16).to(DEV)
    new = torch.randn((B, steps, Hq + 2 * Hkv, d), generator=g).to(BF16).to(DEV)
    rules = dict(softcap=8.0, slopes=slopes(Hq).to(DEV))
    # every sequence in full
    x = torch.cat((prompt.expand(B, -1, -1, -1), new), 1).contiguous()
    q, k, v = fa().qk_norm_rope(*split(x), w, w, cos, sin)
    want, want_lse = fa().fwd_rules(q, k, v, causal=True, out_dtype=F32, **rules)
    # the prompt once, then token by token (positions go on behind the prompt)
    _, kp, vp = fa().qk_norm_rope(*split(prompt), w, w, cos, sin)
    kc = torch.zeros((B, Hkv, steps, d), dtype=BF16, device=DEV)
    vc = torch.zeros_like(kc)
    n = torch.zeros(B, dtype=torch.int32, device=DEV)
    for t in range(steps):
        qt = fa().qk_norm_rope_append(*split(new[:, t:t + 1].contiguous()), w, w, cos[P:].contiguous(), sin[P:].contiguous(), kc, vc, n)
        n += 1
        o, lse = fa().decode_prefix(qt, kp[0], vp[0], kc, vc, n, out_dtype=F32, **rules)
        # the two round weights at other maxima: 2^-8 of each
        assert float((o - want[:, :, P + t:P + t + 1]).abs().max()) < 2.0 ** -7 * float(v.float().abs().max())
        assert float((lse - want_lse[:, :, P + t:P + t + 1]).abs().max()) < 1e-4
    assert fa().get_device_error() == 0
