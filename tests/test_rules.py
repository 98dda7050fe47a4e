"""fa_fwd_rules and fa_bwd_rules against the plain fp64 form, at the sizes and masks where they can go wrong."""
from __future__ import annotations

import math

import pytest
import torch

from tests.rules_reference import Rules, attention, check_forward, check_gradients, documents, visible

BF16, F32 = torch.bfloat16, torch.float32
DEV = "cuda"


def fa():
    import exact_tiled_attention_fa_gb300 as m
    return m


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


def slopes(Hq):
    return torch.exp2(-8.0 * torch.arange(1, Hq + 1) / Hq).float()


def inputs(B, Hq, Hkv, N, Nk, d, seed=0, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    return (gain * r(B, Hq, N, d)).to(BF16), r(B, Hkv, Nk, d).to(BF16), r(B, Hkv, Nk, d).to(BF16), r(B, Hq, N, d).to(BF16)


def run(q, k, v, do, rules, out_dtype=F32, grad_dtype=F32, **kw):
    q, k, v, do = (t.to(DEV) for t in (q, k, v, do))
    a = rules.kwargs(DEV)
    o, lse = fa().fwd_rules(q, k, v, out_dtype=out_dtype, **a, **kw)
    grads = fa().bwd_rules(q, k, v, o, lse, do, out_dtype=grad_dtype, **a)
    torch.cuda.synchronize()
    return o, lse, grads


def check_all(shape, rules, seed=0, gain=1.0, dtypes=((F32, F32),), what=""):
    x = inputs(*shape, seed=seed, gain=gain)
    ref = attention(*x[:3], rules, x[3])
    for od, gd in dtypes:
        o, lse, grads = run(*x, rules, od, gd)
        assert fa().get_device_error() == 0
        check_forward(o, lse, ref, what)
        check_gradients(grads, ref, what)
    return ref


# ------------------------------------------------------------------------------------ the reference itself
@pytest.mark.parametrize("rules", [
    Rules(causal=True, softcap=2.0), Rules(slopes=torch.tensor([0.3, 0.1])), Rules(causal=True, prefix_lens=i32(4)),
    Rules(causal=True, softcap=1.5, slopes=torch.tensor([0.3, 0.1]), documents=i32(0, 0, 0, 1, 1, -1, 2, 2, 2)[None]),
])
def test_reference_gradients_against_differences(rules):
    """The formula's gradients against central differences of the fp64 forward, and against what autograd makes
    of a softmax written out."""
    N, Nk, d = 7, 9, 4
    g = torch.Generator().manual_seed(1)
    q, k, v, do = (torch.randn(s, generator=g, dtype=torch.float64) for s in ((1, 2, N, d), (1, 1, Nk, d), (1, 1, Nk, d), (1, 2, N, d)))
    ref = attention(q, k, v, rules, do)
    f = lambda *t: float((attention(*t, rules)["O"] * do).sum())  # noqa: E731
    h = 1e-5
    for n, i in (("dq", 0), ("dk", 1), ("dv", 2)):
        x = [q, k, v]
        for at in [(0, 0, 0, 1), (0, 0, 4, 2), (0, 0, 6, 0)]:
            lo, hi = [t.clone() for t in x], [t.clone() for t in x]
            lo[i][at] -= h
            hi[i][at] += h
            diff = (f(*hi) - f(*lo)) / (2 * h)
            assert abs(diff - float(ref[n][at])) < 1e-8 * (1 + abs(diff)), (n, at)
    assert torch.equal(visible(3, 4, True), torch.tensor([[1, 1, 0, 0], [1, 1, 1, 0], [1, 1, 1, 1]], dtype=torch.bool))


# ------------------------------------------------------------------------------------ sizes and rules
def rule_set(name, B, Hq, N, Nk):
    docs = documents(B, Nk, [37, 1, 130, 5, 200], pads=[(17 * b) % 40 % max(1, Nk // 2) for b in range(B)])
    pre = torch.tensor([(b * Nk) // max(1, B - 1) if B > 1 else Nk // 2 for b in range(B)], dtype=torch.int32)
    return {
        "none": Rules(), "causal": Rules(causal=True),
        "cap": Rules(causal=True, softcap=5.0), "bias": Rules(slopes=slopes(Hq)), "causal_bias": Rules(causal=True, slopes=slopes(Hq)),
        "prefix": Rules(causal=True, prefix_lens=pre), "prefix_bias": Rules(causal=True, prefix_lens=pre, slopes=slopes(Hq)),
        "docs": Rules(causal=True, documents=docs), "docs_full": Rules(documents=docs, softcap=20.0),
        "all": Rules(causal=True, scale=0.2, softcap=8.0, slopes=slopes(Hq), documents=docs, prefix_lens=pre),
    }[name]


SHAPES = [(2, 2, 1, 1, 1), (2, 3, 1, 1, 300), (3, 4, 2, 77, 513), (2, 2, 2, 300, 300), (2, 4, 1, 513, 200), (3, 2, 1, 129, 129),
          (1, 6, 2, 256, 384), (2, 2, 1, 640, 640)]


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["none", "causal", "cap", "bias", "causal_bias", "prefix", "prefix_bias", "docs", "docs_full", "all"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_rules_and_sizes(name, d):
    for i, (B, Hq, Hkv, N, Nk) in enumerate(SHAPES):
        rules = rule_set(name, B, Hq, N, Nk)
        dtypes = ((F32, F32), (BF16, BF16)) if i in (2, 3) else ((F32, F32),)
        check_all((B, Hq, Hkv, N, Nk, d), rules, seed=i, gain=3.0 if rules.cap else 1.0, dtypes=dtypes, what=f"{name} {SHAPES[i]} d={d}")


@pytest.mark.gpu
@pytest.mark.parametrize("d,causal", [(64, True), (64, False), (128, True)])
def test_documents_at_tile_borders_and_beyond_a_look(d, causal):
    """Documents that begin and end at, before and behind a tile's border, of one position, and longer than the 2048
    numbers the ranges kernel looks at in one go; a sequence of padding alone; one whose first document is padding."""
    Nk = 5003
    ids = torch.full((4, Nk), 3, dtype=torch.int32)
    for b, cuts in enumerate([[127, 128, 129, 4224, 4225], [1, 2100, 2101, 4993], [], [128, 256, 2304, 2432]]):
        for n, c in enumerate(cuts):
            ids[b, c:] = n + 4
    ids[2] = -5
    ids[3, :128] = -1
    ids[3, 2304:2432] = -7
    check_all((4, 2, 1, Nk, Nk, d), Rules(causal=causal, documents=ids), seed=d, what="borders")
    # fewer queries than keys, and more: their positions decide
    check_all((4, 2, 1, 300, Nk, d), Rules(causal=causal, documents=ids), seed=d + 1, what="last queries")
    check_all((4, 2, 1, 700, 500, d), Rules(causal=causal, documents=ids[:, 2000:2500].contiguous()), seed=d + 2, what="more queries")


@pytest.mark.gpu
def test_one_number_in_two_runs_is_two_documents():
    ids = torch.zeros((1, 300), dtype=torch.int32)
    ids[0, 100:110] = 1
    check_all((1, 1, 1, 300, 300, 64), Rules(documents=ids), what="runs")


@pytest.mark.gpu
@pytest.mark.parametrize("d", [32, 128])
def test_cap_over_its_whole_range(d):
    """Scores from far inside the cap's linear part to far beyond it: both forms of tanh, and rows that mix them."""
    B, Hq, Hkv, N, Nk = 1, 2, 1, 200, 260
    q, k, v, do = inputs(B, Hq, Hkv, N, Nk, d, seed=3)
    q = (q.float() * torch.logspace(-3, 3, N)[None, None, :, None]).to(BF16)
    for cap in (1e-3, 1.0, 30.0, 1e4):
        rules = Rules(softcap=cap)
        ref = attention(q, k, v, rules, do)
        o, lse, grads = run(q, k, v, do, rules)
        check_forward(o, lse, ref, f"cap {cap}")
        # a gradient of q is as large as 1 / |q|'s scale allows: the bound's 1e-4 is for magnitudes of 1
        check_gradients(grads, ref, f"cap {cap}")


@pytest.mark.gpu
@pytest.mark.parametrize("cap", [1e5, 1e7, 1e30])
def test_cap_far_above_the_scores(cap):
    """A cap that none of the scores comes near leaves them as they are.  The bounds are those without a cap: they take
    the products' 2^-24 d |q| |k| four times over, and the cap's 1.2e-6 of a score is less than one of these times."""
    q, k, v, do = inputs(2, 4, 2, 200, 260, 64, seed=21)
    for sl in (None, slopes(4)):
        ref = attention(q, k, v, Rules(causal=True, slopes=sl), do)
        o, lse, grads = run(q, k, v, do, Rules(causal=True, softcap=cap, slopes=sl))
        check_forward(o, lse, ref, f"cap {cap}")
        check_gradients(grads, ref, f"cap {cap}")


@pytest.mark.gpu
def test_capped_scores_that_overflow():
    """q . k beyond fp32's range: the cap makes it +-cap."""
    q, k, v, _ = inputs(1, 1, 1, 130, 140, 64, seed=4)
    q, k = (q.float().sign() * 2.0 ** 100).to(BF16), (k.float().sign() * 2.0 ** 60).to(BF16)
    k[0, 0, :, 1:] = 0  # one product each: no infinity less infinity
    q[0, 0, 5] = 0
    ref = attention(q, k, v, Rules(softcap=10.0))
    ref["dO"] = ref["O"].abs() * 0 + 2.0 ** -6  # (the bound above goes by |q| |k|; weights here are e^+-10 or equal)
    o, lse = fa().fwd_rules(q.to(DEV), k.to(DEV), v.to(DEV), softcap=10.0, out_dtype=F32)
    assert bool(torch.isfinite(o).all())
    assert float((o.double().cpu() - ref["O"]).abs().max()) < 2.0 ** -6 * float(v.abs().max())
    assert float((lse.double().cpu() - ref["L"]).abs().max()) < 1e-4


@pytest.mark.gpu
@pytest.mark.parametrize("d", [32, 64, 128])
def test_hidden_keys_may_hold_anything_in_the_forward(d):
    """Scores of hidden keys are NaN or infinite: in another document, and behind a causal position."""
    B, Hq, Hkv, N, Nk = 2, 2, 1, 330, 330
    q, k, v, _ = inputs(B, Hq, Hkv, N, Nk, d, seed=5)
    ids = torch.zeros((B, Nk), dtype=torch.int32)
    ids[0, 150:], ids[1, 128:] = 1, 1
    rules = Rules(causal=True, softcap=9.0, documents=ids, slopes=slopes(Hq))
    clean = attention(q, k, v, rules)
    for bad in (math.nan, math.inf, -math.inf):
        kk = k.clone()
        for b, first in enumerate((150, 128)):
            kk[b, :, :first] = bad
        o, lse = fa().fwd_rules(q.to(DEV), kk.to(DEV), v.to(DEV), out_dtype=F32, **rules.kwargs(DEV))
        for b, first in enumerate((150, 128)):
            ref = {n: t[b:b + 1, :, first:] for n, t in clean.items()}
            check_forward(o[b:b + 1, :, first:], lse[b:b + 1, :, first:], ref, f"d={d} {bad}")
    kk = k.clone()
    kk[:, :, -1] = math.nan  # the last key is seen by the last query alone
    o, lse = fa().fwd_rules(q.to(DEV), kk.to(DEV), v.to(DEV), causal=True, out_dtype=F32)
    ref = attention(q[:, :, :-1], k[:, :, :-1], v[:, :, :-1], Rules(causal=True))
    check_forward(o[:, :, :-1], lse[:, :, :-1], ref, "last key")
    assert bool(o[:, :, -1].isnan().all()) and bool(lse[:, :, -1].isnan().all())


@pytest.mark.gpu
def test_scores_far_below_zero():
    """Rows whose every score is far below the 0 that a key past the end would have."""
    q, k, v, do = inputs(1, 2, 1, 140, 150, 64, seed=6)
    k, q = (0.1 * k.float() - 20.0).to(BF16), (0.1 * q.float() + 20.0).to(BF16)
    check_all_given(q, k, v, do, Rules(), "low")
    check_all_given(q, k, v, do, Rules(softcap=300.0, causal=True), "low capped")


def check_all_given(q, k, v, do, rules, what):
    ref = attention(q, k, v, rules, do)
    o, lse, grads = run(q, k, v, do, rules)
    check_forward(o, lse, ref, what)
    check_gradients(grads, ref, what)


@pytest.mark.gpu
def test_prefix_out_of_range_is_clamped_and_recorded():
    for bad in (-1, 301):
        q, k, v, do = inputs(2, 2, 2, 300, 300, 64, seed=7)
        rules = Rules(causal=True, prefix_lens=i32(40, bad))
        ref = attention(q, k, v, rules, do)
        fa().get_device_error()
        o, lse, grads = run(q, k, v, do, rules)
        assert fa().get_device_error() == fa().FA_ERR_INVALID_ARG
        check_forward(o, lse, ref, "prefix")
        check_gradients(grads, ref, "prefix")


# ------------------------------------------------------------------------------------ division of the work
@pytest.mark.gpu
@pytest.mark.parametrize("B,Hq,Hkv,N,d", [(1, 8, 1, 300, 64), (1, 8, 1, 300, 128), (1, 7, 1, 150, 32), (1, 3, 3, 1000, 64), (40, 8, 2, 300, 32),
                                          (13, 16, 16, 260, 64)])
def test_parts_and_rounds(B, Hq, Hkv, N, d):
    """A group's query heads in one item and divided over several, fewer items than CTAs and several rounds of them."""
    docs = documents(B, N, [90, 140, 30, 7])
    for rules in (Rules(causal=True, softcap=10.0), Rules(documents=docs), Rules(causal=True, documents=docs, slopes=slopes(Hq))):
        check_all((B, Hq, Hkv, N, N, d), rules, seed=B, dtypes=((BF16, BF16), (F32, F32)), what=f"{B, Hq, Hkv, N, d}")


@pytest.mark.gpu
def test_the_same_from_run_to_run():
    x = inputs(3, 8, 2, 1000, 1000, 64, seed=8)
    rules = Rules(causal=True, softcap=20.0, slopes=slopes(8), documents=documents(3, 1000, [300, 10, 450]))
    o, lse, (dq, dk, dv) = run(*x, rules)
    for _ in range(3):
        o2, lse2, (dq2, dk2, dv2) = run(*x, rules)
        assert torch.equal(o, o2) and torch.equal(lse, lse2) and torch.equal(dk, dk2) and torch.equal(dv, dv2)
        assert float((dq - dq2).abs().max()) < 1e-5


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_without_rules_as_the_plain_forward(d, causal):
    """The same arithmetic in the same order as fwd."""
    q, k, v, _ = (t.to(DEV) for t in inputs(2, 4, 4, 500, 500, d, seed=9))
    o, lse = fa().fwd(q, k, v, causal=causal, out_dtype=F32)
    o2, lse2 = fa().fwd_rules(q, k, v, causal=causal, out_dtype=F32)
    assert float((o - o2).abs().max()) < 2e-6 and float((lse - lse2).abs().max()) < 2e-6


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_slopes_of_every_kind(d, causal):
    """Slopes of none, below zero, so steep that a tile's nearest and furthest key differ by more than 2^64, and just not."""
    sl = torch.tensor([0.0, -0.01, 5.0, 0.34, 0.36, 1e-4])
    pre = i32(0, 200)
    for rules in (Rules(causal=causal, slopes=sl), Rules(causal=causal, slopes=sl, prefix_lens=pre), Rules(causal=causal, slopes=sl, softcap=5.0)):
        check_all((2, 6, 3, 300, 420, d), rules, seed=d, what=f"slopes {d} {causal}")


@pytest.mark.gpu
@pytest.mark.parametrize("causal", [False, True])
def test_many_heads_at_once(causal):
    """More heads than go out at once: several chunks of them, the last tiles ragged.  Against fwd and bwd."""
    B, H, N, d = 21, 10, 2000, 128
    q, k, v, do = (t.to(DEV) for t in inputs(B, H, H, N, N, d, seed=15))
    o, lse = fa().fwd(q, k, v, causal=causal, out_dtype=F32)
    o2, lse2 = fa().fwd_rules(q, k, v, causal=causal, out_dtype=F32)
    assert float((o - o2).abs().max()) < 2e-6 and float((lse - lse2).abs().max()) < 2e-6
    want = fa().bwd(q, k, v, o, lse, do, causal=causal, out_dtype=F32)
    got = fa().bwd_rules(q, k, v, o, lse, do, causal=causal, out_dtype=F32)
    # dq's sums come in any order; dk and dv in another one, of up to 16 tiles of fp32 sums
    for a, b in zip(got, want):
        assert float((a - b).abs().max()) < 2.0 ** -16 * float(b.abs().max())
    # shared heads: a group's gradients are the sums of its heads'
    o3, lse3 = fa().fwd_rules(q, k[:, ::5].contiguous(), v[:, ::5].contiguous(), causal=causal, out_dtype=F32)
    kk, vv = (t[:, ::5].repeat_interleave(5, 1).contiguous() for t in (k, v))
    o4, lse4 = fa().fwd(q, kk, vv, causal=causal, out_dtype=F32)
    assert float((o3 - o4).abs().max()) < 2e-6
    got = fa().bwd_rules(q, k[:, ::5].contiguous(), v[:, ::5].contiguous(), o3, lse3, do, causal=causal, out_dtype=F32)
    want = fa().bwd(q, kk, vv, o4, lse4, do, causal=causal, out_dtype=F32)
    for a, b in zip(got[1:], want[1:]):
        b = b.view(B, 2, 5, N, d).sum(2)
        assert float((a - b).abs().max()) < 2.0 ** -16 * float(b.abs().max())


@pytest.mark.gpu
def test_rows_past_32_bit_offsets():
    """More than 2^31 elements of q, k and v, in short documents: the last sequence's last heads."""
    B, Hq, Hkv, N, d = 33, 64, 64, 16384, 64
    if torch.cuda.mem_get_info()[0] < 70 << 30:
        pytest.skip("needs 70 GB")
    g = torch.Generator(device=DEV).manual_seed(16)
    q, k, v, do = (torch.randn((B, h, N, d), generator=g, device=DEV, dtype=BF16) for h in (Hq, Hkv, Hkv, Hq))
    ids = (torch.arange(N, device=DEV) // 100).to(torch.int32).expand(B, N).contiguous()
    o, lse = fa().fwd_rules(q, k, v, causal=True, documents=ids)
    dq, dk, dv = fa().bwd_rules(q, k, v, o, lse, do, causal=True, documents=ids)
    assert q.numel() > 1 << 31 and fa().get_device_error() == 0
    last = [t[-1:, -2:].clone() for t in (q, k, v, do)]
    o1, lse1 = fa().fwd_rules(*last[:3], causal=True, documents=ids[:1].contiguous())
    assert torch.equal(o[-1:, -2:], o1) and torch.equal(lse[-1:, -2:], lse1)
    g1 = fa().bwd_rules(*last[:3], o1, lse1, last[3], causal=True, documents=ids[:1].contiguous())
    assert torch.equal(dk[-1:, -2:], g1[1]) and torch.equal(dv[-1:, -2:], g1[2])
    assert float((dq[-1:, -2:].float() - g1[0].float()).abs().max()) < 2.0 ** -6


@pytest.mark.gpu
@pytest.mark.parametrize("d,causal", [(32, True), (64, True), (128, True), (128, False)])
def test_wait_limit_is_reported_and_the_next_call_is_right(d, causal):
    """With a limit of 1 ns waits run out: the status says so, every role ends, and the next call is right."""
    B, Hq, Hkv, N = 3, 6, 2, 700
    rules = Rules(causal=causal, softcap=9.0 if causal else 0.0, documents=documents(B, N, [300, 200]))
    x = inputs(B, Hq, Hkv, N, N, d, seed=17)
    ref = attention(*x[:3], rules, x[3])
    o, lse, _ = run(*x, rules)
    fa().set_wait_timeout_ns(1)
    try:
        fa().fwd_rules(*(t.to(DEV) for t in x[:3]), **rules.kwargs(DEV))
        first = fa().get_device_error()
        fa().bwd_rules(*(t.to(DEV) for t in x[:3]), o, lse, x[3].to(DEV), **rules.kwargs(DEV))
        second = fa().get_device_error()
    finally:
        fa().set_wait_timeout_ns(0)
    assert first == second == fa().FA_ERR_TIMEOUT
    o, lse, grads = run(*x, rules)
    assert fa().get_device_error() == 0
    check_forward(o, lse, ref, "after")
    check_gradients(grads, ref, "after")


# ------------------------------------------------------------------------------------ streams, graphs, buffers
@pytest.mark.gpu
def test_two_streams_at_once():
    """Calls on two streams with workspaces of their own."""
    B, Hq, Hkv, N, d = 4, 8, 4, 900, 64
    rules = Rules(causal=True, documents=documents(B, N, [350, 20, 400]))
    xs = [inputs(B, Hq, Hkv, N, N, d, seed=s) for s in (18, 19)]
    dev = [[t.to(DEV) for t in x] for x in xs]
    a = rules.kwargs(DEV)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in xs], [[], []]
    for _ in range(3):
        for i, (x, st) in enumerate(zip(dev, streams)):
            with torch.cuda.stream(st):
                o, lse = fa().fwd_rules(*x[:3], out_dtype=F32, **a)
                got[i] = (o, lse, fa().bwd_rules(*x[:3], o, lse, x[3], out_dtype=F32, **a))
    torch.cuda.synchronize()
    assert fa().get_device_error() == 0
    for x, (o, lse, grads) in zip(xs, got):
        ref = attention(*x[:3], rules, x[3])
        check_forward(o, lse, ref, "streams")
        check_gradients(grads, ref, "streams")


@pytest.mark.gpu
def test_outputs_and_workspaces_given():
    B, Hq, Hkv, N, d = 2, 4, 2, 333, 64
    q, k, v, do = (t.to(DEV) for t in inputs(B, Hq, Hkv, N, N, d, seed=10))
    docs = documents(B, N, [100, 50]).to(DEV)
    need = fa().fwd_rules_workspace_size(B, N)
    guard = 4096
    for dt in (BF16, F32):
        ws = torch.full((need + guard,), 0xAB, dtype=torch.uint8, device=DEV)
        out = torch.full((B * Hq * N * d + guard,), 7.0, dtype=dt, device=DEV)
        lse = torch.full((B * Hq * N + guard,), 7.0, device=DEV)
        o = out[:B * Hq * N * d].view(B, Hq, N, d)
        l = lse[:B * Hq * N].view(B, Hq, N)  # noqa: E741
        r = fa().fwd_rules(q, k, v, documents=docs, out=o, lse=l, workspace=ws[:need])
        assert r[0].data_ptr() == o.data_ptr() and r[1].data_ptr() == l.data_ptr()
        o0, l0 = fa().fwd_rules(q, k, v, documents=docs, out_dtype=dt)
        assert torch.equal(o, o0) and torch.equal(l, l0)
        assert bool((ws[need:] == 0xAB).all()) and bool((out[B * Hq * N * d:] == 7).all()) and bool((lse[B * Hq * N:] == 7).all())
        need_b = fa().bwd_rules_workspace_size(B, Hq, Hkv, N, N, d, fa().num_sms())
        ws = torch.full((need_b + guard,), 0xAB, dtype=torch.uint8, device=DEV)
        g = [torch.full((t.numel() + guard,), 7.0, dtype=dt, device=DEV) for t in (q, k, v)]
        views = tuple(b[:t.numel()].view(t.shape) for b, t in zip(g, (q, k, v)))
        fa().bwd_rules(q, k, v, o0, l0, do, documents=docs, grads=views, workspace=ws[:need_b])
        want = fa().bwd_rules(q, k, v, o0, l0, do, documents=docs, out_dtype=dt)
        assert torch.equal(views[1], want[1]) and torch.equal(views[2], want[2])
        assert float((views[0].float() - want[0].float()).abs().max()) < (1e-5 if dt == F32 else 0.02)
        assert bool((ws[need_b:] == 0xAB).all()) and all(bool((b[t.numel():] == 7).all()) for b, t in zip(g, (q, k, v)))


@pytest.mark.gpu
def test_captured_and_replayed_on_another_stream():
    """A captured training step replayed on new inputs, twice in a row, with one workspace for both calls."""
    B, Hq, Hkv, N, d = 2, 8, 2, 500, 128
    rules = Rules(causal=True, softcap=15.0, documents=documents(B, N, [200, 31, 90], pads=[0, 40]))
    a = rules.kwargs(DEV)
    x = [t.to(DEV) for t in inputs(B, Hq, Hkv, N, N, d, seed=11)]
    ws = torch.empty(max(fa().fwd_rules_workspace_size(B, N), fa().bwd_rules_workspace_size(B, Hq, Hkv, N, N, d, fa().num_sms())),
                     dtype=torch.uint8, device=DEV)

    def step():
        o, lse = fa().fwd_rules(*x[:3], workspace=ws, **a)
        return o, lse, fa().bwd_rules(*x[:3], o, lse, x[3], workspace=ws, **a)

    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
        st.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            o, lse, grads = step()
        for seed in (12, 13):
            new = inputs(B, Hq, Hkv, N, N, d, seed=seed)
            for t, u in zip(x, new):
                t.copy_(u)
            graph.replay()
            graph.replay()
            st.synchronize()
            ref = attention(*new[:3], rules, new[3])
            check_forward(o, lse, ref, "replayed")
            # the backward took the forward's bf16 output
            check_gradients(grads, ref, "replayed")
    assert fa().get_device_error() == 0


# ------------------------------------------------------------------------------------ as they are used
@pytest.mark.gpu
def test_training_step_from_projections():
    """qk_norm_rope -> fwd_rules -> bwd_rules -> qk_norm_rope_bwd over packed documents: each document's gradients are those
    of the document on its own."""
    B, N, Hq, Hkv, d = 1, 400, 4, 2, 64
    g = torch.Generator().manual_seed(14)
    x = torch.randn((B, N, Hq + 2 * Hkv, d), generator=g).to(BF16).to(DEV)
    do = torch.randn((B, Hq, N, d), generator=g).to(BF16).to(DEV)
    w = torch.ones(d, device=DEV)
    ang = torch.arange(N)[:, None] * 10000.0 ** (-torch.arange(d // 2) / (d // 2))
    cos, sin = ang.cos().float().to(DEV), ang.sin().float().to(DEV)
    cuts = [0, 130, 131, 400]

    def step(x, do, positions, docs):
        q, k, v = x[:, :, :Hq], x[:, :, Hq:Hq + Hkv], x[:, :, Hq + Hkv:]
        qn, kn, vn = fa().qk_norm_rope(q, k, v, w, w, cos, sin, positions=positions)
        rules = dict(causal=True, softcap=10.0, documents=docs)
        o, lse = fa().fwd_rules(qn, kn, vn, **rules)
        grads = fa().bwd_rules(qn, kn, vn, o, lse, do, out_dtype=F32, **rules)
        return o, fa().qk_norm_rope_bwd(*grads, q, k, w, w, cos, sin, positions=positions, out_dtype=F32)

    docs = torch.zeros((B, N), dtype=torch.int32)
    pos = torch.zeros((B, N), dtype=torch.int32)
    for n, (a, e) in enumerate(zip(cuts, cuts[1:])):
        docs[:, a:e] = n
        pos[:, a:e] = torch.arange(e - a)
    o, grads = step(x, do, pos.to(DEV), docs.to(DEV))
    dw = [torch.zeros(d, device=DEV) for _ in range(2)]
    for a, e in zip(cuts, cuts[1:]):
        o1, g1 = step(x[:, a:e].contiguous(), do[:, :, a:e].contiguous(), pos[:, :e - a].contiguous().to(DEV) * 0 +
                      torch.arange(e - a, dtype=torch.int32, device=DEV), None)
        # other tile borders: sums in another order, and another rounding of a weight now and then
        assert float((o[:, :, a:e].float() - o1.float()).abs().max()) < 2.0 ** -6
        for i in range(3):
            assert float((grads[i][:, a:e] - g1[i]).abs().max()) < 2.0 ** -5
        dw = [s + t for s, t in zip(dw, g1[3:])]
    assert all(float((s - t).abs().max()) < 0.05 * float(t.abs().max()) + 0.05 for s, t in zip(dw, grads[3:]))
    assert fa().get_device_error() == 0
