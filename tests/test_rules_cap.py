"""A capped score is its own matter: its accuracy goes by its own size, not by scores beyond the cap that its tile holds too,
and what hidden keys and rows hold does not reach it in any bit.

Bounds.  A cap of 1e5 and more leaves scores up to 30 as they are to within s^3 / (3 cap^2) < 1e-6, so the references
have none, and with them no error that is counted in caps.  The kernels' tanh is off by 1.2e-6 of its value, which the
references' bound of the products, 4 d 2^-24 sum |q_c k_c| >= 7.6e-6 |s|, holds together with the products' own d 2^-24.
"""
from __future__ import annotations

import math

import pytest
import torch

from tests.rules_reference import Rules, attention, check_forward, check_gradients
from tests.test_decode_prefix import inputs as decode_inputs
from tests.test_decode_prefix import reference as decode_reference

BF16, F32 = torch.bfloat16, torch.float32
DEV = "cuda"
pytestmark = pytest.mark.gpu


def fa():
    import exact_tiled_attention_fa_gb300 as m
    return m


def slopes(Hq):
    return torch.exp2(-8.0 * torch.arange(1, Hq + 1) / Hq).float()


def inputs(B, Hq, Hkv, N, Nk, d, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g).to(BF16)  # noqa: E731
    return r(B, Hq, N, d), r(B, Hkv, Nk, d), r(B, Hkv, Nk, d), r(B, Hq, N, d)


def run(q, k, v, do, rules):
    """Forward and gradients, fp32."""
    q, k, v, do = (t.to(DEV) for t in (q, k, v, do))
    a = rules.kwargs(DEV)
    o, lse = fa().fwd_rules(q, k, v, out_dtype=F32, **a)
    grads = fa().bwd_rules(q, k, v, o, lse, do, out_dtype=F32, **a)
    torch.cuda.synchronize()
    assert fa().get_device_error() == 0
    return o, lse, grads


# ------------------------------------------------------------------------------------ accuracy
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("cap", [1e5, 1e7, 1e30])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("causal", [False, True])
def test_scores_beside_a_key_far_below_the_cap(d, cap, bias, causal):
    """Key 0 has a score of -3 caps in every row, and so no weight: the others are what they are without it."""
    q, k, v, do = inputs(2, 4, 2, 200, 261, d, seed=1)
    sl = slopes(4) if bias else None
    q[..., 0] = 4.0
    k[:, :, 0] = 0.0
    k[:, :, 0, 0] = -3.0 * cap * math.sqrt(d) / 4.0
    o, lse, (dq, dk, dv) = run(q, k, v, do, Rules(causal=causal, softcap=cap, slopes=sl))
    # (positions from the end and distances are the same without the first key)
    ref = attention(q, k[:, :, 1:], v[:, :, 1:], Rules(causal=causal, slopes=sl), do)
    what = f"d={d} cap={cap} bias={bias}"
    check_forward(o, lse, ref, what)
    check_gradients((dq, dk[:, :, 1:], dv[:, :, 1:]), ref, what)
    assert bool((dk[:, :, 0] == 0).all()) and bool((dv[:, :, 0] == 0).all())


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("cap", [1e5, 1e7, 1e30])
@pytest.mark.parametrize("bias", [False, True])
def test_rows_beside_one_far_beyond_the_cap(d, cap, bias):
    """One row of 32 has scores of many caps; the gradient of its output is 0, so that it adds nothing to those of keys and
    values.  (Up to a cap of 1e7: fp32 has no weights for scores around 1e30, whose steps are 1e22.)"""
    q, k, v, do = inputs(2, 4, 2, 200, 261, d, seed=2)
    sl = slopes(4) if bias else None
    far = torch.arange(200) % 32 == 5
    q[:, :, far] = (q[:, :, far].float() * 8.0 * cap).to(BF16)
    do[:, :, far] = 0.0
    o, lse, grads = run(q, k, v, do, Rules(causal=True, softcap=cap, slopes=sl))
    ref = attention(q, k, v, Rules(causal=True, slopes=sl), do)  # (its bounds for the far rows mean nothing)
    what = f"d={d} cap={cap} bias={bias}"
    assert bool(torch.isfinite(o).all())
    rest = {n: ref[n][:, :, ~far] for n in ("O", "dO", "L", "dL")}
    check_forward(o[:, :, ~far], lse[:, :, ~far], rest, what)
    if cap > 1e7:
        return
    assert bool((grads[0][:, :, far] == 0).all())
    rows = {n: t[:, :, ~far] if n in ("dq", "bdq") else t for n, t in ref.items()}
    check_gradients((grads[0][:, :, ~far], *grads[1:]), rows, what)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("cap", [1e5, 1e7, 1e30])
@pytest.mark.parametrize("B,R,bias", [(5, 4, False), (5, 4, True), (70, 3, False), (70, 3, True)])
def test_decode_beside_scores_far_beyond_the_cap(d, cap, B, R, bias):
    """Behind a prefix whose first key has a score of -3 caps, beside sequences whose scores are of many caps."""
    Hq, Hkv, P, Nk = 2 * R, 2, 400, 200
    lens = (torch.arange(B, dtype=torch.int32) * 29) % (Nk + 1)
    q, kp, vp, k, v = decode_inputs(B, Hq, Hkv, P, Nk, d, lens, seed=3, fill=0.0)
    sl = slopes(Hq) if bias else None
    q[..., 0] = 4.0
    kp[:, 0] = 0.0
    kp[:, 0, 0] = -3.0 * cap * math.sqrt(d) / 4.0
    far = torch.arange(B) % 4 == 2
    q[far] = (q[far].float() * 8.0 * cap).to(BF16)
    to = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    o, lse = fa().decode_prefix(to(q), to(kp), to(vp), to(k), to(v), to(lens), softcap=cap, slopes=to(sl), out_dtype=F32)
    assert fa().get_device_error() == 0
    ref = decode_reference(q[~far], kp[:, 1:], vp[:, 1:], k[~far], v[~far], lens[~far], P - 1, Rules(slopes=sl))
    near = ~far.to(DEV)
    check_forward(o[near], lse[near], ref, f"d={d} cap={cap} B={B}")


# ------------------------------------------------------------------------------------ what is hidden
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("cap", [50.0, 1e5, 1e7])
@pytest.mark.parametrize("bias", [False, True])
def test_hidden_keys_do_not_choose_the_form_of_the_cap(d, cap, bias):
    """Whatever keys of another document and keys behind a causal position hold, other rows' results are bit by bit those
    with zeros there.  (The borders are between 32 rows: a row that sees such a key may share its own form of the cap with
    the rows beside it.)"""
    q, k, v, _ = inputs(2, 2, 1, 330, 330, d, seed=4)
    ids = torch.zeros((2, 330), dtype=torch.int32)
    ids[:, 160:] = 1
    sl = slopes(2) if bias else None
    cases = [(Rules(causal=c, softcap=cap, slopes=sl, documents=ids), slice(0, 160), slice(160, 330)) for c in (False, True)]
    cases.append((Rules(causal=True, softcap=cap, slopes=sl), slice(288, 330), slice(0, 288)))
    for rules, keys, rows in cases:
        got = []
        for x in (0.0, math.inf, -math.inf, math.nan, 1e38, -1e38):
            kk = k.clone()
            kk[:, :, keys] = x
            o, lse = fa().fwd_rules(q.to(DEV), kk.to(DEV), v.to(DEV), out_dtype=F32, **rules.kwargs(DEV))
            got.append((x, o[:, :, rows], lse[:, :, rows]))
        for x, o, lse in got[1:]:
            assert torch.equal(o, got[0][1]) and torch.equal(lse, got[0][2]), (x, rules.causal, rules.docs is not None)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("cap", [50.0, 1e5, 1e7])
@pytest.mark.parametrize("bias", [False, True])
def test_hidden_queries_do_not_choose_the_form_of_the_cap(d, cap, bias):
    """The gradients of a document do not depend on the queries of another one in the same tile.  (One key tile: a query's
    gradient is then one term, and no order of sums plays in.)"""
    q, k, v, do = inputs(2, 2, 1, 128, 128, d, seed=5)
    ids = torch.zeros((2, 128), dtype=torch.int32)
    ids[:, 64:] = 1
    rules = Rules(softcap=cap, slopes=slopes(2) if bias else None, documents=ids)
    got = []
    for x in (0.0, 2.0 ** 100):
        qq = q.clone()
        qq[:, :, :64] = (qq[:, :, :64].float().sign() * x).to(BF16)
        o, lse, grads = run(qq, k, v, do, rules)
        got.append([t[:, :, 64:] for t in (o, lse, *grads)])
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("cap", [50.0, 1e5, 1e7])
@pytest.mark.parametrize("B,R,bias", [(3, 4, False), (3, 4, True), (70, 3, False), (70, 3, True)])
def test_rows_behind_the_lengths_do_not_choose_the_form_of_the_cap(d, cap, B, R, bias):
    """Decode: whatever rows behind the prefix and behind the sequences' own keys hold, the result is bit by bit the same."""
    Hq, Hkv, P, P_max, Nk = 2 * R, 2, 333, 400, 200
    lens = ((torch.arange(B, dtype=torch.int32) * 29) % (Nk + 1)).to(torch.int32)
    sl = slopes(Hq).to(DEV) if bias else None
    first = None
    for x in (0.0, math.inf, -math.inf, math.nan, 1e38):
        t = [a.to(DEV) for a in decode_inputs(B, Hq, Hkv, P_max, Nk, d, lens, P=P, seed=6, fill=x)]
        n, plen = lens.to(DEV), torch.tensor([P], dtype=torch.int32, device=DEV)
        o, lse = fa().decode_prefix(*t, n, prefix_len=plen, softcap=cap, slopes=sl, out_dtype=F32)
        assert bool(torch.isfinite(o).all())
        first = first or (o, lse)
        assert torch.equal(o, first[0]) and torch.equal(lse, first[1]), x
    assert fa().get_device_error() == 0
