"""fa_decode_tree against the plain fp64 form, at the sizes and trees where it can go wrong."""
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


def inputs(B, Hq, Hkv, T, Nk_max, d, lens, n_nodes=None, seed=0, fill=float("nan")):
    """q, caches with `fill` behind each sequence's tree, lengths."""
    g = torch.Generator().manual_seed(seed)
    q = torch.randn((B, Hq, T, d), generator=g).to(BF16)
    k = torch.randn((B, Hkv, Nk_max, d), generator=g).to(BF16)
    v = torch.randn((B, Hkv, Nk_max, d), generator=g).to(BF16)
    for b in range(B):
        end = int(lens[b]) + (int(n_nodes[b]) if n_nodes is not None else T)
        k[b, :, end:] = fill
        v[b, :, end:] = fill
    return q, k, v


def call(q, k, v, lens, parents=None, n_nodes=None, **kw):
    to = lambda t: None if t is None else t.to(DEV)  # noqa: E731
    o, lse = fa().decode_tree(to(q), to(k), to(v), to(lens), parents=to(parents), n_nodes=to(n_nodes), **kw)
    torch.cuda.synchronize()
    return o, lse


def i32(*x):
    return torch.tensor(x, dtype=torch.int32)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("R,T", [(1, 1), (3, 1), (2, 5), (4, 8), (5, 13), (1, 100), (4, 32), (1, 128),
                                 (3, 43), (2, 65), (2, 128), (5, 64), (9, 60)])
def test_sizes(d, R, T):
    """Groups of 1 to 540 rows: one query tile, two, two units with one and with two tiles."""
    lens = i32(0, 1, 127, 128, 500)
    B, Hkv, Nk_max = 5, 2, 500 + T
    q, k, v = inputs(B, Hkv * R, Hkv, T, Nk_max, d, lens, seed=R * 1000 + T)
    par = random_parents(B, T, seed=T)
    ref = tree_attention(q, k, v, lens, par, None, 1 / math.sqrt(d))
    for dt in (torch.float32, BF16):
        o, lse = call(q, k, v, lens, par, out_dtype=dt)
        assert fa().get_device_error() == 0
        check_tree(o, lse, ref, f"d={d} R={R} T={T} {dt}")


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("R,T", [(3, 10), (2, 100)])
def test_ragged_trees(d, R, T):
    """Node counts from none to all, with empty caches among them: rows of absent nodes are 0 and -inf."""
    lens = i32(0, 0, 0, 300, 300, 129, 255, 64)
    cnt = i32(0, 1, T, 0, T - 1, T, 1, T // 2)
    B, Hkv, Nk_max = 8, 3, 300 + T
    q, k, v = inputs(B, Hkv * R, Hkv, T, Nk_max, d, lens, cnt, seed=5)
    par = random_parents(B, T, seed=6)
    ref = tree_attention(q, k, v, lens, par, cnt, 0.3)
    o, lse = call(q, k, v, lens, par, cnt, scale=0.3, out_dtype=torch.float32)
    assert fa().get_device_error() == 0
    check_tree(o, lse, ref, f"d={d}")
    assert torch.all(o[0] == 0) and torch.all(torch.isneginf(lse[0]))


@pytest.mark.parametrize("B,Hkv,hi,T", [(70, 8, 140, 4), (300, 2, 60, 3), (3, 1, 6000, 7), (1, 1, 20000, 4),
                                        (40, 5, 900, 40), (1, 1, 1, 1)])
def test_shares_cross_units(B, Hkv, hi, T):
    """More units than CTAs with one or two tiles each (a CTA walks several, some wholly its own), and
    single units over many CTAs."""
    R, d = 4, 64
    g = torch.Generator().manual_seed(B)
    lens = torch.randint(0, hi + 1, (B,), generator=g).to(torch.int32)
    cnt = torch.randint(0, T + 1, (B,), generator=g).to(torch.int32)
    q, k, v = inputs(B, Hkv * R, Hkv, T, hi + T, d, lens, cnt, seed=B + 1)
    par = random_parents(B, T, seed=B)
    ref = tree_attention(q, k, v, lens, par, cnt, 1 / 8)
    o, lse = call(q, k, v, lens, par, cnt, out_dtype=torch.float32)
    o2, lse2 = call(q, k, v, lens, par, cnt, out_dtype=torch.float32)
    assert fa().get_device_error() == 0
    check_tree(o, lse, ref, f"B={B}")
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("R,T", [(4, 4), (2, 64), (1, 1)])
def test_many_units(d, R, T):
    """Enough (sequence, head) pairs that each warpgroup has a share of its own, with lengths of 0 to 5 key
    tiles, one long sequence among them, and absent nodes; up to 128 rows."""
    B, Hkv, hi = 310, 3, 600
    g = torch.Generator().manual_seed(d + T)
    lens = torch.randint(0, hi + 1, (B,), generator=g).to(torch.int32)
    lens[5], lens[6], lens[7] = 0, 2500, 127
    cnt = torch.randint(0, T + 1, (B,), generator=g).to(torch.int32)
    q, k, v = inputs(B, Hkv * R, Hkv, T, 2500 + T, d, lens, cnt, seed=T)
    par = random_parents(B, T, seed=d)
    ref = tree_attention(q, k, v, lens, par, cnt, 1 / math.sqrt(d))
    o, lse = call(q, k, v, lens, par, cnt, out_dtype=torch.float32)
    o2, lse2 = call(q, k, v, lens, par, cnt, out_dtype=torch.float32)
    assert fa().get_device_error() == 0
    check_tree(o, lse, ref, f"d={d} R={R} T={T}")
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    check_tree(*call(q, k, v, lens, par, cnt), ref, "bf16")


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("R,T", [(4, 40), (2, 128), (5, 60), (3, 100)])
def test_many_units_of_more_rows(d, R, T):
    """More than 128 rows (one block whose second half is short or full, or a second block of 44 rows), enough
    units that a CTA walks several: growing and falling maxima across tiles, empty and absent ones among them."""
    B, Hkv, hi = 90, 2, 500
    g = torch.Generator().manual_seed(d + T)
    lens = torch.randint(0, hi + 1, (B,), generator=g).to(torch.int32)
    lens[5], lens[6], lens[7] = 0, 1500, 127
    cnt = torch.randint(0, T + 1, (B,), generator=g).to(torch.int32)
    q, k, v = inputs(B, Hkv * R, Hkv, T, 1500 + T, d, lens, cnt, seed=T)
    k[6, :, :1500] *= torch.linspace(0.1, 8, 1500)[None, :, None].to(BF16)
    par = random_parents(B, T, seed=d)
    ref = tree_attention(q, k, v, lens, par, cnt, 1 / math.sqrt(d))
    o, lse = call(q, k, v, lens, par, cnt, out_dtype=torch.float32)
    o2, lse2 = call(q, k, v, lens, par, cnt, out_dtype=torch.float32)
    assert fa().get_device_error() == 0
    check_tree(o, lse, ref, f"d={d} R={R} T={T}")
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("B,R,T", [(3, 4, 8), (300, 4, 8), (20, 4, 64)])
def test_wait_limit_is_reported_and_the_next_call_is_right(B, R, T, d):
    """With a limit of 1 ns waits run out in each form of the kernel: the status says so, every role ends, and
    the next call with the usual limit is right."""
    lens = torch.full((B,), 300, dtype=torch.int32)
    q, k, v = inputs(B, 2 * R, 2, T, 400, d, lens, seed=3)
    fa().set_wait_timeout_ns(1)
    try:
        call(q, k, v, lens)
        status = fa().get_device_error()
    finally:
        fa().set_wait_timeout_ns(0)
    assert status == fa().FA_ERR_TIMEOUT
    o, lse = call(q, k, v, lens, out_dtype=torch.float32)
    assert fa().get_device_error() == 0
    check_tree(o, lse, tree_attention(q, k, v, lens, None, None, 1 / math.sqrt(d)), "after")


@pytest.mark.parametrize("B,R,T,Nk,d,hi", [(1, 300, 128, 700, 64, 500), (5000, 2, 2, 8, 32, 3), (600, 3, 100, 110, 128, 5),
                                           (3, 130, 1, 900, 128, 800), (2, 128, 1, 900, 128, 800), (152, 1, 1, 130, 128, 129)])
def test_many_rows_and_many_sequences(B, R, T, Nk, d, hi):
    """Far more rows than two blocks', thousands of sequences of a few tokens, a row more or less than a block."""
    g = torch.Generator().manual_seed(B + T)
    lens = torch.randint(0, hi + 1, (B,), generator=g).to(torch.int32)
    cnt = torch.randint(0, T + 1, (B,), generator=g).to(torch.int32)
    cnt[0] = T
    q, k, v = inputs(B, R, 1, T, Nk, d, lens, cnt, seed=1)
    par = random_parents(B, T, seed=2)
    o, lse = call(q, k, v, lens, par, cnt, out_dtype=torch.float32)
    assert fa().get_device_error() == 0
    check_tree(o, lse, tree_attention(q, k, v, lens, par, cnt, 1 / math.sqrt(d)), f"B={B} R={R} T={T}")


@pytest.mark.parametrize("d,T,R", [(128, 9, 4), (64, 60, 3)])
def test_chain_and_shallow_trees(d, T, R):
    """No parents: a chain, the same as parents t - 1.  All nodes children of the last token: each sees itself only."""
    lens = i32(200, 121)
    q, k, v = inputs(2, 2 * R, 2, T, 300, d, lens, seed=9)
    chain = (torch.arange(T, dtype=torch.int32) - 1).repeat(2, 1)
    a, b = call(q, k, v, lens), call(q, k, v, lens, chain)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check_tree(*a, tree_attention(q, k, v, lens, None, None, 1 / math.sqrt(d)), "chain")
    flat = torch.full((2, T), -1, dtype=torch.int32)
    check_tree(*call(q, k, v, lens, flat), tree_attention(q, k, v, lens, flat, None, 1 / math.sqrt(d)), "flat")
    assert fa().get_device_error() == 0


@pytest.mark.parametrize("Hq,Hkv", [(8, 8), (8, 2), (8, 1)])
def test_one_node_is_grouped_decode(Hq, Hkv):
    """T = 1: the grouped decode over one token more.  Both are within their own bound of the exact value."""
    lens = i32(0, 77, 512, 1000)
    q, k, v = inputs(4, Hq, Hkv, 1, 1001, 128, lens, seed=Hq + Hkv)
    o, lse = call(q, k, v, lens, out_dtype=torch.float32)
    og, lg = fa().decode_splitkv_gqa(q.to(DEV), k.to(DEV), v.to(DEV), (lens + 1).to(DEV), out_dtype=torch.float32)
    torch.cuda.synchronize()
    ref = tree_attention(q, k, v, lens, None, None, 1 / math.sqrt(128))
    check_tree(o, lse, ref, "tree")
    check_tree(og, lg, ref, "grouped decode")


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("d,R", [(128, 2), (64, 40)])
def test_hidden_keys_do_not_reach_other_branches(bad, d, R):
    """Two branches below one root; a node's key is not finite: only the rows that see it change."""
    par = torch.tensor([[-1, 0, 0, 1, 2, 3]], dtype=torch.int32)  # 0 -> 1 -> 3 -> 5, 0 -> 2 -> 4
    lens = i32(130)
    q, k, v = inputs(1, R, 1, 6, 200, d, lens, seed=3)
    ref = tree_attention(q, k, v, lens, par, None, 1 / math.sqrt(d))
    k[0, 0, 130 + 3] = bad
    o, lse = call(q, k, v, lens, par, out_dtype=torch.float32)
    clean = [0, 1, 2, 4]
    check_tree(o[:, :, clean], lse[:, :, clean], tuple(t[:, :, clean] for t in ref), "branches")


def test_large_scores():
    """Keys of growing size: the running max moves at every tile, the early tiles' weights vanish."""
    lens = i32(900, 30)
    q, k, v = inputs(2, 4, 1, 4, 1000, 64, lens, seed=4)
    k[0, :, :904] *= torch.linspace(0.1, 60, 904)[None, :, None].to(BF16)
    par = random_parents(2, 4, 1)
    check_tree(*call(q, k, v, lens, par, out_dtype=torch.float32),
               tree_attention(q, k, v, lens, par, None, 1 / 8), "large")


def test_bad_lengths_and_parents_are_recorded():
    lens = i32(-4, 500, 60, 60)  # below 0, beyond the cache with its tree
    q, k, v = inputs(4, 4, 2, 5, 300, 64, i32(0, 295, 60, 60), fill=0.0, seed=8)
    o, lse = call(q, k, v, lens, out_dtype=torch.float32)
    assert fa().get_device_error() == fa().FA_ERR_INVALID_ARG and fa().get_device_error() == 0
    # clamped: no cached token; 300 cached tokens and no room for nodes
    ref = tree_attention(q, k, v, i32(0, 300, 60, 60), None, i32(5, 0, 5, 5), 1 / 8)
    check_tree(o, lse, ref, "clamped")
    par = torch.tensor([[-1, 0, 1, 2, 3]] * 4, dtype=torch.int32)
    par[2] = i32(0, 7, -3, 2, 4)  # itself, a later node, nonsense, fine, itself
    o, lse = call(q, k, v, i32(0, 295, 60, 60), par, out_dtype=torch.float32)
    assert fa().get_device_error() == fa().FA_ERR_INVALID_ARG
    par[2] = i32(-1, -1, -1, 2, -1)
    check_tree(o, lse, tree_attention(q, k, v, i32(0, 295, 60, 60), par, None, 1 / 8), "parents")


def test_outputs_are_written_whole_and_nothing_else():
    B, Hq, Hkv, T, d = 3, 6, 2, 7, 64
    lens, cnt = i32(0, 140, 33), i32(7, 3, 0)
    q, k, v = inputs(B, Hq, Hkv, T, 200, d, lens, cnt, seed=1)
    n, m = B * Hq * T * d, B * Hq * T
    buf = torch.full((n + 256,), float("nan"), device=DEV)
    lbuf = torch.full((m + 256,), float("nan"), device=DEV)
    ws = torch.full((fa().decode_tree_workspace_size(Hq, Hkv, T, d, fa().num_sms()) + 256,), 255, dtype=torch.uint8, device=DEV)
    call(q, k, v, lens, None, cnt, out=buf[128:128 + n].view(B, Hq, T, d), lse=lbuf[128:128 + m].view(B, Hq, T),
         workspace=ws[:-256])
    assert not buf[128:128 + n].isnan().any() and not lbuf[128:128 + m].isnan().any()
    for t, s in ((buf, n), (lbuf, m)):
        assert t[:128].isnan().all() and t[128 + s:].isnan().all()
    assert torch.all(ws[-256:] == 255)
    with pytest.raises(fa().FaError, match="workspace"):
        call(q, k, v, lens, None, cnt, workspace=ws[:256])


def test_two_streams_and_graphs():
    """Two calls at once on two streams (a workspace each), and a captured call on new inputs, equal the eager call."""
    lens = i32(700, 3, 450)
    q, k, v = inputs(3, 8, 2, 16, 800, 128, lens, seed=2)
    par = random_parents(3, 16, 3).to(DEV)
    x = [t.to(DEV) for t in (q, k, v, lens)]
    want = fa().decode_tree(*x, parents=par)
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(fa().decode_tree(*x, parents=par))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[0]) and torch.equal(l, want[1]) for o, l in got)
    ws = torch.empty(fa().decode_tree_workspace_size(8, 2, 16, 128, fa().num_sms()), dtype=torch.uint8, device=DEV)
    o, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fa().decode_tree(*x, parents=par, out=o, lse=lse, workspace=ws)
    x[0].copy_(torch.randn(x[0].shape, device=DEV))
    x[3].copy_(i32(5, 640, 0))  # other lengths than at capture
    x[1].nan_to_num_(0.0)
    x[2].nan_to_num_(0.0)
    for _ in range(3):
        g.replay()
    want = fa().decode_tree(*x, parents=par)
    torch.cuda.synchronize()
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1]) and fa().get_device_error() == 0
