"""Decode behind a shared prefix that several query tiles meet: at d = 128 a query tile begins further on in the prefix the
later it comes to it, and goes round (fa_tree_kernel.cuh, SharedWalk).  Every share of a unit, and the walks of K and of V in it, have
to agree on where that is.

Keys and values name their tile of 128 keys, and a row's query asks for one tile: its score there is 40, elsewhere 0.  Its
output is that tile's name, and its log-sum-exp 40 + log(the tile's keys), which tells a tile that was read twice or not at all.
Bounds: weights elsewhere are e^-40 each; the rounding of the weights to bf16 2^-8, of the log-sum-exp 2^-20 (1 + |LSE|).
"""
from __future__ import annotations

import math
import random

import pytest
import torch

BF16 = torch.bfloat16
DEV = "cuda"
D = 128
pytestmark = pytest.mark.gpu


def fa():
    import exact_tiled_attention_fa_gb300 as m
    return m


def check(B, R, Hkv, P, P_max, Nk, seed):
    tiles = (P + 127) // 128
    assert tiles <= D  # a channel each
    Hq = R * Hkv
    g = torch.Generator(device=DEV).manual_seed(seed)
    key = torch.arange(P_max, device=DEV)
    rows = torch.full((P_max, D), math.nan, device=DEV)  # behind the prefix
    rows[:P] = torch.nn.functional.one_hot(key[:P] // 128, D).float()
    # which tile a row asks for: all of them in turn, another one to begin with in each key/value head
    ask = (torch.arange(B * R, device=DEV)[:, None] * 7 + torch.arange(Hkv, device=DEV) * 5 + seed) % tiles  # [B * R, Hkv]
    ask = ask.view(B, R, Hkv).transpose(1, 2).reshape(B, Hq)
    q = (40.0 * torch.nn.functional.one_hot(ask, D).float()).to(BF16)[:, :, None]
    k_prefix = rows.to(BF16).expand(Hkv, -1, -1).contiguous()
    cache = torch.zeros((B, Hkv, Nk, D), dtype=BF16, device=DEV)
    lens = torch.randint(0, Nk + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    plen = torch.tensor([P], dtype=torch.int32, device=DEV)
    o, lse = fa().decode_prefix(q, k_prefix, k_prefix, cache, cache, lens, prefix_len=plen, scale=1.0, out_dtype=torch.float32)
    what = f"B={B} R={R} Hkv={Hkv} P={P}/{P_max} Nk={Nk}"
    want = torch.nn.functional.one_hot(ask, D).float()[:, :, None]
    assert float((o - want).abs().max()) <= 2.0 ** -8 + 1e-6, what
    keys = torch.where(ask == tiles - 1, P - 128 * (tiles - 1), 128).double()
    L = (40.0 + keys.log())[:, :, None]
    assert float((lse.double() - L).abs().max()) <= 2.0 ** -20 * 47, what


@pytest.mark.parametrize("R", [1, 3, 5, 8, 65, 100])
def test_every_tile_of_a_prefix_once(R):
    """Groups that fill a query tile and such that leave some of it, 2 to 10 query tiles, prefixes that end at a tile's end
    and beside it, from units a few tiles long to such of several shares."""
    rng = random.Random(500 + R)
    seqs = 128 // R
    for i in range(120):
        n_qp = rng.randint(2, 10)
        B = seqs * (n_qp - 1) + rng.randint(1, seqs)
        P = 128 * rng.randint(2, 127) + rng.choice([0, 1, 2, 64, 65, 127])
        check(B, R, rng.choice([1, 2, 3, 8]), P, P + rng.choice([0, 1, 70, 300]), rng.choice([1, 60, 500]), i)
    assert fa().get_device_error() == 0
