"""Attention over a shared prefix and own tokens, on the GPU against the fp64 oracle.  The prefix's part is
kvarn_prompt_attention's (test_gpu_prompt.py derives its bound); joining two parts by their log-sum-exps adds twice
2^-23 of them (their own rounding) and 2^-20, the own part's bound lies below the prefix's."""
import math

import numpy as np
import pytest
import torch

from oracle import serving as o
from tests.test_gpu_prompt import BF, HF, SCALE, bounds, i32, make_cache, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error(kv):
    kv.kvarn_device_error()
    yield
    assert kv.kvarn_device_error() == 0


def case(seed, prefix, sizes, tails, hq, hkv, P=16, dt=BF, layout="hnd", before=0, **kw):
    """before: sequences before the first group; those behind the last one are what tails has left."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    G, B = len(prefix), len(tails)
    lens = list(prefix) + list(tails)
    kc, vc, table = make_cache(g, lens, [0] * len(lens), hkv, P, dt, layout, **kw)
    q = torch.randn(B, hq, 128, generator=g, device="cuda").to(dt)
    cu = np.concatenate([[0], np.cumsum(sizes)]) + before
    return dict(q=q, kc=kc, vc=vc, prefix_table=table[:G].contiguous(), table=table[G:].contiguous(), cu=i32(cu.tolist()),
                prefix_lens=i32(list(prefix)), lens=i32(list(tails)), dt=dt)


def call(kv, c, scale=SCALE, softcap=0.0, ws=None, stream=None, out=None, lse=None):
    B, hq = c["q"].shape[:2]
    if ws is None:
        n = kv.kvarn_prefix_attention_workspace_size(B, hq, c["kc"].shape[1])
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    if out is None:
        out = torch.full((B, hq, 128), math.nan, dtype=c["dt"], device="cuda")
    if lse is None:
        lse = torch.full((B, hq), math.nan, device="cuda")
    kv.kvarn_prefix_attention(c["q"], c["kc"], c["vc"], c["prefix_table"], c["prefix_lens"], c["cu"], c["table"], c["lens"],
                              out, scale, ws, softcap=softcap, lse=lse, stream=stream)
    return out, lse


def check(c, out, lse, scale=SCALE, softcap=0.0):
    want, want_lse, mass, reach, count = o.prefix_attention(
        np64(c["q"]), np64(c["kc"]), np64(c["vc"]), c["prefix_table"].cpu().numpy(), c["prefix_lens"].cpu().numpy(),
        c["cu"].cpu().numpy(), c["table"].cpu().numpy(), c["lens"].cpu().numpy(), scale, softcap)
    tol, lse_tol = bounds(want, want_lse, mass, reach, count, c["dt"], softcap)
    fin = np.isfinite(want_lse)
    tol += ((2.0 ** -20 + 2.0 ** -22 * np.abs(np.where(fin, want_lse, 0.0)))[..., None]) * mass
    got, got_lse = np64(out), np64(lse)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], bad.mean(), np.abs(got - want)[bad][:4], tol[bad][:4])
    assert np.array_equal(np.isneginf(got_lse), np.isneginf(want_lse))
    assert np.all(np.abs(got_lse[fin] - want_lse[fin]) <= lse_tol[fin] + 2.0 ** -20)


@pytest.mark.parametrize("hq,hkv", [(1, 1), (8, 2), (5, 1), (32, 2), (71, 1), (12, 12)])
@pytest.mark.parametrize("P,layout,dt", [(16, "hnd", BF), (48, "nhd", HF), (128, "both", BF)])
def test_matches_the_oracle(kv, hq, hkv, P, layout, dt):
    c = case(hq + P, [300, 5, 129], [4, 1, 7], [1, 30, 0, 200, 17, 1, 1, 2, 3, 4, 5, 6], hq, hkv, P, dt, layout)
    check(c, *call(kv, c))


@pytest.mark.parametrize("prefix,sizes,tails,before", [
    ([0], [2], [1, 0], 0), ([1], [1], [0], 0), ([128], [1], [1], 0), ([4000], [70], [3] * 70, 0), ([9000], [1], [1], 0),
    ([50, 60], [0, 3], [5, 5, 5], 0), ([50], [2], [5, 0, 9, 0, 4], 2), ([700] * 20, [2] * 20, [40] * 40, 0),
    ([257, 0, 31], [3, 3, 3], [0] * 9, 0), ([2000, 1], [300, 1], [1] * 301, 0)])
def test_lengths(kv, prefix, sizes, tails, before):
    c = case(sum(prefix) + len(tails), prefix, sizes, tails, 8, 2, 16, before=before)
    check(c, *call(kv, c))


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("kw", [dict(softcap=20.0), dict(scale=-0.2), dict(scale=0.6), dict(scale=0.0)])
def test_modifiers(kv, kw, dt):
    c = case(3, [500, 90], [6, 4], [100, 1, 5, 60, 2, 3, 128, 16, 9, 10], 8, 2, 32, dt)
    check(c, *call(kv, c, **kw), **kw)


def test_equals_plain_decode_attention_over_prefix_and_own_tokens(kv):
    # pages of the prefix are full: the same keys as one page table, through the decode attention
    c = case(11, [512], [5], [70, 1, 33, 64, 128], 8, 2, 64)
    out, lse = call(kv, c)
    table = torch.cat([c["prefix_table"][:, :8].expand(5, 8), c["table"]], 1).contiguous()
    ws = torch.empty(kv.kvarn_paged_attention_workspace_size(5, 8, 2), dtype=torch.uint8, device="cuda")
    want, want_lse = torch.empty(5, 8, 128, device="cuda"), torch.empty(5, 8, device="cuda")
    kv.kvarn_paged_attention(c["q"], c["kc"], c["vc"], table, c["lens"] + 512, want, SCALE, ws, lse=want_lse)
    assert (lse - want_lse).abs().max() <= 1e-4
    assert (out.float() - want).norm() <= 2.0 ** -8 * want.norm()
