"""Attention over a shared prefix and own tokens, on the GPU against the fp64 oracle.  The prefix's part is
kvarn_prompt_attention's (test_gpu_prompt.py derives its bound); joining two parts by their log-sum-exps adds twice
2^-23 of them (their own rounding) and 2^-20, the own part's bound lies below the prefix's."""
import math

import numpy as np
import pytest
import torch

from oracle import serving as o
from tests.test_gpu_graph import _capture
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


def test_no_groups_is_the_decode_attention(kv):
    c = case(12, [], [], [70, 1, 0], 8, 2, 32)
    assert c["prefix_table"].shape[0] == 0
    out, lse = call(kv, c)
    check(c, out, lse)


def test_bad_pages_count_as_zeros_and_are_reported(kv):
    c = case(13, [100, 40], [2, 1], [30, 5, 9, 70], 4, 2, 16)
    c["prefix_table"][0, 3], c["table"][3, 1] = -7, 2 ** 30
    out, lse = call(kv, c)
    assert kv.kvarn_device_error() == 64
    check(c, out, lse)


def test_strided_queries_repeat_bit_for_bit_and_ignore_the_workspace(kv):
    c = case(14, [3000, 5], [9, 2], list(range(12)), 8, 2, 16)
    wide = torch.randn(12, 13, 136, device="cuda").to(BF)
    c["q"] = wide[:, 2:10, :128]
    n = kv.kvarn_prefix_attention_workspace_size(12, 8, 2)
    a = call(kv, c, ws=torch.zeros(n, dtype=torch.uint8, device="cuda"))
    b = call(kv, c, ws=torch.full((n,), 127, dtype=torch.uint8, device="cuda"))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check(c, *a)
    c["q"] = wide[:1, :8, :128].expand(12, 8, 128)
    check(c, *call(kv, c))


def test_graphs_share_a_workspace_and_follow_the_lengths(kv):
    c1, c2 = case(15, [2000], [8], [50] * 8, 8, 2, 32), case(16, [40, 900], [3, 5], [70, 1, 2, 3, 300, 5, 6, 7], 8, 2, 16)
    ws = torch.empty(kv.kvarn_prefix_attention_workspace_size(8, 8, 2), dtype=torch.uint8, device="cuda")
    outs = [(torch.empty_like(c["q"]), torch.empty(8, 8, device="cuda")) for c in (c1, c2)]
    g1 = _capture(lambda: call(kv, c1, ws=ws, out=outs[0][0], lse=outs[0][1]))
    g2 = _capture(lambda: call(kv, c2, ws=ws, out=outs[1][0], lse=outs[1][1]))
    for cu, prefix, tail in (([0, 8], [2000], 50), ([2, 5], [1], 0), ([0, 0], [77], 33)):
        c1["cu"].copy_(i32(cu))
        c1["prefix_lens"].copy_(i32(prefix))
        c1["lens"].fill_(tail)
        for t in outs[0] + outs[1]:
            t.fill_(math.nan)
        for _ in range(3):
            g1.replay()
            g2.replay()
        torch.cuda.synchronize()
        for c, got in ((c1, outs[0]), (c2, outs[1])):
            want = call(kv, c)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_side_streams_with_their_own_workspaces(kv):
    cs = [case(17 + i, [500 * i, 3], [4, 2], [20, 1, 0, 9, 300, 8], 8, 2, 32) for i in range(3)]
    want = [call(kv, c) for c in cs]
    torch.cuda.synchronize()
    got = []
    for i, s in enumerate([torch.cuda.Stream() for _ in cs] * 3):
        with torch.cuda.stream(s):
            got.append((i % 3, call(kv, cs[i % 3])))
    torch.cuda.synchronize()
    for i, (out, lse) in got:
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


@pytest.mark.parametrize("seed", range(8))
def test_random_cases(kv, seed):
    rng = np.random.default_rng(2000 + seed)
    G = int(rng.integers(1, 5))
    sizes = [int(x) for x in rng.integers(0, 20, G)]
    before, after = (int(x) for x in rng.integers(0, 3, 2))
    B = sum(sizes) + before + after
    if B == 0:
        sizes[0], B = 1, 1
    hq, hkv = [(8, 2), (5, 1), (6, 6), (16, 1), (12, 4), (40, 2)][int(rng.integers(6))]
    c = case(seed, [int(x) for x in rng.integers(0, rng.choice([3, 300, 3000]), G)], sizes,
             [int(x) for x in rng.integers(0, rng.choice([2, 60, 600]), B)], hq, hkv, int(rng.choice([16, 48, 128])),
             BF if rng.random() < 0.5 else HF, str(rng.choice(["hnd", "nhd", "both"])), before=before)
    softcap = 25.0 if rng.random() < 0.3 else 0.0
    check(c, *call(kv, c, softcap=softcap), softcap=softcap)


def test_python_refusals(kv):
    c = case(20, [20], [2], [5, 6], 4, 2)
    for change, match in ((dict(prefix_lens=c["prefix_lens"].long()), "prefix_lens"), (dict(cu=c["cu"][:1]), "cu_seqs"),
                          (dict(table=c["table"][:1]), "page_table"), (dict(prefix_table=c["prefix_table"][0]), "prefix_table"),
                          (dict(q=c["q"].half()), "k_cache"), (dict(lens=i32([1])), "kv_lens")):
        with pytest.raises(ValueError, match=match):
            call(kv, {**c, **change})
    with pytest.raises(kv.KvarnError, match="workspace"):
        call(kv, c, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
