"""Attention of many new tokens per sequence over a paged cache, on the GPU against the fp64 oracle.

Tolerances, from the arithmetic.  A product step takes 16 terms, aligned to its largest with 21 bits at least below
it, and adds them to an fp32 sum: off by at most 17 * 2^-22 of the step's largest term and 2^-23 of the sum, so a
score (8 steps) is off by 2^-17 of reach = |scale| max_j sum |q k|; capping keeps that (tanh has slope <= 1, and its
own 2^-21 cap), the bias adds 2^-23 of itself.  A probability is off by twice the score's error plus 2^-20 (exp2),
and by its rounding to the cache's type: half a step (2^-8 bf16, 2^-11 fp16), for fp16 below the normal numbers
2^-32 of the row's largest.  Its product with the values adds 2^-17 and 2^-23 for each 16 keys.  So out is off by
that times sum p |v|, plus the output's rounding; lse by the score's error and the sum's, 2^-24 for each of a
thread's additions (64 and one for each 128 keys), 2^-20 and 2^-22 of itself.
"""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import serving as o
from tests.test_gpu_graph import _capture

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
HALF_STEP = {BF: 2.0 ** -8, HF: 2.0 ** -11}
SCALE = 1 / math.sqrt(128)
FILL = 0.75  # what rows outside the sequences hold before and after


@pytest.fixture(autouse=True)
def _no_device_error(kv):
    kv.kvarn_device_error()
    yield
    assert kv.kvarn_device_error() == 0


def np64(t):
    return t.detach().double().cpu().numpy()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def make_cache(g, lens, lows, hkv, P, dt, layout="hnd", garbage=float("nan"), spare=3, spread=1.0, width=None):
    """Pages of sequences of these lengths; every slot outside tokens lows[b] .. lens[b] holds `garbage`, every unused
    page table entry an id far outside."""
    B, used = len(lens), [-(-n // P) for n in lens]
    width, n_pages = width or max(used + [0]) + 1, sum(used) + spare
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, width), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    shape = {"hnd": (n_pages, hkv, P, 128), "nhd": (n_pages, P, hkv, 128), "both": (n_pages, 2, hkv, P, 136)}[layout]
    if layout == "both":
        both = torch.full(shape, garbage, dtype=dt, device="cuda")
        kc, vc = both[:, 0, :, :, :128], both[:, 1, :, :, :128]
    else:
        kc, vc = (torch.full(shape, garbage, dtype=dt, device="cuda") for _ in range(2))
        if layout == "nhd":
            kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    at = 0
    for b, n in enumerate(lens):
        lo = min(max(lows[b], 0), n)
        if n > lo:
            j = torch.arange(lo, n, device="cuda")
            pages = perm[at:at + used[b]]
            table[b, lo // P:used[b]] = pages[lo // P:]
            kc[pages[j // P].long(), :, j % P] = (spread * torch.randn(n - lo, hkv, 128, generator=g, device="cuda")).to(dt)
            vc[pages[j // P].long(), :, j % P] = torch.randn(n - lo, hkv, 128, generator=g, device="cuda").to(dt)
        at += used[b]
    return kc, vc, table


def case(seed, new, ctx, hq, hkv, P=16, dt=BF, layout="hnd", starts=None, window=0, causal=True, spare_rows=0, **kw):
    g = torch.Generator(device="cuda").manual_seed(seed)
    lens = [a + b for a, b in zip(new, ctx)]
    lows = [max(0 if starts is None else starts[b], (c + 1 - window) if window else 0) for b, c in enumerate(ctx)]
    kc, vc, table = make_cache(g, lens, lows, hkv, P, dt, layout, **kw)
    T = sum(new) + spare_rows
    q = torch.randn(T, hq, 128, generator=g, device="cuda").to(dt)
    cu = i32(np.concatenate([[0], np.cumsum(new)]).tolist())
    return dict(q=q, kc=kc, vc=vc, table=table, cu=cu, lens=i32(lens), starts=None if starts is None else i32(starts),
                window=window, causal=causal, dt=dt)


def call(kv, c, scale=SCALE, softcap=0.0, slopes=None, ws=None, stream=None, out=None, lse=None, with_lse=True):
    T, hq = c["q"].shape[:2]
    if ws is None:
        n = kv.kvarn_prompt_attention_workspace_size(T, hq, c["kc"].shape[1])
        ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    if out is None:
        out = torch.full((T, hq, 128), FILL, dtype=c["dt"], device="cuda")
    if lse is None and with_lse:
        lse = torch.full((T, hq), FILL, device="cuda")
    kv.kvarn_prompt_attention(c["q"], c["kc"], c["vc"], c["table"], c["cu"], c["lens"], out, scale, ws, causal=c["causal"],
                              softcap=softcap, slopes=slopes, window=c["window"], kv_starts=c["starts"], lse=lse, stream=stream)
    return out, lse


def bounds(want, want_lse, mass, reach, count, dt, softcap=0.0, bias=0.0):
    err = reach * 2.0 ** -17 + softcap * 2.0 ** -21 + np.abs(bias) * 2.0 ** -22
    p = 2 * err + 2.0 ** -20 + HALF_STEP[dt] + 2.0 ** -17 + count / 16 * 2.0 ** -23
    tol = p[..., None] * mass + HALF_STEP[dt] * np.abs(want) + float(torch.finfo(dt).smallest_normal)
    if dt == HF:
        tol += (count * 2.0 ** -32)[..., None] * 8  # values of the tests' N(0, 1)
    return tol, err + (64 + count / 128) * 2.0 ** -24 + 2.0 ** -20 + 2.0 ** -22 * np.abs(want_lse)


def check(c, out, lse, scale=SCALE, softcap=0.0, slopes=None):
    want, want_lse, mass, reach, count = o.prompt_attention(
        np64(c["q"]), np64(c["kc"]), np64(c["vc"]), c["table"].cpu().numpy(), c["cu"].cpu().numpy(), c["lens"].cpu().numpy(),
        scale, c["causal"], softcap, None if slopes is None else np64(slopes), c["window"],
        None if c["starts"] is None else c["starts"].cpu().numpy())
    got, rows = np64(out), ~np.isnan(want_lse)
    assert np.all(got[~rows] == FILL)
    bias = 0.0 if slopes is None else np64(slopes)[None] * float(c["lens"].max())
    tol, lse_tol = bounds(want, want_lse, mass, reach, count, c["dt"], softcap, bias)
    nan = np.isnan(want)
    assert not np.isfinite(got[nan & rows[..., None]]).any()
    with np.errstate(invalid="ignore"):
        bad = ~(np.abs(got - want) <= tol) & ~nan & rows[..., None]
    assert not bad.any(), (np.argwhere(bad)[:4], bad.mean(), np.abs(got - want)[bad][:4], tol[bad][:4])
    if lse is None:
        return
    got_lse = np64(lse)
    assert np.all(got_lse[~rows] == FILL)
    assert np.array_equal(np.isneginf(got_lse), np.isneginf(want_lse))
    fin = np.isfinite(want_lse)
    assert np.all(np.abs(got_lse[fin] - want_lse[fin]) <= lse_tol[fin])


def test_one_tile(kv):
    c = case(0, [128], [0], 1, 1)
    check(c, *call(kv, c))


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (8, 1), (8, 2), (5, 1), (32, 2), (17, 1), (71, 1), (12, 4)])
@pytest.mark.parametrize("P,layout,dt", [(16, "hnd", BF), (48, "nhd", HF), (128, "both", BF), (32, "hnd", HF), (256, "nhd", BF)])
def test_matches_the_oracle(kv, hq, hkv, P, layout, dt):
    c = case(hq * 100 + P, [5, 1, 0, 130, 300, 64, 1], [0, 40, 17, 200, 0, 0, 700], hq, hkv, P, dt, layout, spare_rows=3)
    check(c, *call(kv, c))


@pytest.mark.parametrize("new,ctx", [
    ([1], [0]), ([1], [1]), ([0], [5]), ([1], [127]), ([1], [128]), ([1, 0, 0, 1], [0, 0, 9, 5000]), ([2] * 40, [1] * 40),
    ([0, 0, 0], [1, 2, 3]), ([31, 33, 127, 129], [0, 0, 0, 0]), ([1500], [0]), ([1], [9000]), ([700], [3000]),
    ([1] * 300, list(range(300)))])
def test_lengths(kv, new, ctx):
    c = case(sum(new) + sum(ctx), new, ctx, 8, 2, 16)
    check(c, *call(kv, c))


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("kw", [
    dict(softcap=30.0), dict(slopes=True), dict(window=1), dict(window=100), dict(window=129), dict(window=5000),
    dict(starts=True), dict(starts=True, window=200, softcap=5.0), dict(slopes=True, window=77, starts=True), dict(causal=False),
    dict(causal=False, starts=True, softcap=20.0), dict(scale=-0.1), dict(scale=0.0), dict(scale=0.5)])
def test_modifiers(kv, kw, dt):
    new, ctx = [300, 7, 1, 129, 40], [0, 900, 600, 33, 128]
    kw = dict(kw)
    if kw.pop("starts", False):
        kw["starts"] = [10, 700, 601, 0, 500]  # behind some rows' positions, and behind all of a sequence's keys
    slopes = 2.0 ** -torch.arange(1, 9, device="cuda", dtype=F32) if kw.pop("slopes", False) else None
    softcap, scale = kw.pop("softcap", 0.0), kw.pop("scale", SCALE)
    c = case(7, new, ctx, 8, 2, 48, dt, **kw)
    check(c, *call(kv, c, scale=scale, softcap=softcap, slopes=slopes), scale=scale, softcap=softcap, slopes=slopes)


def test_many_rows_without_keys_between_others(kv):
    # runs of units that see nothing, longer than any look-ahead, behind units that do
    new = [40, 3, 70, 9, 1, 33, 64, 5] * 80
    starts = [0 if i % 8 == 0 else 10000 for i in range(len(new))]
    c = case(21, new, [30] * len(new), 8, 2, 16, starts=starts)
    check(c, *call(kv, c))
    # and inside one sequence, for each head
    c = case(22, [2500, 60], [0, 10], 8, 8, 48, HF, starts=[2000, 0], window=200)
    check(c, *call(kv, c))


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("kw", [dict(), dict(window=100), dict(window=300, starts=[60, 0, 0]), dict(softcap=20.0), dict(causal=False)])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (3, 3), (16, 1)])
def test_infinite_and_nan_values_reach_only_the_rows_that_see_them(kv, dt, kw, hq, hkv):
    kw = dict(kw)
    softcap = kw.pop("softcap", 0.0)
    c = case(31, [400, 130, 70], [0, 300, 5], hq, hkv, 16, dt, **kw)
    start = 0 if c["starts"] is None else 60
    for b, j, h, ch, x in ((0, 70, 0, 3, math.nan), (0, 255, 0, 64, math.inf), (0, 256, hkv - 1, 127, -math.inf), (0, 399, 0, 0, math.nan),
                           (1, 301, 0, 31, math.nan), (1, 10, hkv - 1, 32, math.inf), (2, 74, 0, 95, math.inf), (2, 6, 0, 96, math.nan)):
        page = int(c["table"][b, j // 16])
        if page < c["vc"].shape[0] and (j >= start or b):  # (a window may leave a page unused)
            c["vc"][page, h, j % 16, ch] = x
    # keys that a row does not see have no part either
    c["kc"][int(c["table"][0, 399 // 16]), 0, 399 % 16] = math.nan
    want = o.prompt_attention(np64(c["q"]), np64(c["kc"]), np64(c["vc"]), c["table"].cpu().numpy(), c["cu"].cpu().numpy(),
                              c["lens"].cpu().numpy(), SCALE, c["causal"], softcap, None, c["window"],
                              None if c["starts"] is None else c["starts"].cpu().numpy())[0]
    out, lse = call(kv, c, softcap=softcap)
    got = np64(out)
    if c["causal"]:  # the row with the NaN key is one token's; the others are as without it
        rows = np.ones(len(got), bool)
        rows[399] = False
        assert np.array_equal(np.isfinite(got[rows]), np.isfinite(want[rows]))
        ok = np.isfinite(want) & rows[:, None, None]
        assert np.abs(got - want)[ok].max() <= 0.05
    assert not np.isfinite(got[np.isnan(want)]).any()


@pytest.mark.parametrize("garbage", [math.inf, -math.inf, 6e4, -6e4])
def test_garbage_of_every_kind_stays_out(kv, garbage):
    c = case(41, [200, 3, 40], [70, 0, 1000], 8, 2, 48, BF, starts=[11, 0, 300], window=500, garbage=garbage)
    check(c, *call(kv, c))


def test_bad_pages_count_as_zeros_and_are_reported(kv):
    c = case(42, [200, 60], [100, 0], 4, 2, 16)
    c["table"][0, 3], c["table"][0, 17], c["table"][1, 2] = -1, c["kc"].shape[0], 2 ** 30
    out, lse = call(kv, c)
    assert kv.kvarn_device_error() == 64
    check(c, out, lse)


def test_lengths_past_the_table_and_rows_without_a_place_are_clamped(kv):
    c = case(43, [50, 20, 9], [0, 30, 0], 4, 2, 16)
    c["lens"].copy_(i32([10 ** 9, 50, -5]))  # the first is cut to what its table holds, the last to 0
    c["kc"][~torch.isfinite(c["kc"])] = 0
    c["vc"][~torch.isfinite(c["vc"])] = 0
    out, lse = call(kv, c)
    check(c, out, lse)
    assert torch.all(out[70:] == 0) and torch.isneginf(lse[70:]).all()
    kv.kvarn_device_error()  # (the first sequence's last page table entries name no page)
    # cu_tokens past the rows that there are
    c = case(44, [50, 20], [0, 30], 4, 2, 16)
    c["q"] = c["q"][:60].contiguous()
    out, lse = call(kv, c)
    c["cu"] = i32([0, 50, 60])
    check(c, out, lse)


@pytest.mark.parametrize("hq,hkv", [(8, 2), (10, 2)])
def test_strided_and_repeated_queries(kv, hq, hkv):
    c = case(45, [130, 5], [10, 400], hq, hkv, 32)
    wide = torch.randn(135, hq + 5, 136, device="cuda").to(BF)
    for q in (wide[:, 2:2 + hq, :128], wide.transpose(0, 1)[:hq].transpose(0, 1)[..., 8:], wide[:1, :hq, :128].expand(135, hq, 128),
              wide[:, :1, :128].expand(135, hq, 128)):
        check({**c, "q": q}, *call(kv, {**c, "q": q}))


def test_outputs_at_odd_places(kv):
    # 16-byte but not 32-byte aligned
    c = case(46, [100, 3], [0, 50], 8, 2)
    flat = torch.full((103 * 8 * 128 + 8,), FILL, dtype=BF, device="cuda")
    out = flat[8:].view(103, 8, 128)
    lse = torch.full((103 * 8 + 1,), FILL, device="cuda")[1:].view(103, 8)
    check(c, *call(kv, c, out=out, lse=lse))
    assert torch.all(flat[:8] == FILL)


def test_repeats_bit_for_bit_and_ignores_the_workspace(kv):
    c = case(47, [700, 17, 300, 1], [2000, 0, 9, 5000], 16, 2, 64)
    n = kv.kvarn_prompt_attention_workspace_size(c["q"].shape[0], 16, 2)
    a = call(kv, c, ws=torch.zeros(n, dtype=torch.uint8, device="cuda"))
    b = call(kv, c, ws=torch.full((n,), 127, dtype=torch.uint8, device="cuda"))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    out, _ = call(kv, c, with_lse=False)
    assert torch.equal(out, a[0])


def test_single_tokens_equal_the_decode_attention(kv):
    lens = [1, 40, 900, 128, 3001]
    c = case(48, [1] * 5, [n - 1 for n in lens], 8, 2, 32, window=700)
    out, lse = call(kv, c)
    ws = torch.empty(kv.kvarn_paged_attention_workspace_size(5, 8, 2), dtype=torch.uint8, device="cuda")
    want, want_lse = torch.empty(5, 8, 128, device="cuda"), torch.empty(5, 8, device="cuda")
    kv.kvarn_paged_attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], want, SCALE, ws, window=700, lse=want_lse)
    assert (lse - want_lse).abs().max() <= 1e-4 and (out.float() - want).norm() <= 2.0 ** -8 * want.norm()


def test_cache_past_32_bit_offsets(kv):
    P, n_pages, hkv = 128, 17000, 8  # 2.2e9 elements per cache: the pages in use are the last ones
    kc, vc = (torch.empty(n_pages, P, hkv, 128, dtype=BF, device="cuda").transpose(1, 2) for _ in range(2))
    c = case(49, [200, 30], [100, 99], 16, hkv, P, layout="nhd", garbage=0.0)
    small = c["kc"].shape[0]
    for big, src in ((kc, c["kc"]), (vc, c["vc"])):
        big[n_pages - small:] = src
    want = call(kv, c)
    far = dict(c, kc=kc, vc=vc, table=torch.where(c["table"] < small, c["table"] + (n_pages - small), c["table"]))
    got = call(kv, far)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    check(c, *got)


def test_graphs_share_a_workspace_and_follow_the_lengths(kv):
    c1, c2 = case(50, [300, 60], [900, 0], 8, 2, 32), case(51, [40, 9, 500], [0, 70, 100], 8, 2, 16)
    ws = torch.empty(kv.kvarn_prompt_attention_workspace_size(549, 8, 2), dtype=torch.uint8, device="cuda")
    outs = [(torch.empty_like(c["q"]), torch.empty(c["q"].shape[:2], device="cuda")) for c in (c1, c2)]
    g1 = _capture(lambda: call(kv, c1, ws=ws, out=outs[0][0], lse=outs[0][1]))
    g2 = _capture(lambda: call(kv, c2, ws=ws, out=outs[1][0], lse=outs[1][1]))
    for cu, lens in (([0, 300, 360], [1200, 60]), ([0, 1, 1], [700, 0]), ([5, 300, 340], [300, 41])):
        c1["cu"].copy_(i32(cu))
        c1["lens"].copy_(i32(lens))
        for t in outs[0] + outs[1]:
            t.fill_(FILL)
        for _ in range(3):
            g1.replay()
            g2.replay()
        torch.cuda.synchronize()
        for c, got in ((c1, outs[0]), (c2, outs[1])):
            want = call(kv, c)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_side_streams_with_their_own_workspaces(kv):
    cs = [case(52 + i, [200, 10 * i, 99], [1000, 5, 0], 8, 2, 32) for i in range(3)]
    want = [call(kv, c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = []
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((i, call(kv, cs[i])))
    torch.cuda.synchronize()
    for i, (out, lse) in got:
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


def test_many_sequences(kv):
    # more than one CTA's warps can count at once, most of them without rows
    new = [0] * 5000
    for b in range(0, 5000, 37):
        new[b] = 1 + b % 5
    c = case(60, new, [b % 90 if n else 0 for b, n in enumerate(new)], 4, 1, 16)
    check(c, *call(kv, c))


def test_as_many_sequences_as_a_call_takes(kv):
    new = [0] * 16384
    for b in (0, 1, 31, 8191, 8192, 16383):
        new[b] = 1 + b % 3
    c = case(62, new, [b % 50 if n else 0 for b, n in enumerate(new)], 4, 2, 16)
    check(c, *call(kv, c))


@pytest.mark.parametrize("window", [0, 1, 40, 2 ** 31 - 1])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_more_rows_than_tokens(kv, window, softcap):
    # rows before position 0 see nothing; the widest window there is hides nothing from the others
    c = case(63, [300, 70, 9], [0, 0, 0], 8, 2, 32)
    c["lens"], c["window"] = i32([170, 1, 0]), window
    check(c, *call(kv, c, softcap=softcap), softcap=softcap)


@pytest.mark.parametrize("scale,softcap", [(0.0, 30.0), (-SCALE, 30.0), (SCALE, 0.02), (30 * SCALE, 5.0), (3e38, 2.0 ** -126)])
def test_capped_scores_beside_hidden_garbage(kv, scale, softcap):
    # hidden keys hold NaN or infinities; scores of 0, of either sign, far past the cap; a scale over the cap past fp32
    for garbage in (float("nan"), float("inf")):
        c = case(64, [150, 3], [61, 0], 8, 2, 16, garbage=garbage, starts=[17, 0])
        if scale > 1:
            c["q"].zero_()
        check(c, *call(kv, c, scale=scale, softcap=softcap), scale=scale, softcap=softcap)


def test_a_capped_row_with_a_nan_score_is_nan(kv):
    c = case(65, [200], [0], 4, 1, 16)
    page, slot = int(c["table"][0, 100 // 16]), 100 % 16
    c["kc"][page, 0, slot, 3] = float("nan")
    out, lse = call(kv, c, softcap=30.0)
    assert torch.isnan(out[100:]).all() and torch.isnan(lse[100:]).all()
    assert torch.isfinite(out[:100]).all() and torch.isfinite(lse[:100]).all()


@pytest.mark.parametrize("seed", range(12))
def test_random_cases(kv, seed):
    rng = np.random.default_rng(1000 + seed)
    B = int(rng.integers(1, 9))
    new = [int(x) for x in rng.integers(0, rng.choice([3, 40, 400]), B)]
    ctx = [int(x) for x in rng.integers(0, rng.choice([2, 200, 3000]), B)]
    hq, hkv = [(8, 2), (5, 1), (6, 6), (16, 1), (12, 4), (40, 2)][int(rng.integers(6))]
    causal = bool(rng.random() < 0.8)
    kw = dict(causal=causal, window=int(rng.integers(1, 700)) if causal and rng.random() < 0.5 else 0,
              starts=[int(x) for x in rng.integers(-3, 300, B)] if rng.random() < 0.4 else None)
    softcap = 25.0 if rng.random() < 0.3 else 0.0
    slopes = 2.0 ** -torch.arange(1, hq + 1, device="cuda", dtype=F32) if causal and rng.random() < 0.3 else None
    c = case(seed, new, ctx, hq, hkv, int(rng.choice([16, 48, 64, 128, 272])), BF if rng.random() < 0.5 else HF,
             str(rng.choice(["hnd", "nhd", "both"])), spare_rows=int(rng.integers(0, 5)), **kw)
    check(c, *call(kv, c, softcap=softcap, slopes=slopes), softcap=softcap, slopes=slopes)


def test_python_refusals(kv):
    c = case(61, [20], [0], 4, 2)
    for change, match in ((dict(lens=c["lens"].long()), "kv_lens"), (dict(q=c["q"].half()), "k_cache"), (dict(cu=c["cu"][:1]), "cu_tokens"),
                          (dict(table=c["table"][0]), "page_table"), (dict(q=c["q"].cpu()), "current CUDA"), (dict(lens=i32([20, 3])), "kv_lens"),
                          (dict(vc=c["vc"].transpose(1, 2)), "v_cache"), (dict(q=c["q"][..., :64]), "q")):
        with pytest.raises(ValueError, match=match):
            call(kv, {**c, **change})
    with pytest.raises(ValueError, match="out"):
        call(kv, c, out=torch.empty(20, 4, 128, device="cuda"))
    with pytest.raises(kv.KvarnError, match="workspace"):
        call(kv, c, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(kv.KvarnError, match="window"):
        call(kv, {**c, "causal": False, "window": 5})


def test_first_calls_of_a_process_may_be_captured(kv):
    code = """
import torch, bit_kv_cache_kvarn_gb300 as kv
kv.load()
i32 = dict(dtype=torch.int32, device="cuda")
q = torch.randn(40, 4, 128, device="cuda").to(torch.bfloat16)
kc, vc = (torch.randn(4, 2, 16, 128, device="cuda").to(torch.bfloat16) for _ in range(2))
table, cu, lens = torch.arange(4, **i32)[None], torch.tensor([0, 40], **i32), torch.tensor([60], **i32)
out, lse = torch.empty_like(q), torch.empty(40, 4, device="cuda")
ws = torch.empty(kv.kvarn_prefix_attention_workspace_size(40, 4, 2), dtype=torch.uint8, device="cuda")
pre, pre_lse = torch.empty_like(q), torch.empty(40, 4, device="cuda")
own, none = table.expand(40, 4).contiguous(), torch.full((40,), 9, **i32)
c8 = [torch.zeros(4, 2, 16, 128, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
e8 = [torch.zeros(4, 2, 16, dtype=torch.int8, device="cuda") for _ in range(2)]
dec = torch.empty(1, 4, 128, device="cuda")
flat = [x.transpose(1, 2).reshape(64, 2, 128) for x in (kc, vc)]

def step():
    kv.kvarn_prompt_attention(q, kc, vc, table, cu, lens, out, 0.1, ws, lse=lse)
    kv.kvarn_prefix_attention(q, kc, vc, table, lens, cu, own, none, pre, 0.1, ws, lse=pre_lse)
    kv.kvarn_quantize_kv(*flat, *c8, *e8)
    kv.kvarn_paged_attention_q8(q[39:], *c8, *e8, table, lens, dec, 0.1, ws)

torch.cuda.synchronize()
s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
with torch.cuda.stream(s):
    with torch.cuda.graph(g, stream=s):
        step()
g.replay()
torch.cuda.synchronize()
first = [t.clone() for t in (out, lse, pre, pre_lse, dec)]
assert all(torch.isfinite(t).all() and t.abs().max() > 0 for t in first)
step()
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(first, (out, lse, pre, pre_lse, dec))) and kv.kvarn_device_error() == 0
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
