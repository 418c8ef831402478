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
