"""Infinite values that a row sees make its channel infinite with their sign, NaN beside the other infinity or a NaN,
wherever the value lies: in a tile that all rows of a unit see, at its edges, in a part of a unit.  Scores are small
enough (N(0, 1)) that no probability rounds to 0."""
import math

import numpy as np
import pytest
import torch

from tests import test_gpu_prefix as prefix
from tests import test_gpu_prompt as prompt
from tests.test_gpu_prompt import BF, HF, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error(kv):
    kv.kvarn_device_error()
    yield
    assert kv.kvarn_device_error() == 0


def put(c, b, j, h, ch, x):
    """x into the value of token j, where some row may see it."""
    P = c["vc"].shape[2]
    page = int(c["table"][b, j // P])
    if page < c["vc"].shape[0] and torch.isfinite(c["vc"][page, h, j % P]).all():
        c["vc"][page, h, j % P, ch] = x


def wanted(c, clean):
    """The sums of infinities and NaNs that each row sees added to the finite result."""
    want = np64(clean).copy()
    hq, hkv, P = c["q"].shape[1], c["vc"].shape[1], c["vc"].shape[2]
    vc, table, cu, lens = np64(c["vc"]), c["table"].cpu().numpy(), c["cu"].cpu().numpy(), c["lens"].cpu().numpy()
    starts = np.zeros(len(lens), int) if c["starts"] is None else np.maximum(c["starts"].cpu().numpy(), 0)
    for b in range(len(lens)):
        n, L = int(cu[b + 1] - cu[b]), int(lens[b])
        pos = L - n + np.arange(n)
        lo = np.maximum(starts[b], pos + 1 - c["window"] if c["window"] else 0)
        hi = np.minimum(pos + 1, L) if c["causal"] else np.full(n, L)
        j = np.arange(starts[b], L)
        page = table[b, j // P]
        j, page = j[page < len(vc)], page[page < len(vc)]
        v = vc[page, :, j % P]  # [tokens, Hkv, 128]
        odd = np.argwhere(~np.isfinite(v))
        for i, h, ch in odd:
            rows = cu[b] + np.flatnonzero((j[i] >= lo) & (j[i] < hi))
            heads = slice(h * hq // hkv, (h + 1) * hq // hkv)
            with np.errstate(invalid="ignore"):
                want[rows, heads, ch] += v[i, h, ch]
    return want


def check(got, want):
    assert np.array_equal(np.isnan(got), np.isnan(want))
    assert np.array_equal(np.isposinf(got), np.isposinf(want)) and np.array_equal(np.isneginf(got), np.isneginf(want))
    fin = np.isfinite(want)
    assert np.abs(got[fin] - want[fin]).max() <= 0.05


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("kw", [dict(), dict(window=100), dict(window=300, starts=[60, 0, 0]), dict(softcap=20.0), dict(causal=False)])
@pytest.mark.parametrize("hq,hkv", [(8, 2), (3, 3), (16, 1)])
def test_prompt(kv, dt, kw, hq, hkv):
    kw = dict(kw)
    softcap = kw.pop("softcap", 0.0)
    c = prompt.case(81, [400, 130, 70], [0, 3000, 5], hq, hkv, 16, dt, garbage=math.nan, **kw)
    clean, lse = prompt.call(kv, c, softcap=softcap)
    for b, j, h, ch, x in ((0, 70, 0, 3, math.inf), (0, 255, 0, 64, math.inf), (0, 256, hkv - 1, 127, -math.inf), (0, 399, 0, 0, math.inf),
                           (0, 5, 0, 3, math.inf), (0, 300, 0, 3, -math.inf), (0, 128, hkv - 1, 127, math.nan), (0, 390, 0, 64, math.inf),
                           (1, 3001, 0, 31, -math.inf), (1, 10, hkv - 1, 32, math.inf), (1, 1500, 0, 31, math.inf), (1, 2990, 0, 33, -math.inf),
                           (1, 3100, hkv - 1, 32, math.inf), (2, 74, 0, 95, math.inf), (2, 6, 0, 96, math.nan), (2, 40, 0, 95, math.inf)):
        put(c, b, j, h, ch, x)
    got, got_lse = prompt.call(kv, c, softcap=softcap)
    assert torch.equal(lse, got_lse)  # (values have no part in it)
    check(np64(got), wanted(c, clean))


def test_prompt_far_apart_edges_in_long_windows(kv):
    # the odd values lie at both edges of units thousands of tiles long
    c = prompt.case(82, [300], [200000], 4, 1, 128, BF, window=190000)
    clean, _ = prompt.call(kv, c)
    for j, ch, x in ((10200, 1, math.inf), (10150, 2, -math.inf), (200100, 1, math.inf), (200290, 2, math.inf), (200020, 5, math.nan)):
        put(c, 0, j, 0, ch, x)
    got, _ = prompt.call(kv, c)
    check(np64(got), wanted(c, clean))


@pytest.mark.parametrize("dt", [BF, HF])
def test_prefix(kv, dt):
    c = prefix.case(83, [500, 90], [6, 4], [40] * 12, 8, 2, 16, dt)
    clean, lse = prefix.call(kv, c)
    want = np64(clean).copy()
    for g, j, h, ch, x in ((0, 3, 0, 5, math.inf), (0, 499, 1, 6, -math.inf), (0, 250, 1, 7, math.nan), (1, 89, 0, 8, math.inf), (1, 1, 0, 8, -math.inf)):
        c["vc"][int(c["prefix_table"][g, j // 16]), h, j % 16, ch] = x
        with np.errstate(invalid="ignore"):
            want[6 * g:6 * g + (6, 4)[g], 4 * h:4 * h + 4, ch] += x
    got, got_lse = prefix.call(kv, c)
    assert torch.equal(lse, got_lse)
    check(np64(got), want)
