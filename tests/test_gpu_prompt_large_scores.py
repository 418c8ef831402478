"""Scores far past 2^24, where neighbouring fp32 numbers lie a power of two or more apart in the exponent.

The products are exact (few non-zero channels, or equal ones), so a probability is off by the rounding of its
difference to the maximum: 2^-24 of that, 2^-24 of it again by the scale's own rounding and the log's, below 2^-17 of a probability
that counts (differences up to 64).  With reach 1 in test_gpu_prompt.py's bounds a score is off by 2^-17, which covers it;
lse by 2^-22 of itself, as there.  The biased kernel rounds each score to fp32 in the log2 domain before its maximum is
known: 2^-24 of the score by that, 2^-24 by the scale's rounding, so 2^-23 of the score more, which is several powers of two
here: its outputs have to be finite averages of the values, its lse what it is."""
import numpy as np
import pytest
import torch

from oracle import serving as o
from tests import test_gpu_prefix as prefix
from tests import test_gpu_prompt as prompt
from tests.test_gpu_prompt import BF, HF, SCALE, bounds, np64

pytestmark = pytest.mark.gpu
LN2 = float(np.log(2.0))


@pytest.fixture(autouse=True)
def _no_device_error(kv):
    kv.kvarn_device_error()
    yield
    assert kv.kvarn_device_error() == 0


def check(c, out, lse, scale, want, rounded=False):
    want, want_lse, mass, reach, count = want
    reach = 1 + (2.0 ** -6 * np.abs(want_lse) if rounded else np.zeros_like(reach))
    tol, lse_tol = bounds(want, want_lse, mass, reach, count, c["dt"])
    got, got_lse = np64(out), np64(lse)
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], bad.mean(), got[bad][:4], want[bad][:4], tol[bad][:4])
    assert np.all(np.abs(got_lse - want_lse) <= lse_tol)


def prompt_want(c, scale):
    return o.prompt_attention(np64(c["q"]), np64(c["kc"]), np64(c["vc"]), c["table"].cpu().numpy(), c["cu"].cpu().numpy(),
                              c["lens"].cpu().numpy(), scale, c["causal"], 0.0, None, c["window"], None)


def rising(c, base, dt, sign=1.0):
    """Scores sign 2048 base + (a step of 1 for each 128 keys, 0 or 2 below that at random)."""
    g = torch.Generator().manual_seed(5)
    c["q"].zero_()
    c["q"][..., 0], c["q"][..., 1] = 2048.0 * sign, 1.0
    for b in range(c["table"].shape[0]):
        for j in range(int(c["lens"][b])):
            page, P = int(c["table"][b, j // c["kc"].shape[2]]), c["kc"].shape[2]
            c["kc"][page, :, j % P] = 0.0
            c["kc"][page, :, j % P, 0], c["kc"][page, :, j % P, 1] = base, j // 128 - 2.0 * int(torch.randint(0, 2, (1,), generator=g))


@pytest.mark.parametrize("base,sign", [(1917, 1), (1968, 1), (2002, 1), (2019, 1), (1917, -1), (2002, -1)])
@pytest.mark.parametrize("slopes", [False, True])
def test_a_maximum_that_rises_slowly(kv, base, sign, slopes):
    # a step is 7.9 powers of two: the maximum in use lags behind by nearly the 8 that it may
    scale = 7.9 * LN2
    c = prompt.case(91, [300, 40], [300, 500], 8, 2, 32, HF)
    rising(c, base, HF, sign)
    zero = torch.zeros(8, device="cuda") if slopes else None  # (biased by nothing, through the biased kernel)
    out, lse = prompt.call(kv, c, scale=scale, slopes=zero)
    check(c, out, lse, scale, prompt_want(c, scale), rounded=slopes)
    assert out.abs().max() <= c["vc"][torch.isfinite(c["vc"])].abs().max()


@pytest.mark.parametrize("dt", [BF, HF])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("new,ctx", [([200, 5], [40, 600]), ([3], [9000])])
def test_scores_of_the_largest_products(kv, dt, sign, new, ctx):
    # equal channels: 128 q k; neighbouring scores differ by 2^23 at least, so each row has its largest keys only
    c = prompt.case(92, new, ctx, 4, 1, 16, dt)
    c["q"].fill_(sign * 32768.0)
    steps = 1024 if dt == HF else 128
    for b in range(len(new)):
        for j in range(new[b] + ctx[b]):
            c["kc"][int(c["table"][b, j // 16]), 0, j % 16] = 32768.0 * (1 + (j * 37 % steps) / steps)
    out, lse = prompt.call(kv, c)
    check(c, out, lse, SCALE, prompt_want(c, SCALE))


@pytest.mark.parametrize("dt", [BF, HF])
def test_prefix(kv, dt):
    c = prefix.case(93, [700, 130], [6, 4], [40] * 12, 8, 2, 16, dt)
    c["q"].fill_(32768.0)
    for table, lens in ((c["prefix_table"], c["prefix_lens"]), (c["table"], c["lens"])):
        for b in range(len(lens)):
            for j in range(int(lens[b])):
                c["kc"][int(table[b, j // 16]), :, j % 16] = 32768.0 * (1 + ((j + 5 * b) * 37 % 128) / 128)
    out, lse = prefix.call(kv, c)
    check(c, out, lse, SCALE, o.prefix_attention(
        np64(c["q"]), np64(c["kc"]), np64(c["vc"]), c["prefix_table"].cpu().numpy(), c["prefix_lens"].cpu().numpy(),
        c["cu"].cpu().numpy(), c["table"].cpu().numpy(), c["lens"].cpu().numpy(), SCALE))
