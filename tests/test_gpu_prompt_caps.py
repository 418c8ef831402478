"""Capped scores at every size of the cap, on the GPU against the fp64 oracle.

Tolerances are test_gpu_prompt.py's (test_gpu_prefix.py's for the prefix), but for the cap's own: its polynomial is off by
2^-22 of the score with its roundings, the formula of larger scores by 2^-22.2 of the cap where the score is 0.245 of it
at least: 2^-20 of min(cap, reach), whatever the cap."""
import numpy as np
import pytest
import torch

from oracle import serving as o
from tests import test_gpu_prefix as prefix
from tests import test_gpu_prompt as prompt
from tests.test_gpu_prompt import BF, F32, HF, SCALE, bounds, np64

pytestmark = pytest.mark.gpu
CAPS = [2.0 ** -126, 0.02, 5.0, 50.0, 1e3, 1e4, 1e5, 1e6, 1e8, 1e20, 1e30, 1.2e38, 3e38, float(np.finfo(np.float32).max)]


@pytest.fixture(autouse=True)
def _no_device_error(kv):
    kv.kvarn_device_error()
    yield
    assert kv.kvarn_device_error() == 0


def prompt_oracle(c, scale, softcap, slopes=None, kc=None):
    return o.prompt_attention(np64(c["q"]), np64(c["kc"] if kc is None else kc), np64(c["vc"]), c["table"].cpu().numpy(), c["cu"].cpu().numpy(),
                              c["lens"].cpu().numpy(), scale, c["causal"], softcap, None if slopes is None else np64(slopes), c["window"],
                              None if c["starts"] is None else c["starts"].cpu().numpy())


def compare(got, want, tol):
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], bad.mean(), got[bad][:4], want[bad][:4], tol[bad][:4])


def check_prompt(c, out, lse, scale, softcap, slopes=None, reach=None):
    want, want_lse, mass, reach0, count = prompt_oracle(c, scale, softcap, slopes)
    reach = reach0 if reach is None else reach
    bias = 0.0 if slopes is None else np64(slopes)[None] * float(c["lens"].max())
    tol, lse_tol = bounds(want, want_lse, mass, reach, count, c["dt"], 2 * np.minimum(softcap, reach), bias)
    rows, some = ~np.isnan(want_lse), np.isfinite(want_lse)
    compare(np64(out)[rows], want[rows], tol[rows])
    compare(np64(lse)[some], want_lse[some], lse_tol[some])
    assert np.array_equal(np.isneginf(np64(lse)), np.isneginf(want_lse))


@pytest.mark.parametrize("softcap", CAPS)
@pytest.mark.parametrize("dt", [BF, HF])
def test_prompt_at_every_size_of_the_cap(kv, dt, softcap):
    c = prompt.case(71, [300, 7, 1, 40], [0, 200, 600, 128], 8, 2, 16, dt)
    out, lse = prompt.call(kv, c, softcap=softcap)
    check_prompt(c, out, lse, SCALE, softcap)


@pytest.mark.parametrize("softcap,scale", [(5.0, 0.5), (5.0, -0.5), (0.5, SCALE), (20.0, 1.0), (1e3, 40.0), (1e30, 0.5), (5.0, 1e-30)])
@pytest.mark.parametrize("kw", [dict(), dict(window=100, starts=[17, 0, 300]), dict(causal=False), dict(slopes=True)])
def test_prompt_with_scores_on_both_sides_of_half_the_cap(kv, kw, softcap, scale):
    kw = dict(kw)
    slopes = 2.0 ** -torch.arange(1, 9, device="cuda", dtype=F32) if kw.pop("slopes", False) else None
    c = prompt.case(72, [200, 130, 3], [0, 70, 900], 8, 2, 48, BF, **kw)
    out, lse = prompt.call(kv, c, scale=scale, softcap=softcap, slopes=slopes)
    check_prompt(c, out, lse, scale, softcap, slopes)


@pytest.mark.parametrize("dt,key,softcap", [(BF, -3e6, 1e5), (BF, -3e6, 2e6), (HF, -6e4, 5e3), (BF, -3e30, 1e30)])
def test_prompt_beside_a_score_far_below_the_others(kv, dt, key, softcap):
    # one key scores about minus the cap (and has no weight); the others' scores are ordinary ones beside it
    c = prompt.case(73, [150, 20], [40, 300], 4, 1, 16, dt)
    c["q"][..., 0] = 1.0
    clean = c["kc"].clone()
    for b, j in ((0, 33), (1, 2), (1, 290)):
        page = int(c["table"][b, j // 16])
        c["kc"][page, 0, j % 16, 0] = key
        clean[page, 0, j % 16] = 0.0
    reach = prompt_oracle(c, SCALE, 0.0, kc=clean)[3]  # of the keys with weight
    check_prompt(c, *prompt.call(kv, c, softcap=softcap), SCALE, softcap, reach=reach)


@pytest.mark.parametrize("softcap", CAPS)
@pytest.mark.parametrize("dt", [BF, HF])
def test_prefix_at_every_size_of_the_cap(kv, dt, softcap):
    c = prefix.case(74, [500, 90, 0], [6, 4, 1], [100, 1, 5, 60, 2, 3, 128, 16, 9, 10, 33, 2], 8, 2, 32, dt)
    out, lse = prefix.call(kv, c, softcap=softcap)
    want, want_lse, mass, reach, count = o.prefix_attention(
        np64(c["q"]), np64(c["kc"]), np64(c["vc"]), c["prefix_table"].cpu().numpy(), c["prefix_lens"].cpu().numpy(),
        c["cu"].cpu().numpy(), c["table"].cpu().numpy(), c["lens"].cpu().numpy(), SCALE, softcap)
    tol, lse_tol = bounds(want, want_lse, mass, reach, count, dt, 2 * np.minimum(softcap, reach))
    tol += (2.0 ** -20 + 2.0 ** -22 * np.abs(want_lse))[..., None] * mass
    compare(np64(out), want, tol)
    compare(np64(lse), want_lse, lse_tol + 2.0 ** -20)
