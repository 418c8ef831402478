"""Launch shapes of the serving step's calls that small cases do not reach, against the oracle: several slices
and passes of a token, the wide tables, blocks of 9 to 16 query heads with every modifier, and random cases
from fixed seeds.  Tolerances are those derived in test_gpu_serving.py."""
import math
import random

import numpy as np
import pytest
import torch

from oracle import serving as o
from tests.test_gpu_serving import (BF, F32, HF, _no_device_error, attn_call, attn_case, attn_check, i32, np64, rope_call,  # noqa: F401
                                    rope_case, rope_check, run_tables, same_tables, table_state)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [3, 256, 400, 1000, 1300])
@pytest.mark.parametrize("kw", [dict(hq=32, hkv=8, fused=True, P=64), dict(hq=32, hkv=8, xt=F32, rot=64, interleaved=True),
                                dict(hq=1, hkv=1), dict(hq=64, hkv=8, xt=HF, ct=HF, norm="k")])
def test_rope_slices_and_passes(kv, T, kw):
    # few tokens: up to four CTAs' slices of a token's rows, with a last pass past the rows; 1300: a warp a token
    c = rope_case(80 + T, T, **kw)
    before = [c[k].clone() for k in ("qo", "kc", "vc")]
    rope_check(c, rope_call(kv, c), *before)


@pytest.mark.parametrize("max_new,rows", [(270, 33000), (1000, 132000)])
@pytest.mark.parametrize("finish", [0.0, 0.2])
@pytest.mark.parametrize("in_place", [False, True])
def test_tables_of_many_rows(kv, max_new, rows, finish, in_place):
    # more than 32768 rows: CTAs of 1024 threads; more than 131072: warps take a second run of 256 rows
    s = table_state(81, 1100 if finish == 0.0 else 1400, 16, 500, max_new, finish=finish, hkv=2, rollback=in_place)
    assert s["rows"] > rows
    assert same_tables(run_tables(kv, s, in_place), s)["status"] == 0


MODIFIERS = [dict(), dict(softcap=15.0, slopes=True), dict(window=23, starts=True, slopes=True), dict(window=70, softcap=4.0)]
TYPES = [(BF, BF), (HF, HF), (BF, F32)]


def _modified(kv, seed, lens, group, hkv, dt, out_dtype, wide, window=0, softcap=0.0, slopes=False, starts=False, P=16):
    hq = group * hkv
    first = [(7 * i) % max(n, 1) for i, n in enumerate(lens)] if starts else None
    c = attn_case(seed, lens, hq, hkv, P=P, dt=dt, starts=first, window=window, wide=wide)
    m = dict(softcap=softcap, slopes=2.0 ** (-8 * torch.arange(1, hq + 1, device="cuda") / hq) if slopes else None)
    attn_check(c, *attn_call(kv, c, out_dtype=out_dtype, **m), **m)


@pytest.mark.parametrize("group,hkv", [(9, 1), (11, 2), (12, 2), (13, 1), (15, 2), (16, 2), (24, 1)])
@pytest.mark.parametrize("types", range(3))
@pytest.mark.parametrize("wide", [False, True])
def test_attention_of_nine_to_sixteen_heads(kv, group, hkv, types, wide):
    # B 40: more than the 32 sequences that a warp scans by itself
    lens = [(37 * i) % 190 for i in range(40)]
    for i, m in enumerate(MODIFIERS):
        _modified(kv, 82 + i, lens, group, hkv, *TYPES[types], wide, **m)


@pytest.mark.parametrize("group,hkv", [(4, 2), (12, 1), (16, 1), (24, 1)])
@pytest.mark.parametrize("wide", [False, True])
def test_attention_of_several_scan_rounds(kv, group, hkv, wide):
    # more sequences than a CTA has threads (384 up to 8 heads, 256 past them)
    lens = [(13 * i) % 40 for i in range(450)]
    for i, m in enumerate(MODIFIERS[:3]):
        _modified(kv, 86 + i, lens, group, hkv, *TYPES[i], wide, **m)


def test_attention_of_wide_groups_over_long_contexts(kv):
    # units cut over several CTAs, two blocks of heads
    for group in (9, 16, 40):
        _modified(kv, 89, [9000, 17, 3001], group, 1, BF, F32, True, P=64)
        _modified(kv, 90, [9000, 17, 3001], group, 1, HF, HF, True, P=64, window=5000, softcap=10.0, slopes=True)


def test_rope_writes_everything_else_beside_a_slot_out_of_the_cache(kv):
    # caches and outputs are fresh: nothing of an earlier call can stand in for this one's rows
    for T in (6, 1300):
        c = rope_case(91, T, 4, 2)
        c["slots"][5] = c["kc"].shape[0] * c["P"]
        before = [c[k].clone() for k in ("qo", "kc", "vc")]
        rope_check(c, rope_call(kv, c), *before)
        assert kv.kvarn_device_error() == 32
        assert not torch.equal(c["kc"], before[1])


def test_log_sums_of_a_pseudo_decoded_block(kv):
    """The log sums that the pseudo-decode does not ask for, on its own queries and pages."""
    from bit_kv_cache_kvarn_gb300 import pseudo_decode as pd

    w, x = pd.make_weights(42, 1, 256, 4, 2), pd.make_input(42, 3 * 128, 256)
    cap = {(j, 0): None for j in range(3)}
    pd.run(kv, None, w, x, 4, 2, quantised=False, paged=True, capture=cap)
    for (j, _), c in cap.items():
        lens = i32([128 * j + t + 1 for t in range(128)])
        case = dict(q=c["q"], kc=c["k_pages"], vc=c["v_pages"], table=c["table"].expand(128, -1).contiguous(), lens=lens, starts=None, window=0)
        out, lse = attn_call(kv, case)
        assert torch.equal(out, c["attn"])
        attn_check(case, out, lse)


# ---- random cases ------------------------------------------------------------------------------------------
def _log_int(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


@pytest.mark.parametrize("seed", range(12))
def test_random_attention(kv, seed):
    rng = random.Random(seed)
    for n in range(6):
        group, hkv = rng.choice([(1, 1), (4, 2), (4, 1), (8, 1), (1, 5), (7, 1), (9, 1), (16, 1), (17, 1), (3, 2), (33, 1)])
        B = _log_int(rng, 1, 120)
        most = _log_int(rng, 1, max(1, 12000 // B))
        lens = [rng.choice([0, rng.randint(0, most), rng.randint(0, most), most]) for _ in range(B)]
        if rng.random() < 0.3:  # mostly empty
            lens = [x if rng.random() < 0.1 else 0 for x in lens]
        dt = rng.choice([BF, HF])
        _modified(kv, 1000 * seed + n, lens, group, hkv, dt, rng.choice([F32, dt]), rng.random() < 0.5,
                  window=rng.choice([0, 0, 1, 17, _log_int(rng, 1, 3000)]), softcap=rng.choice([0.0, 0.0, 20.0]),
                  slopes=rng.random() < 0.3, starts=rng.random() < 0.3, P=rng.choice([16, 32, 48, 128]))


@pytest.mark.parametrize("seed", range(8))
def test_random_tables(kv, seed):
    rng = random.Random(seed)
    for n in range(6):
        B = _log_int(rng, 1, 3000)
        s = table_state(1000 * seed + n, B, rng.choice([1, 3, 16, 48, 128]), _log_int(rng, 1, max(2, 200000 // B)),
                        _log_int(rng, 1, max(1, 60000 // B)), finish=rng.choice([0.0, 0.1, 0.9]), hkv=rng.choice([0, 1, 5]),
                        slack=rng.choice([0, 3]), rollback=rng.random() < 0.3)
        if rng.random() < 0.2:
            s["n_free"] = max(0, s["n_free"] - 3)
        if same_tables(run_tables(kv, s, rng.random() < 0.5), s)["status"]:
            assert kv.kvarn_device_error() == 16


@pytest.mark.parametrize("seed", range(8))
def test_random_rope(kv, seed):
    rng = random.Random(seed)
    for n in range(4):
        hq, hkv = rng.choice([(32, 8), (5, 5), (8, 1), (12, 2), (1, 1), (28, 4)])
        xt, ct = rng.choice([(BF, BF), (HF, HF), (F32, BF), (F32, HF)])
        T = _log_int(rng, 1, 3000 * 8 // (hq + 2 * hkv))
        pos = torch.tensor([rng.choice([rng.randint(0, 40000), rng.randint(0, 2 ** 31 - 1), -1]) for _ in range(T)], dtype=torch.int32)
        c = rope_case(1000 * seed + n, T, hq, hkv, xt=xt, ct=ct, P=rng.choice([1, 7, 16, 128]), rot=rng.choice([0, 128, 64, 16, 112]),
                      interleaved=rng.random() < 0.5, norm=rng.choice(["", "q", "k", "qk"]), layout=rng.choice(["hnd", "nhd", "both"]),
                      fused=rng.random() < 0.5, positions=pos.cuda())
        before = [c[k].clone() for k in ("qo", "kc", "vc")]
        rope_check(c, rope_call(kv, c), *before)
