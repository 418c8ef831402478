"""The serving step's calls on the GPU against the fp64 oracle.

Tolerances, from the arithmetic:
  kvarn_rope_qkv       one rounding to the output type (half a step: 2^-8 bf16, 2^-11 fp16) of a value
                       computed in fp32 from a pair (a, b): 32 fp32 half steps of |a| + |b| cover the
                       mean of 128 squares (7 levels + 16 terms in a lane), root, quotient, two products
                       with weight and turn, sin and cos (2 ulp of the functions, 1 of the argument times
                       pi); the frequency's own 2^-53, once more for its product with 1 / 2 pi, times the
                       angle adds angle * 2^-51.
  kvarn_paged_attention  a score is two chains of four 16-term products, each addition off by at most 2^-23
                       (truncating) of its partial sum: 2^-19 of reach = scale max_j sum |q k| covers it
                       together with the scaling; capping keeps it (tanh has slope <= 1, and its own
                       2^-21 cap), the bias adds 2^-23 of itself.  A probability is then off by twice
                       the score's error (its own and the maximum's, numerator and sum) plus 2^-20 (exp2)
                       plus what its 16-bit pieces leave: 2^-24 of it for three bf16 pieces, 2^-22 for two
                       fp16 ones (both with fp32 results), 2^-16 for two bf16 ones (bf16 results); so out is
                       off by at most that times sum p |v|, plus the output's rounding, and lse by the
                       score's error plus 2^-22 of itself.
"""
import math
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

from oracle import kvarn_oracle as ko
from oracle import serving as o
from tests._parity import rel_l2
from tests.test_gpu_graph import _capture

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
HALF_STEP = {BF: 2.0 ** -8, HF: 2.0 ** -11, F32: 2.0 ** -24}


@pytest.fixture(autouse=True)
def _no_device_error(kv):
    kv.kvarn_device_error()
    yield
    assert kv.kvarn_device_error() == 0


def np64(t):
    return t.detach().double().cpu().numpy()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ---- tables ------------------------------------------------------------------------------------------
def table_state(seed, B, P, max_len, max_new, finish=0.1, hkv=0, slack=3, extra_rows=5, width=None, rollback=False):
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, max_len + 1, B).astype(np.int32)
    new = np.where(rng.random(B) < 0.7, rng.integers(0, 2, B), rng.integers(0, max_new + 1, B)).astype(np.int32)
    new[rng.random(B) < finish] = -1
    counts = -(-lens // P)
    if rollback:  # some hold a page or two more than their length needs
        counts = counts + rng.integers(0, 3, B)
    counts = counts.astype(np.int32)
    need = np.where(new < 0, 0, np.maximum(0, -(-(lens + new) // P) - counts))
    width = width or int(max((-(-(lens + np.maximum(new, 0)) // P)).max(), counts.max(), 1))
    pool = rng.permutation(int(counts.sum() + need.sum()) + slack).astype(np.int32)
    table = np.full((B, width), -1, np.int32)
    at = 0
    for b in range(B):
        table[b, :counts[b]] = pool[at:at + counts[b]]
        at += counts[b]
    free = np.full(len(pool), -7, np.int32)
    free[:len(pool) - at] = pool[at:]
    blocks = None
    if hkv:
        blocks = np.where(table[:, None] < 0, -1, table[:, None] * hkv + np.arange(hkv, dtype=np.int32)[None, :, None]).astype(np.int32)
    rows = int(np.maximum(new, 0).sum()) + extra_rows
    return dict(lens=lens, new=new, counts=counts, table=table, free=free, n_free=len(pool) - at, P=P, rows=rows, blocks=blocks)


def run_tables(kv, s, in_place=False, call=None):
    d = {k: i32(s[k].copy()) for k in ("lens", "new", "counts", "table", "free")}
    n_free = i32([s["n_free"]])
    B, rows = len(s["lens"]), s["rows"]
    out = dict(kv_lens=d["lens"] if in_place else torch.full_like(d["lens"], -99),
               page_counts=d["counts"] if in_place else torch.full_like(d["lens"], -99),
               free_count=n_free if in_place else i32([-99]), cu_tokens=torch.full((B + 1,), -99, dtype=torch.int32, device="cuda"),
               positions=torch.full((rows,), -99, dtype=torch.int32, device="cuda"),
               slot_map=torch.full((rows,), -99, dtype=torch.int32, device="cuda"), status=i32([-99]),
               page_table=d["table"], free_pages=d["free"], block_table=None if s["blocks"] is None else i32(s["blocks"].copy()))

    def step():
        kv.kvarn_step_tables(d["lens"], d["new"], d["counts"], d["table"], d["free"], n_free, s["P"], out["kv_lens"],
                             out["page_counts"], out["free_count"], out["cu_tokens"], out["positions"], out["slot_map"],
                             out["status"], block_table=out["block_table"])

    (call or (lambda f: f()))(step)
    return out


def same_tables(got, s):
    want = o.step_tables(s["lens"], s["new"], s["counts"], s["table"], s["free"], s["n_free"], s["P"], s["rows"], s["blocks"])
    for k, w in want.items():
        if w is None:
            continue
        g = got[k].cpu().numpy()
        assert np.array_equal(g.reshape(-1), np.asarray(w).reshape(-1)), k
    return want


@pytest.mark.parametrize("B,P,max_len,max_new,hkv,in_place", [
    (1, 16, 0, 0, 0, False), (1, 1, 5, 3, 1, True), (1, 128, 40000, 6000, 8, False), (3, 48, 100, 70, 2, True),
    (64, 128, 32768, 1, 8, False), (257, 7, 300, 50, 3, True), (1024, 16, 900, 9, 0, False), (1025, 16, 200, 4, 1, True),
    (3000, 32, 500, 40, 0, False), (16384, 16, 60, 3, 0, True)])
def test_tables_match_the_oracle(kv, B, P, max_len, max_new, hkv, in_place):
    for seed in range(2):
        s = table_state(seed, B, P, max_len, max_new, hkv=hkv, rollback=seed == 1)
        assert same_tables(run_tables(kv, s, in_place), s)["status"] == 0


def test_tables_all_finished_and_nothing_new(kv):
    s = table_state(5, 40, 16, 300, 1, slack=0)
    s["new"][:] = -1
    s["rows"] = 0  # empty positions and slots
    assert same_tables(run_tables(kv, s), s)["free_count"] == int(s["counts"].sum()) + s["n_free"]
    s["new"][:] = 0
    same_tables(run_tables(kv, s, True), s)


def test_tables_pages_given_back_are_taken_again_in_the_same_step(kv):
    # no free page at all: the new sequences live on what the finished ones give back
    s = table_state(6, 30, 16, 200, 0, finish=0.0, slack=0)
    s["n_free"], s["free"] = 0, np.full(3, -5, np.int32)
    s["new"] = np.where(np.arange(30) % 3 == 0, -1, 10).astype(np.int32)
    s["rows"] = 200
    s["table"] = np.concatenate([s["table"], np.full((30, 2), -1, np.int32)], axis=1)
    # a stack of three entries is too short for what is left over: refused, and reported
    assert same_tables(run_tables(kv, s), s)["status"] == o.FREE_FULL
    assert kv.kvarn_device_error() == 16
    s["free"] = np.full(500, -5, np.int32)
    assert same_tables(run_tables(kv, s, True), s)["status"] == 0


@pytest.mark.parametrize("B", [5, 4000])
def test_tables_failures_change_nothing(kv, B):
    for change, bit in ((lambda s: s.update(n_free=0), o.NO_PAGES), (lambda s: s.update(rows=max(0, s["rows"] - 6)), o.ROWS),
                        (lambda s: s["lens"].__setitem__(1, -3), o.INVALID), (lambda s: s["counts"].__setitem__(1, -1), o.INVALID),
                        (lambda s: s["counts"].__setitem__(0, 10 ** 6), o.INVALID), (lambda s: s.update(n_free=10 ** 7), o.INVALID),
                        (lambda s: s.update(n_free=-1), o.INVALID),
                        (lambda s: (s["lens"].__setitem__(2, 2 ** 31 - 2), s["new"].__setitem__(2, 5)), o.INVALID),
                        (lambda s: s["new"].__setitem__(0, 10 ** 5), o.ROW_FULL)):
        s = table_state(7, B, 16, 50, 40, finish=0.0, slack=0, hkv=2)
        s["new"][0] = max(s["new"][0], 17)  # at least one page is taken and one row filled
        s["rows"] = int(s["new"].sum()) + 5
        s["table"] = np.concatenate([s["table"], np.full((B, 2), -1, np.int32)], axis=1)
        s["blocks"] = np.full((B, 2, s["table"].shape[1]), -1, np.int32)
        s["free"] = np.concatenate([s["free"], np.full(8, -7, np.int32)])
        change(s)
        want = same_tables(run_tables(kv, s, in_place=True), s)
        assert want["status"] & bit, (bit, want["status"])
        assert kv.kvarn_device_error() == 16


def test_tables_overfull_stack_is_refused(kv):
    s = table_state(8, 10, 16, 100, 1, finish=0.0, slack=0)
    s["new"][:] = -1
    s["n_free"], s["free"] = 2, np.array([500, 501, -7], np.int32)
    assert same_tables(run_tables(kv, s), s)["status"] == o.FREE_FULL
    assert kv.kvarn_device_error() == 16


def test_tables_replay(kv):
    # in place under capture: each replay is the next step
    s = table_state(9, 20, 16, 100, 1, finish=0.0, slack=60)
    s["new"][:] = 1
    s["rows"] = 20
    s["table"] = np.concatenate([s["table"], np.full((20, 4), -1, np.int32)], axis=1)
    keep = {}

    def call(step):
        keep["g"] = _capture(step)  # one eager call outside the capture
        for _ in range(30):
            keep["g"].replay()
        torch.cuda.synchronize()

    got = run_tables(kv, s, in_place=True, call=call)
    for _ in range(31):
        r = o.step_tables(s["lens"], s["new"], s["counts"], s["table"], s["free"], s["n_free"], 16, 20)
        assert r["status"] == 0
        s.update(lens=r["kv_lens"], counts=r["page_counts"], table=r["page_table"], free=r["free_pages"], n_free=r["free_count"])
    assert np.array_equal(got["kv_lens"].cpu().numpy(), s["lens"]) and np.array_equal(got["page_table"].cpu().numpy(), s["table"])
    assert np.array_equal(got["slot_map"].cpu().numpy(), r["slot_map"])


def test_tables_of_a_long_chunk_replay(kv):
    # a cluster of CTAs under capture, not in place: the same step again and again
    s = table_state(10, 300, 16, 500, 90, hkv=2)
    keep = {}

    def call(step):
        keep["g"] = _capture(step)
        keep["g"].replay()
        torch.cuda.synchronize()

    assert s["rows"] > 2048
    same_tables(run_tables(kv, s, call=call), s)


# ---- norm, rotation, cache write -------------------------------------------------------------------------
def rope_case(seed, T, hq, hkv, xt=BF, ct=BF, P=16, rot=128, interleaved=False, norm="qk", layout="hnd", fused=False,
              positions=None, spare=2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    chan = torch.exp(0.7 * torch.randn(128, generator=g, device="cuda"))
    if fused:
        rows = (torch.randn(T, hq + 2 * hkv + 1, 128, generator=g, device="cuda") * chan).to(xt)
        q, k, v = rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:hq + 2 * hkv]
    else:
        q, k, v = ((torch.randn(T, h, 128, generator=g, device="cuda") * chan).to(xt) for h in (hq, hkv, hkv))
    n_pages = -(-T // P) + spare
    if layout == "hnd":
        kc, vc = (torch.randn(n_pages, hkv, P, 128, generator=g, device="cuda").to(ct) for _ in range(2))
    elif layout == "nhd":
        kc, vc = (torch.randn(n_pages, P, hkv, 128, generator=g, device="cuda").to(ct).transpose(1, 2) for _ in range(2))
    else:  # K and V pages in one array, rows padded to 136
        both = torch.randn(n_pages, 2, hkv, P, 136, generator=g, device="cuda").to(ct)
        kc, vc = both[:, 0, :, :, :128], both[:, 1, :, :, :128]
    if positions is None:
        positions = torch.randint(0, 100000, (T,), generator=g, device="cuda").to(torch.int32)
    slots = torch.randperm(n_pages * P, generator=g, device="cuda")[:T].to(torch.int32)
    w = [1 + 0.3 * torch.randn(128, generator=g, device="cuda") if n in norm else None for n in "qk"]
    return dict(q=q, k=k, v=v, kc=kc, vc=vc, positions=positions, slots=slots, qw=w[0], kw=w[1], rot=rot,
                interleaved=interleaved, P=P, ct=ct, eps=1e-5, scale=1.0,
                qo=torch.full((T, hq, 128), 7.0, dtype=ct, device="cuda"))


def rope_call(kv, c, **kw):
    freqs, _ = kv.kvarn_rope_frequencies(c["rot"], 1e6) if c["rot"] else (None, 1.0)
    kv.kvarn_rope_qkv(c["q"], c["k"], c["v"], c["positions"], None if freqs is None else freqs.cuda(), c["qo"], c["kc"],
                      c["vc"], slot_map=c["slots"], q_weight=c["qw"], k_weight=c["kw"], eps=c["eps"],
                      rope_scale=c["scale"], interleaved=c["interleaved"], **kw)
    return freqs


def rope_check(c, freqs, before_q, before_k, before_v, q=None, k=None):
    f = np.zeros(0) if freqs is None else freqs.numpy()
    pos = c["positions"].cpu().numpy()
    live = pos >= 0
    safe = np.where(live, pos, 0)
    step = HALF_STEP[c["ct"]]
    tiny = float(torch.finfo(c["ct"]).smallest_normal)

    def want(x, w):
        w = None if w is None else np64(w)
        y = o.norm_rotate(np64(x), safe, f, w, c["eps"], c["scale"], c["interleaved"])
        plain = np.abs(o.norm_rotate(np64(x), safe, f[:0], w, c["eps"]))
        pair = plain.copy()
        if len(f):
            i = np.arange(len(f))
            a, b = (2 * i, 2 * i + 1) if c["interleaved"] else (i, i + len(f))
            both = plain[..., a] + plain[..., b]
            pair[..., a] = pair[..., b] = both * abs(c["scale"])
        angle = safe.max(initial=0) * (f.max() if len(f) else 0.0)
        return y, step * np.abs(y) + pair * (32 * 2.0 ** -24 + angle * 2.0 ** -51) + tiny * 2.0 ** -8

    y, tol = want(c["q"] if q is None else q, c["qw"])
    got = np64(c["qo"])
    assert np.all(np.abs(got - y)[live] <= tol[live])
    assert np.array_equal(got[~live], np64(before_q)[~live])
    slots = (torch.arange(len(pos)) if c["slots"] is None else c["slots"].cpu()).numpy()
    ek, ev = np64(before_k), np64(before_v)
    tk = np.zeros_like(ek)
    y, tol = want(c["k"] if k is None else k, c["kw"])
    vr = np64(c["v"].to(c["ct"]))
    n = ek.shape[0] * c["P"]
    for t in range(len(pos)):
        if live[t] and 0 <= slots[t] < n:
            p, off = divmod(int(slots[t]), c["P"])
            ek[p, :, off], tk[p, :, off], ev[p, :, off] = y[t], tol[t], vr[t]
    assert np.all(np.abs(np64(c["kc"]) - ek) <= tk)  # untouched slots: exactly as they were
    assert np.array_equal(np64(c["vc"]), ev)


@pytest.mark.parametrize("T", [1, 3, 130, 1500])
@pytest.mark.parametrize("kw", [
    dict(hq=4, hkv=2), dict(hq=5, hkv=1, fused=True, norm="q"), dict(hq=3, hkv=3, xt=HF, ct=HF, rot=64, interleaved=True, layout="nhd"),
    dict(hq=8, hkv=1, xt=F32, norm="", rot=32, P=48, layout="both"), dict(hq=2, hkv=1, xt=F32, ct=HF, rot=96, fused=True, norm="k", P=1),
    dict(hq=2, hkv=2, rot=0), dict(hq=1, hkv=1, rot=128, interleaved=True, norm="", P=128), dict(hq=7, hkv=5, rot=16, layout="both")])
def test_rope_matches_the_oracle(kv, T, kw):
    c = rope_case(11 + T, T, **kw)
    c["scale"] = 1.25
    before = [c[k].clone() for k in ("qo", "kc", "vc")]
    rope_check(c, rope_call(kv, c), *before)


def test_rope_long_chunk_matches_the_oracle(kv):
    # more tokens than run at once: warps go on from token to token
    c = rope_case(19, 11003, 2, 1, rot=16, P=64, norm="qk", fused=True)
    before = [c[k].clone() for k in ("qo", "kc", "vc")]
    rope_check(c, rope_call(kv, c), *before)


@pytest.mark.parametrize("T", [6, 1200])
def test_rope_far_positions_padding_and_slots(kv, T):
    pos = torch.randint(2 ** 30, 2 ** 31 - 1, (T,)).to(torch.int32)
    pos[0], pos[1], pos[2] = 2 ** 31 - 1, 0, -1
    pos[4] = -(2 ** 31)
    c = rope_case(3, T, 4, 2, xt=F32, positions=pos.cuda())
    c["slots"][3] = -1  # key and value dropped, the query written
    c["q"][2] = float("nan")  # rows of padding are not read
    c["q"][4], c["k"][4] = float("inf"), float("nan")
    before = [c[k].clone() for k in ("qo", "kc", "vc")]
    freqs = rope_call(kv, c)
    c["q"][2] = c["q"][4] = c["k"][4] = 0
    rope_check(c, freqs, *before)
    # slots outside the cache are dropped and reported
    c["slots"][5] = c["kc"].shape[0] * c["P"]
    before = [c[k].clone() for k in ("qo", "kc", "vc")]
    c["kc"].copy_(before[1]), c["vc"].copy_(before[2])
    rope_call(kv, c)
    rope_check(c, freqs, *before)
    assert kv.kvarn_device_error() == 32


def test_rope_in_place_on_strided_queries_and_partial_sides(kv):
    c = rope_case(21, 70, 6, 2, fused=True, rot=64)
    q = c["q"].clone()
    c["qo"] = c["q"]  # rotated where the projection left it
    kept = [c["k"].clone(), c["v"].clone()]
    before = [c[k].clone() for k in ("qo", "kc", "vc")]
    rope_check(c, rope_call(kv, c), *before, q=q)
    assert torch.equal(c["k"], kept[0]) and torch.equal(c["v"], kept[1])
    # queries alone, keys alone
    freqs = kv.kvarn_rope_frequencies(64, 1e6)[0].cuda()
    out = torch.empty_like(q)
    kv.kvarn_rope_qkv(q, None, None, c["positions"], freqs, out, None, None, q_weight=c["qw"], eps=c["eps"])
    assert torch.equal(out, c["qo"])
    kc, vc = before[1].clone(), before[2].clone()
    kv.kvarn_rope_qkv(None, c["k"], c["v"], c["positions"], freqs, None, kc, vc, slot_map=c["slots"], k_weight=c["kw"], eps=c["eps"])
    assert torch.equal(kc, c["kc"]) and torch.equal(vc, c["vc"])


def test_rope_special_values_and_zero_rows(kv):
    c = rope_case(22, 4, 2, 2, norm="qk")
    c["q"][0] = 0  # mean square 0: eps keeps it at 0
    c["q"][1, 0, 5] = float("nan")
    c["v"][2, 1, 7], c["v"][2, 1, 8] = float("inf"), float("nan")
    rope_call(kv, c)
    assert not c["qo"][0].any()
    assert torch.isnan(c["qo"][1, 0]).all() and torch.isfinite(c["qo"][1, 1]).all()
    p, off = divmod(int(c["slots"][2]), c["P"])
    assert torch.isinf(c["vc"][p, 1, off, 7]) and torch.isnan(c["vc"][p, 1, off, 8])


def test_rope_python_refusals(kv):
    c = rope_case(23, 4, 2, 2)
    for change, match in ((dict(k=c["k"][:, :1]), "k and v|shape"), (dict(q=c["q"].half()), "k must be"), (dict(q=c["q"].cpu()), "current CUDA"),
                          (dict(positions=c["positions"].long()), "positions"), (dict(slots=c["slots"][:2]), "slot_map"),
                          (dict(vc=c["vc"][:1]), "v_cache"), (dict(kc=None), "goes with"), (dict(qw=torch.ones(128, dtype=BF, device="cuda")), "q_weight")):
        with pytest.raises((ValueError, kv.KvarnError), match=match):
            rope_call(kv, {**c, **change})


# ---- paged attention ---------------------------------------------------------------------------------------
def attn_case(seed, lens, hq, hkv, P=16, dt=BF, layout="hnd", starts=None, window=0, garbage=float("nan"), spread=1.0, spare=3,
              wide=False):
    """Every slot outside the visible tokens holds `garbage`, every unused page table entry an id far outside.
    wide: a page table for 100 000 tokens, so that the split over the stream serves short sequences too."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, width = len(lens), max(1, -(-max(lens) // P), -(-100000 // P) if wide else 0) + 1
    used = [-(-n // P) for n in lens]
    n_pages = sum(used) + spare
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
        pages = perm[at:at + used[b]]
        at += used[b]
        lo = max(0 if starts is None else starts[b], n - window if window else 0, 0)
        for i in range(lo // P, used[b]):
            table[b, i] = pages[i]
            a, e = max(lo - i * P, 0), min(n - i * P, P)
            if e > a:
                page = int(pages[i])
                kc[page, :, a:e] = (spread * torch.randn(hkv, e - a, 128, generator=g, device="cuda")).to(dt)
                vc[page, :, a:e] = torch.randn(hkv, e - a, 128, generator=g, device="cuda").to(dt)
    q = torch.randn(B, hq, 128, generator=g, device="cuda").to(dt)
    return dict(q=q, kc=kc, vc=vc, table=table, lens=i32(lens), starts=None if starts is None else i32(starts), window=window, P=P, dt=dt)


def attn_call(kv, c, scale=1 / math.sqrt(128), softcap=0.0, slopes=None, out_dtype=F32, ws=None, stream=None, out=None, lse=None):
    B, hq = c["q"].shape[:2]
    if ws is None:
        ws = torch.full((kv.kvarn_paged_attention_workspace_size(B, hq, c["kc"].shape[1]),), 255, dtype=torch.uint8, device="cuda")
    if out is None:
        out = torch.full((B, hq, 128), float("nan"), dtype=out_dtype, device="cuda")
    if lse is None:
        lse = torch.full((B, hq), float("nan"), device="cuda")
    kv.kvarn_paged_attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], out, scale, ws, softcap=softcap, slopes=slopes,
                             window=c["window"], kv_starts=c["starts"], lse=lse, stream=stream)
    return out, lse


def attn_check(c, out, lse, scale=1 / math.sqrt(128), softcap=0.0, slopes=None):
    want, want_lse, mass, reach = o.paged_attention(
        np64(c["q"]), np64(c["kc"]), np64(c["vc"]), c["table"].cpu().numpy(), c["lens"].cpu().numpy(), scale, softcap,
        None if slopes is None else np64(slopes), c["window"], None if c["starts"] is None else c["starts"].cpu().numpy())
    got, got_lse = np64(out), np64(lse)
    bias = 0.0 if slopes is None else np64(slopes)[None] * np64(c["lens"])[:, None]
    err = reach * 2.0 ** -19 + softcap * 2.0 ** -21 + np.abs(bias) * 2.0 ** -23 + np.abs(bias + reach) * 2.0 ** -22
    pieces = 2.0 ** -16 if out.dtype == BF else 2.0 ** -22
    tol = (2 * err + pieces + 2.0 ** -20)[..., None] * mass + HALF_STEP[out.dtype] * np.abs(want) * (out.dtype != F32)
    tol += float(torch.finfo(out.dtype).smallest_normal)
    assert np.array_equal(np.isneginf(got_lse), np.isneginf(want_lse))
    bad = np.abs(got - want) > tol
    assert not bad.any(), (np.argwhere(bad)[:4], np.abs(got - want)[bad][:4], tol[bad][:4])
    fin = np.isfinite(want_lse)
    assert np.all(np.abs(got_lse[fin] - want_lse[fin]) <= err[fin] + 2.0 ** -22 * np.abs(want_lse[fin]) + 2.0 ** -17)


LENS = [0, 1, 15, 16, 17, 127, 128, 129, 500, 0, 1000, 33]


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (8, 1), (8, 2), (5, 1), (32, 2), (17, 1), (48, 2), (71, 1)])
@pytest.mark.parametrize("P,layout,dt", [(16, "hnd", BF), (48, "nhd", HF), (128, "both", BF)])
@pytest.mark.parametrize("wide", [False, True])
def test_attention_matches_the_oracle(kv, hq, hkv, P, layout, dt, wide):
    c = attn_case(31, LENS, hq, hkv, P=P, dt=dt, layout=layout, wide=wide)
    attn_check(c, *attn_call(kv, c))


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("lens", [[0], [1], [16], [17], [0, 0, 0], [4000], [3, 5000, 1], [2000] * 3, [1] * 300, list(range(0, 700))])
def test_attention_lengths(kv, lens, wide):
    c = attn_case(32, lens, 4, 2, P=32, wide=wide)
    attn_check(c, *attn_call(kv, c))


@pytest.mark.parametrize("out_dtype", [F32, HF, BF])
@pytest.mark.parametrize("kw", [
    dict(softcap=20.0), dict(slopes=True), dict(window=1), dict(window=16), dict(window=100), dict(window=10 ** 6), dict(starts=True),
    dict(starts=True, window=90, slopes=True, softcap=5.0), dict(scale=0.0), dict(scale=-0.2), dict(scale=1.5)])
def test_attention_modifiers(kv, kw, out_dtype):
    lens = LENS + [2500]
    starts = [0, 1, 15, 3, 16, 126, 200, 17, 499, 5, -4, 32, 1111] if kw.get("starts") else None
    dt = HF if out_dtype == HF else BF
    c = attn_case(33, lens, 12, 3, P=32, dt=dt, starts=starts, window=kw.get("window", 0), wide=out_dtype == BF)
    slopes = 2.0 ** (-8 * torch.arange(1, 13, device="cuda") / 12) if kw.get("slopes") else None
    m = dict(scale=kw.get("scale", 1 / math.sqrt(128)), softcap=kw.get("softcap", 0.0), slopes=slopes)
    attn_check(c, *attn_call(kv, c, out_dtype=out_dtype, **m), **m)


def test_attention_garbage_of_every_kind_stays_out(kv):
    for garbage in (float("inf"), -float("inf"), float("nan")):
        c = attn_case(34, [1, 47, 300], 8, 2, P=64, garbage=garbage, starts=[0, 46, 150])
        attn_check(c, *attn_call(kv, c))


def test_attention_lengths_past_the_table_and_negative_are_clamped(kv):
    c = attn_case(35, [64, 64, 64], 4, 1, P=16)
    c["table"] = c["table"][:, :4].contiguous()
    c["lens"] = i32([10 ** 9, -5, 64])
    attn_check(c, *attn_call(kv, c))


def test_attention_rows_of_minus_infinity_and_sharp_scores(kv):
    c = attn_case(36, [40, 200], 2, 1, spread=12.0)  # scores of tens: one key takes nearly all
    attn_check(c, *attn_call(kv, c, scale=1.0), scale=1.0)
    c["q"].zero_()
    c["q"][0, 0, 0] = 1.0
    c["kc"][int(c["table"][0, 0]), 0, :, 0] = -float("inf")
    c["kc"][int(c["table"][0, 1]), 0, :, 0] = -float("inf")
    c["kc"][int(c["table"][0, 2]), 0, :8, 0] = -float("inf")
    out, lse = attn_call(kv, c)
    assert not out[0, 0].any() and torch.isneginf(lse[0, 0])  # every score is -inf
    c["kc"][int(c["table"][0, 2]), 0, 3, 0] = 1.0  # but one: its value is the output
    out, lse = attn_call(kv, c)
    assert torch.equal(out[0, 0], c["vc"][int(c["table"][0, 2]), 0, 3].float())
    assert torch.isnan(out[0, 1]).all()  # 0 * -inf


def test_attention_many_small_probabilities(kv):
    # one key far above 40 000 others, whose probabilities of about 2^-17 still make half of the sum: a 16-bit
    # number of that size has few digits left
    for dt in (HF, BF):
        c = attn_case(49, [40000], 2, 1, P=128, dt=dt, spread=0.02)
        c["q"].fill_(1.0)
        page = int(c["table"][0, 200])
        c["kc"][page, 0, 5] = 1.0  # score 128 * scale
        scale = 17 * math.log(2) / 128
        out, lse = attn_call(kv, c, scale=scale)
        attn_check(c, out, lse, scale=scale)
        want = o.paged_attention(np64(c["q"]), np64(c["kc"]), np64(c["vc"]), c["table"].cpu().numpy(), [40000], scale)[0]
        # the large score (17 in the log2 domain) is off by two roundings, 2 * 17 ln 2 * 2^-24 = 1.4e-6 of its weight,
        # half of the sum; the small ones' errors average out over the keys
        assert rel_l2(np64(out), want) <= 2e-6


def test_attention_bad_pages_count_as_zeros_and_are_reported(kv):
    c = attn_case(37, [100, 100], 4, 2, P=16, garbage=0.0)
    c["table"][0, 2], c["table"][1, 5] = -1, c["kc"].shape[0]
    attn_check(c, *attn_call(kv, c))
    assert kv.kvarn_device_error() == 64


def test_attention_strided_queries(kv):
    c = attn_case(38, [50, 700, 3], 8, 2)
    wide = torch.randn(3, 13, 136, device="cuda").to(BF)
    c["q"] = wide[:, 2:10, :128]
    attn_check(c, *attn_call(kv, c))


def test_attention_repeats_bit_for_bit_and_ignores_the_workspace(kv):
    c = attn_case(39, [3000, 17, 900, 0, 5000], 16, 2, P=64)
    n = kv.kvarn_paged_attention_workspace_size(5, 16, 2)
    a = attn_call(kv, c, ws=torch.zeros(n, dtype=torch.uint8, device="cuda"))
    b = attn_call(kv, c, ws=torch.full((n,), 127, dtype=torch.uint8, device="cuda"))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_attention_cache_past_32_bit_offsets(kv):
    # 2.2e9 elements per cache: the pages in use are the last ones
    P, n_pages, hkv = 128, 17000, 8
    kc, vc = (torch.empty(n_pages, P, hkv, 128, dtype=BF, device="cuda").transpose(1, 2) for _ in range(2))
    c = attn_case(40, [300, 129], 16, hkv, P=P, garbage=0.0, layout="nhd")
    small = c["kc"].shape[0]
    for big, src in ((kc, c["kc"]), (vc, c["vc"])):
        big[n_pages - small:] = src
    want, want_lse = attn_call(kv, c)
    shift = dict(c, kc=kc, vc=vc, table=torch.where(c["table"] < small, c["table"] + (n_pages - small), c["table"]))
    out, lse = attn_call(kv, shift)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    attn_check(c, out, lse)
    # and the write of a key and value there
    r = rope_case(41, 5, 2, hkv, P=P)
    slots = n_pages * P - 1 - 3 * torch.arange(5, device="cuda", dtype=torch.int32)
    r2 = dict(r, kc=kc, vc=vc, slots=slots)
    rope_call(kv, r2)
    rope_call(kv, dict(r, slots=torch.arange(5, device="cuda", dtype=torch.int32)))
    s = slots.long()
    assert torch.equal(kc[s // P, :, s % P], r["kc"][0, :, :5].transpose(0, 1))
    assert torch.equal(vc[s // P, :, s % P], r["vc"][0, :, :5].transpose(0, 1))


def test_attention_graphs_share_a_workspace_and_follow_the_lengths(kv):
    c1, c2 = attn_case(42, [2500, 600], 8, 2, P=32), attn_case(43, [40, 9, 3100], 8, 2, P=16)
    ws = torch.empty(kv.kvarn_paged_attention_workspace_size(3, 8, 2), dtype=torch.uint8, device="cuda")
    outs = [(torch.empty(n, 8, 128, device="cuda"), torch.empty(n, 8, device="cuda")) for n in (2, 3)]
    g1 = _capture(lambda: attn_call(kv, c1, ws=ws, out=outs[0][0], lse=outs[0][1]))
    g2 = _capture(lambda: attn_call(kv, c2, ws=ws, out=outs[1][0], lse=outs[1][1]))
    for lens in ([2500, 600], [1, 0], [1777, 320]):
        c1["lens"].copy_(i32(lens))
        for t in outs[0] + outs[1]:
            t.fill_(float("nan"))
        for _ in range(3):
            g1.replay()
            g2.replay()
        torch.cuda.synchronize()
        for c, (out, lse) in ((c1, outs[0]), (c2, outs[1])):
            want, want_lse = attn_call(kv, c)
            assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_attention_on_side_streams_with_their_own_workspaces(kv):
    cs = [attn_case(44 + i, [3000, 10 * i, 999], 8, 2, P=32) for i in range(3)]
    want = [attn_call(kv, c) for c in cs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = []
    for _ in range(5):
        for c, s in zip(cs, streams):
            with torch.cuda.stream(s):
                got.append((c, attn_call(kv, c)))
    torch.cuda.synchronize()
    for c, (out, lse) in got:
        i = [x is c for x in cs].index(True)
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


def test_attention_without_log_sums(kv):
    for wide in (False, True):
        c = attn_case(48, [0, 700, 31], 8, 2, P=32, wide=wide)
        want, _ = attn_call(kv, c)
        out = torch.full_like(want, float("nan"))
        ws = torch.empty(kv.kvarn_paged_attention_workspace_size(3, 8, 2), dtype=torch.uint8, device="cuda")
        kv.kvarn_paged_attention(c["q"], c["kc"], c["vc"], c["table"], c["lens"], out, 1 / math.sqrt(128), ws)
        assert torch.equal(out, want)


def test_first_calls_of_a_process_may_be_captured(kv):
    """In a process of its own, so that nothing is loaded or looked up before the capture."""
    code = """
import torch, bit_kv_cache_kvarn_gb300 as kv
kv.load()
i32 = dict(dtype=torch.int32, device="cuda")
B, T, P = 2, 40, 16
lens, new, cnt, nf = torch.zeros(B, **i32), torch.tensor([15, 25], **i32), torch.zeros(B, **i32), torch.tensor([9], **i32)
out = [torch.empty(B, **i32), torch.empty(B, **i32), torch.empty(1, **i32), torch.empty(B + 1, **i32), torch.empty(T, **i32),
       torch.empty(T, **i32), torch.empty(1, **i32)]
table, free = torch.full((B, 4), -1, **i32), torch.arange(9, **i32)
qkv = torch.randn(T, 6, 128, device="cuda").to(torch.bfloat16)
f = kv.kvarn_rope_frequencies()[0].cuda()
qo = torch.empty(T, 4, 128, dtype=torch.bfloat16, device="cuda")
kc, vc = (torch.zeros(9, 1, P, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
wide = torch.zeros(B, 5000, **i32)
ws = torch.empty(kv.kvarn_paged_attention_workspace_size(B, 4, 1), dtype=torch.uint8, device="cuda")
res = [torch.empty(B, 4, 128, device="cuda") for _ in range(2)]

def step():
    kv.kvarn_step_tables(lens, new, cnt, table, free, nf, P, *out, )
    kv.kvarn_rope_qkv(qkv[:, :4], qkv[:, 4:5], qkv[:, 5:], out[4], f, qo, kc, vc, slot_map=out[5])
    kv.kvarn_paged_attention(qo[14:16], kc, vc, table, out[0], res[0], 0.1, ws)
    wide[:, :4] = table
    kv.kvarn_paged_attention(qo[14:16], kc, vc, wide, out[0], res[1], 0.1, ws)

torch.cuda.synchronize()
s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
with torch.cuda.stream(s):
    with torch.cuda.graph(g, stream=s):
        step()
g.replay()
torch.cuda.synchronize()
a, b = res[0].clone(), res[1].clone()
assert torch.isfinite(a).all() and a.abs().max() > 0 and torch.allclose(a, b, rtol=1e-4, atol=1e-5)
step()
torch.cuda.synchronize()
assert torch.equal(a, res[0]) and torch.equal(b, res[1]) and kv.kvarn_device_error() == 0
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


def test_attention_python_refusals(kv):
    c = attn_case(47, [20], 4, 2)
    for change, match in ((dict(lens=c["lens"].long()), "kv_lens"), (dict(q=c["q"].half()), "k_cache"), (dict(vc=c["vc"].transpose(1, 2)), "v_cache"),
                          (dict(table=c["table"][0]), "page_table"), (dict(q=c["q"].cpu()), "current CUDA"), (dict(lens=i32([20, 3])), "kv_lens")):
        with pytest.raises(ValueError, match=match):
            attn_call(kv, {**c, **change})
    with pytest.raises(kv.KvarnError, match="workspace"):
        attn_call(kv, c, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))


# ---- together ---------------------------------------------------------------------------------------------
def test_serving_steps_over_paged_and_packed_caches(kv):
    """Steps of a small server: tables -> norm, rotation, write -> attention over the 16-bit pages; and the
    same tokens through kvarn_append_tokens and kvarn_decode_attention over the packed pool, whose tiles the
    tables name.  Sequences join, draft tokens are taken back and finished ones leave their pages."""
    B, hq, hkv, P, width, n_pages = 6, 8, 2, 128, 4, 14
    g = torch.Generator(device="cuda").manual_seed(50)
    cfg = kv.kvarn_config_from_preset("kvarn_k4v2_g128")
    kc, vc = (torch.full((n_pages, hkv, P, 128), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    freqs, _ = kv.kvarn_rope_frequencies(128, 1e6)
    freqs = freqs.cuda()
    qw, kw = (1 + 0.2 * torch.randn(128, generator=g, device="cuda") for _ in range(2))
    lens, counts, n_free, status = i32([0] * B), i32([0] * B), i32([n_pages]), i32([0])
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    blocks = torch.full((B, hkv, width), 0, dtype=torch.int32, device="cuda")
    free = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    cu, ws = i32([0] * (B + 1)), torch.empty(kv.kvarn_paged_attention_workspace_size(B, hq, hkv), dtype=torch.uint8, device="cuda")
    tiles = n_pages * hkv
    pools = [torch.zeros(tiles, 128 * 16 * bits, dtype=torch.uint8, device="cuda") if i == 0 else
             torch.zeros(tiles, 512, dtype=torch.uint8, device="cuda") if i == 1 else torch.zeros(tiles, device="cuda")
             for bits in (cfg.k_bits, cfg.v_bits) for i in range(3)]
    tails = [torch.zeros(B, hkv, 128, 128, dtype=BF, device="cuda") for _ in range(2)]
    packed_lens = i32([0] * B)
    aws = torch.empty(kv.kvarn_append_workspace_size(B, hkv), dtype=torch.uint8, device="cuda")
    dws = torch.empty(kv.kvarn_decode_workspace_size(cfg, B, hq, hkv, width), dtype=torch.uint8, device="cuda")
    ref_k, ref_v = [[] for _ in range(B)], [[] for _ in range(B)]  # what each sequence holds, fp64
    steps = [[120, 3, 0, 100, 1, 0], [5, 0, 0, 50, 1, 127], [1, 1, 0, 1, 1, 1], [100, -1, 90, 1, -1, 1], [1, 110, 60, 1, 0, 1],
             [-1, 1, 1, 120, 128, 1], [1, 1, 1, -1, 1, 1]]
    for n, new in enumerate(steps):
        new_t = i32(new)
        rows = 520
        positions, slots = i32([-5] * rows), i32([-5] * rows)
        finished = [b for b in range(B) if new[b] < 0]
        kv.kvarn_step_tables(lens, new_t, counts, table, free, n_free, P, lens, counts, n_free, cu, positions, slots, status,
                             block_table=blocks)
        qkv = torch.randn(rows, hq + 2 * hkv, 128, generator=g, device="cuda").to(BF)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        qo = torch.zeros(rows, hq, 128, dtype=BF, device="cuda")
        kv.kvarn_rope_qkv(q, k, v, positions, freqs, qo, kc, vc, slot_map=slots, q_weight=qw, k_weight=kw)
        starts = cu.cpu().tolist()
        assert int(status) == 0
        last = torch.tensor([max(e - 1, 0) for e in starts[1:]], device="cuda")
        attn_q = qo[last].contiguous()
        out, lse = torch.empty(B, hq, 128, device="cuda"), torch.empty(B, hq, device="cuda")
        kv.kvarn_paged_attention(attn_q, kc, vc, table, lens, out, 1 / math.sqrt(128), ws, lse=lse)
        # the packed cache takes the same tokens, in the append layout
        most = max(max(new), 1)
        kn, vn = (torch.zeros(B, hkv, most, 128, dtype=BF, device="cuda") for _ in range(2))
        grid = torch.full((B, most), -1, dtype=torch.int32)
        row_of = torch.zeros(B, most, dtype=torch.long)
        pos_h = positions.cpu()
        for b in range(B):
            for i in range(max(new[b], 0)):
                row_of[b, i], grid[b, i] = starts[b] + i, pos_h[starts[b] + i]
        kr, vr = (x[row_of.cuda().flatten()].contiguous() for x in (k, v))
        kv.kvarn_rope_qkv(None, kr, vr, grid.flatten().cuda(), freqs, None, kn, vn, k_weight=kw)
        if finished:
            packed_lens[torch.tensor(finished, device="cuda")] = 0
        kv.kvarn_append_tokens(cfg, kn, vn, packed_lens, *tails, *pools, blocks, aws, n_accept=i32([max(x, 0) for x in new]))
        pout = torch.empty(B, hq, 128, device="cuda")
        kv.kvarn_decode_attention(cfg, attn_q, hkv, *pools, blocks, packed_lens, *tails, 1 / math.sqrt(128), dws, pout)
        torch.cuda.synchronize()
        assert torch.equal(packed_lens, lens) and kv.kvarn_device_error() == 0
        # oracle: positions, keys and queries of each sequence from the projections
        yk = o.norm_rotate(np64(k), np.maximum(pos_h.numpy(), 0), freqs.cpu().numpy(), np64(kw))
        for b in range(B):
            if new[b] < 0:
                ref_k[b], ref_v[b] = [], []
            for i in range(max(new[b], 0)):
                t = starts[b] + i
                assert int(pos_h[t]) == len(ref_k[b])
                ref_k[b].append(yk[t])
                ref_v[b].append(np64(v[t]))
        assert lens.tolist() == [len(x) for x in ref_k]
        assert (pos_h[starts[B]:] == -1).all() and not qo[starts[B]:].any()
        ref_packed = ko.decode_attention(np64(attn_q), hq, hkv, *(t.cpu().numpy() for t in pools), blocks.cpu().numpy(), lens.tolist(),
                                         np64(tails[0]), np64(tails[1]), 1 / math.sqrt(128), cfg.k_bits, cfg.v_bits)
        for b in range(B):
            L = len(ref_k[b])
            if L == 0:
                assert not out[b].any() and torch.isneginf(lse[b]).all() and not pout[b].any()
                continue
            kk, vv = np.stack(ref_k[b], 1), np.stack(ref_v[b], 1)  # [hkv, L, 128]
            for h in range(hq):
                s = kk[h // (hq // hkv)] @ np64(attn_q[b, h]) / math.sqrt(128)
                p = np.exp(s - s.max())
                want = p @ vv[h // (hq // hkv)] / p.sum()
                # the cached keys are rounded to bf16: a score is off by at most 2^-8 sum |q k|, in practice a
                # random sum of 128 such terms; the bound is the worst case
                reach = (np.abs(kk[h // (hq // hkv)]) @ np.abs(np64(attn_q[b, h]))).max() / math.sqrt(128)
                tol = np.expm1(2 * reach * 2.0 ** -8) * (p @ np.abs(vv[h // (hq // hkv)]) / p.sum()) + 1e-5
                assert np.all(np.abs(np64(out[b, h]) - want) <= tol)
                assert rel_l2(np64(pout[b, h]), ref_packed[b, h]) <= 1e-3
    assert int(n_free) + int(counts.sum()) == n_pages


def test_pseudo_decode_over_the_paged_cache(kv):
    """The unquantised pseudo-decode through the serving step's kernels, block by block and layer by layer:
    its attention from the queries and pages it had, and against the plain PyTorch run."""
    from bit_kv_cache_kvarn_gb300 import pseudo_decode as pd

    hq, hkv, layers, blocks = 4, 2, 2, 4
    w = pd.make_weights(41, layers, 256, hq, hkv)
    x = pd.make_input(41, blocks * 128, 256)
    cap = {(j, l): None for j in range(blocks) for l in range(layers)}
    attn, _ = pd.run(kv, None, w, x, hq, hkv, quantised=False, paged=True, capture=cap)
    plain, _ = pd.run(kv, None, w, x, hq, hkv, quantised=False)
    scale = 1 / math.sqrt(128)
    for (j, l), c in cap.items():
        lens = i32([128 * j + t + 1 for t in range(128)])
        case = dict(q=c["q"], kc=c["k_pages"], vc=c["v_pages"], table=c["table"].expand(128, -1), lens=lens, starts=None, window=0)
        _, lse, mass, reach = o.paged_attention(np64(c["q"]), np64(c["k_pages"]), np64(c["v_pages"]), case["table"].cpu().numpy(),
                                                lens.tolist(), scale)
        attn_check(case, attn[j][l], torch.tensor(lse), scale=scale)
        if l == 0:
            # the runs' queries, keys and values are the same fp32 numbers up to their last bits, so each
            # bf16 value differs by a step (2^-7) at most; a score then by 2 * 2^-7 reach
            tol = np.expm1(4 * reach * 2.0 ** -7)[..., None] * mass + 2.0 ** -7 * mass
            assert np.all(np.abs(np64(attn[j][0]) - np64(plain[j][0])) <= tol)
    with pytest.raises(ValueError, match="paged"):
        pd.run(kv, None, w, x, hq, hkv, quantised=True, paged=True)
