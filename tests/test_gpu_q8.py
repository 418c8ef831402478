"""The 8-bit cache on the GPU: the write against the fp64 oracle, exactly; attention over it against the oracle.

Attention's tolerance is kvarn_paged_attention's (test_gpu_serving.py derives it) with exact codes and exponents; two
fp16 pieces of a probability leave 2^-22 of it, and below the normal numbers 2^-40 of the largest p 2^e, whose product
with a code is at most twice the largest p |v|."""
import math

import numpy as np
import pytest
import torch

from oracle import serving as o
from tests.test_gpu_graph import _capture
from tests.test_gpu_prompt import BF, F32, HF, SCALE, i32, np64

pytestmark = pytest.mark.gpu
E4 = torch.float8_e4m3fn
HALF_STEP = {BF: 2.0 ** -8, HF: 2.0 ** -11, F32: 2.0 ** -24}


@pytest.fixture(autouse=True)
def _no_device_error(kv):
    kv.kvarn_device_error()
    yield
    assert kv.kvarn_device_error() == 0


def empty_cache(n_pages, hkv, P, layout="hnd", code=0x7f, e=127):
    """Codes (NaN unless said otherwise) and exponents of an unwritten cache."""
    shape = {"hnd": (n_pages, hkv, P, 128), "nhd": (n_pages, P, hkv, 128), "both": (n_pages, 2, hkv, P, 144)}[layout]
    if layout == "both":
        both = torch.full(shape, code, dtype=torch.uint8, device="cuda")
        kc, vc = both[:, 0, :, :, :128], both[:, 1, :, :, :128]
    else:
        kc, vc = (torch.full(shape, code, dtype=torch.uint8, device="cuda") for _ in range(2))
        if layout == "nhd":
            kc, vc = kc.transpose(1, 2), vc.transpose(1, 2)
    return kc.view(E4), vc.view(E4), *(torch.full((n_pages, hkv, P), e, dtype=torch.int8, device="cuda") for _ in range(2))


def bytes_of(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


# ---- the write ----------------------------------------------------------------------------------------
def check_write(k, v, cache, slots, before):
    kc, vc, ke, ve = cache
    P = kc.shape[2]
    codes, exps = [np64(t) for t in (kc, vc)], [t.cpu().numpy().copy() for t in (ke, ve)]
    for x, code, e, old_code, old_e in zip((k, v), codes, exps, before[:2], before[2:]):
        want, want_e = o.quantize_row(np64(x))
        seen = np.zeros(code.shape[:3], bool)
        for t, s in enumerate(slots):
            if s < 0:
                continue
            seen[s // P, :, s % P] = True
            got = code[s // P, :, s % P]
            assert np.array_equal(e[s // P, :, s % P], want_e[t]), (t, e[s // P, :, s % P], want_e[t])
            assert np.array_equal(got, want[t], equal_nan=True), (t, np.argwhere(got != want[t])[:4])
        # the rest of the cache is as before
        kept = code.copy()
        assert np.array_equal(kept[~seen], old_code[~seen], equal_nan=True) and np.array_equal(e[~seen], old_e[~seen])


@pytest.mark.parametrize("T,hkv", [(1, 1), (3, 8), (130, 2), (517, 5)])
@pytest.mark.parametrize("dt,P,layout", [(BF, 16, "hnd"), (HF, 48, "nhd"), (F32, 1, "hnd"), (BF, 128, "both")])
def test_write_matches_the_oracle_exactly(kv, T, hkv, dt, P, layout):
    g = torch.Generator(device="cuda").manual_seed(T + hkv)
    fused = (torch.randn(T, 3 * hkv, 128, generator=g, device="cuda") * torch.exp(3 * torch.randn(T, 3 * hkv, 1, generator=g, device="cuda"))).to(dt)
    k, v = fused[:, hkv:2 * hkv], fused[:, 2 * hkv:]
    n_pages = -(-T // P) + 2
    cache = empty_cache(n_pages, hkv, P, layout, code=0x11, e=3)
    before = [np64(cache[0]), np64(cache[1]), cache[2].cpu().numpy().copy(), cache[3].cpu().numpy().copy()]
    slots = torch.randperm(n_pages * P, generator=g, device="cuda")[:T].to(torch.int32)
    slots[torch.rand(T, generator=g, device="cuda") < 0.2] = -1
    kv.kvarn_quantize_kv(k, v, *cache, slot_map=slots)
    check_write(k, v, cache, slots.tolist(), before)


def test_write_of_ties_borders_and_special_values(kv):
    rows = []
    grid = o.e4m3_grid()
    for e in (-20, 0, 7):
        mid = (grid[1:] + grid[:-1]) / 2  # exactly between two codes
        rows += [np.concatenate([mid, [448.0, -448.0]]) * 2.0 ** e, np.concatenate([-mid, [448.0, 0.0]]) * 2.0 ** e]
    for top in (448.0, np.nextafter(np.float32(448), np.float32(449)), 447.99997, 1.75, 1.7500001, 2.0 ** -126, 2.0 ** -140, 3.4e38, 0.0):
        rows.append(np.concatenate([[top], np.linspace(-top, top, 127)]))
    rows.append(np.concatenate([[np.nan, 1.0], np.full(126, 0.3)]))
    rows.append(np.concatenate([[np.inf, -np.inf, 1.0], np.full(125, 3e38)]))
    rows.append(np.full(128, np.nan))
    rows.append(np.full(128, -0.0))
    x = torch.tensor(np.array(rows), dtype=F32, device="cuda")[:, None].contiguous()
    T = x.shape[0]
    cache = empty_cache(T, 1, 1, code=0x11, e=3)
    kv.kvarn_quantize_kv(x, -x, *cache)
    before = [np.zeros((T, 1, 1, 128))] * 2 + [np.zeros((T, 1, 1))] * 2
    check_write(x, -x, cache, list(range(T)), before)
    assert (np.signbit(np64(cache[0])[-1]).all())  # -0 keeps its sign


def test_write_reports_slots_outside_the_cache(kv):
    x = torch.ones(4, 2, 128, dtype=BF, device="cuda")
    cache = empty_cache(2, 2, 16, code=0x11, e=3)
    kv.kvarn_quantize_kv(x, x, *cache, slot_map=i32([0, 32, -2, -1]))
    assert kv.kvarn_device_error() == 32
    kv.kvarn_quantize_kv(x[:0], x[:0], *cache, slot_map=i32([]))
    assert (bytes_of(cache[0]) != 0x11).sum() == 256 and (cache[2] != 3).sum() == 2


# ---- attention -----------------------------------------------------------------------------------------
def case(seed, lens, hq, hkv, P=16, dt=BF, layout="hnd", starts=None, window=0, spread=1.0, wide=False, sizes=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, used = len(lens), [-(-n // P) for n in lens]
    width, n_pages = max(max(used), -(-100000 // P) if wide else 0) + 1, sum(used) + 3
    perm = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, width), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    cache = empty_cache(n_pages, hkv, P, layout)
    at = 0
    for b, n in enumerate(lens):
        lo = min(n, max(0 if starts is None else starts[b], n - window if window else 0, 0))
        if n > lo:
            table[b, lo // P:used[b]] = perm[at + lo // P:at + used[b]]
            j = torch.arange(lo, n, device="cuda")
            slots = perm[at + j // P] * P + (j % P).int()
            size = torch.exp(sizes * torch.randn(2, n - lo, hkv, 1, generator=g, device="cuda"))
            k, v = torch.randn(2, n - lo, hkv, 128, generator=g, device="cuda") * size
            for x, code, e in ((spread * k, cache[0], cache[2]), (v, cache[1], cache[3])):
                want, want_e = o.quantize_row(np64(x))
                s = slots.long()
                code.view(torch.uint8)[s // P, :, s % P] = torch.tensor(want, device="cuda").to(E4).view(torch.uint8)
                e[s // P, :, s % P] = torch.tensor(want_e, dtype=torch.int8, device="cuda")
        at += used[b]
    q = torch.randn(B, hq, 128, generator=g, device="cuda").to(dt)
    return dict(q=q, cache=cache, table=table, lens=i32(lens), starts=None if starts is None else i32(starts), window=window, P=P, dt=dt)


def call(kv, c, scale=SCALE, softcap=0.0, slopes=None, out_dtype=F32, ws=None, stream=None, out=None, lse=None):
    B, hq = c["q"].shape[:2]
    if ws is None:
        ws = torch.full((kv.kvarn_paged_attention_workspace_size(B, hq, c["cache"][0].shape[1]),), 255, dtype=torch.uint8, device="cuda")
    if out is None:
        out = torch.full((B, hq, 128), math.nan, dtype=out_dtype, device="cuda")
    if lse is None:
        lse = torch.full((B, hq), math.nan, device="cuda")
    kv.kvarn_paged_attention_q8(c["q"], *c["cache"], c["table"], c["lens"], out, scale, ws, softcap=softcap, slopes=slopes,
                                window=c["window"], kv_starts=c["starts"], lse=lse, stream=stream)
    return out, lse


def check(c, out, lse, scale=SCALE, softcap=0.0, slopes=None):
    kc, vc, ke, ve = c["cache"]
    k, v = (np64(x) * 2.0 ** e.cpu().numpy().astype(float)[..., None] for x, e in ((kc, ke), (vc, ve)))
    want, want_lse, mass, reach = o.paged_attention(
        np64(c["q"]), k, v, c["table"].cpu().numpy(), c["lens"].cpu().numpy(), scale, softcap,
        None if slopes is None else np64(slopes), c["window"], None if c["starts"] is None else c["starts"].cpu().numpy())
    got, got_lse = np64(out), np64(lse)
    bias = 0.0 if slopes is None else np64(slopes)[None] * np64(c["lens"])[:, None]
    err = reach * 2.0 ** -19 + softcap * 2.0 ** -21 + np.abs(bias) * 2.0 ** -23 + np.abs(bias + reach) * 2.0 ** -22
    tol = (2 * err + 2.0 ** -22 + 2.0 ** -20)[..., None] * mass + HALF_STEP[out.dtype] * np.abs(want) * (out.dtype != F32)
    tol += (np64(c["lens"])[:, None] * 2.0 ** -39 * mass.max(-1))[..., None] + float(torch.finfo(out.dtype).smallest_normal)
    assert np.array_equal(np.isneginf(got_lse), np.isneginf(want_lse))
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:4], np.abs(got - want)[bad][:4], tol[bad][:4])
    fin = np.isfinite(want_lse)
    assert np.all(np.abs(got_lse[fin] - want_lse[fin]) <= err[fin] + 2.0 ** -22 * np.abs(want_lse[fin]) + 2.0 ** -17)


LENS = [0, 1, 15, 16, 17, 127, 128, 129, 500, 0, 1000, 33]


@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (8, 1), (8, 2), (5, 1), (32, 2), (17, 1), (71, 1)])
@pytest.mark.parametrize("P,layout,dt", [(16, "hnd", BF), (48, "nhd", HF), (128, "both", BF)])
@pytest.mark.parametrize("wide", [False, True])
def test_attention_matches_the_oracle(kv, hq, hkv, P, layout, dt, wide):
    c = case(hq + P, LENS, hq, hkv, P, dt, layout, wide=wide)
    check(c, *call(kv, c))


@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("lens", [[0], [1], [16], [17], [0, 0, 0], [4000], [3, 5000, 1], [1] * 300])
def test_attention_lengths(kv, lens, wide):
    c = case(len(lens) + lens[0], lens, 8, 2, wide=wide)
    check(c, *call(kv, c))


@pytest.mark.parametrize("out_dtype", [F32, HF, BF])
@pytest.mark.parametrize("kw", [dict(softcap=30.0), dict(slopes=True), dict(window=100), dict(starts=True),
                                dict(starts=True, window=37, softcap=5.0, slopes=True), dict(scale=-0.3), dict(scale=0.0)])
def test_attention_modifiers(kv, kw, out_dtype):
    kw = dict(kw)
    starts = [0, 1, 20, 3, 5, 64, 200, 0, 490, 7, 300, 0] if kw.pop("starts", False) else None
    slopes = 2.0 ** -torch.arange(1, 9, device="cuda", dtype=F32) if kw.pop("slopes", False) else None
    window = kw.pop("window", 0)
    c = case(5, LENS, 8, 2, 16, HF if out_dtype == HF else BF, starts=starts, window=window)
    check(c, *call(kv, c, slopes=slopes, out_dtype=out_dtype, **kw), slopes=slopes, **kw)


@pytest.mark.parametrize("sizes,spread", [(6.0, 1.0), (6.0, 1e-3), (2.0, 10.0)])
def test_attention_with_exponents_far_apart(kv, sizes, spread):
    c = case(9, [700, 40, 1], 8, 2, sizes=sizes, spread=spread)
    check(c, *call(kv, c))


def test_attention_queries_of_every_size(kv):
    # a bf16 query enters the product as fp16 with a power of two of its own
    c = case(10, [300] * 8, 8, 2)
    c["q"] *= torch.tensor([1e30, 1e-30, 1.0, 2.0 ** -133, 0.0, 3e4, 1e-8, 70000.0], device="cuda").to(BF)[:, None, None]
    for b, scale in ((0, 1e-31), (1, 1e29), (2, 0.1), (3, 1.0), (4, 1.0), (5, 1e-5), (6, 1e7), (7, 1e-6)):
        d = {**c, "q": c["q"][b:b + 1], "table": c["table"][b:b + 1].contiguous(), "lens": c["lens"][b:b + 1].contiguous()}
        check(d, *call(kv, d, scale=scale), scale=scale)


def test_attention_bad_pages_count_as_zeros_and_are_reported(kv):
    c = case(12, [100, 40], 4, 2)
    c["table"][0, 2], c["table"][1, 0] = -5, 2 ** 30
    out, lse = call(kv, c)
    assert kv.kvarn_device_error() == 64
    check(c, out, lse)


def test_attention_of_written_rows_repeats_and_follows_replays(kv):
    """A decode loop over 8-bit pages in one graph: write of the step's rows, attention over all so far."""
    B, hq, hkv, P, steps = 3, 8, 2, 16, 40
    g = torch.Generator(device="cuda").manual_seed(70)
    cache = empty_cache(B * 4, hkv, P)
    table = torch.arange(B * 4, dtype=torch.int32, device="cuda").view(B, 4)
    rows = torch.randn(2, steps, B, hkv, 128, generator=g, device="cuda").to(BF)
    k, v, slots, lens = torch.empty_like(rows[0, 0]), torch.empty_like(rows[0, 0]), i32([0] * B), i32([0] * B)
    q = torch.randn(B, hq, 128, generator=g, device="cuda").to(BF)
    ws = torch.empty(kv.kvarn_paged_attention_workspace_size(B, hq, hkv), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty(B, hq, 128, device="cuda"), torch.empty(B, hq, device="cuda")
    slots.copy_(table[:, 0] * P)

    def step():
        kv.kvarn_quantize_kv(k, v, *cache, slot_map=slots)
        kv.kvarn_paged_attention_q8(q, *cache, table, lens, out, SCALE, ws, lse=lse)

    graph = _capture(step)
    for t in range(steps):
        k.copy_(rows[0, t])
        v.copy_(rows[1, t])
        slots.copy_(table[:, t // P] * P + t % P)
        lens.fill_(t + 1)
        graph.replay()
    torch.cuda.synchronize()
    c = dict(q=q, cache=cache, table=table, lens=lens, starts=None, window=0, P=P, dt=BF)
    check(c, out, lse)
    again, again_lse = call(kv, c)
    assert torch.equal(out, again) and torch.equal(lse, again_lse)
    # what an 8-bit cache costs against the rows themselves: a value and a key are off by up to 2^-4 of each element
    dense_k, dense_v = (x.double().permute(1, 2, 0, 3).cpu().numpy() for x in rows)
    s = np.einsum("bhgc,bhtc->bhgt", np64(q).reshape(B, hkv, hq // hkv, 128), dense_k) * SCALE
    p = np.exp(s - s.max(-1, keepdims=True))
    want = np.einsum("bhgt,bhtc->bhgc", p / p.sum(-1, keepdims=True), dense_v).reshape(B, hq, 128)
    assert np.linalg.norm(np64(out) - want) <= 2.0 ** -4 * np.linalg.norm(want)


def test_attention_cache_past_32_bit_offsets(kv):
    P, n_pages, hkv = 128, 17500, 16  # 4.6e9 bytes per cache: the pages in use are the last ones
    c = case(71, [300, 129], 32, hkv, P, layout="nhd")
    small = c["cache"][0].shape[0]
    far = empty_cache(n_pages, hkv, P, "nhd", code=0)
    for big, src in zip(far, c["cache"]):
        (big.view(torch.uint8) if big.dtype == E4 else big)[n_pages - small:] = src.view(torch.uint8) if src.dtype == E4 else src
    want = call(kv, c)
    table = torch.where(c["table"] < small, c["table"] + (n_pages - small), c["table"])
    got = call(kv, dict(c, cache=far, table=table))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    x = torch.randn(3, hkv, 128, device="cuda").to(BF)
    slots = n_pages * P - 1 - 5 * torch.arange(3, device="cuda", dtype=torch.int32)
    kv.kvarn_quantize_kv(x, x, *far, slot_map=slots)
    s = slots.long()
    want_code, want_e = o.quantize_row(np64(x))
    assert np.array_equal(np64(far[0][s // P, :, s % P]), want_code) and np.array_equal(far[3][s // P, :, s % P].cpu().numpy(), want_e)


def test_attention_repeats_and_side_streams(kv):
    cs = [case(72 + i, [3000, 10 * i, 999], 8, 2, P=32, wide=i == 1) for i in range(3)]
    want = [call(kv, c) for c in cs]
    torch.cuda.synchronize()
    got = []
    for i, s in enumerate([torch.cuda.Stream() for _ in cs] * 3):
        with torch.cuda.stream(s):
            got.append((i % 3, call(kv, cs[i % 3])))
    torch.cuda.synchronize()
    for i, (out, lse) in got:
        assert torch.equal(out, want[i][0]) and torch.equal(lse, want[i][1])


def test_rows_of_minus_infinity_and_strided_queries(kv):
    c = case(75, [200, 3], 8, 2)
    wide = torch.randn(2, 13, 136, device="cuda").to(BF)
    c["q"] = wide[:, 2:10, :128]
    check(c, *call(kv, c))
    c["q"] = torch.full((2, 8, 128), -math.inf, dtype=BF, device="cuda")
    out, lse = call(kv, c)
    assert not torch.isfinite(lse).any()  # infinities of both signs in every score


def test_python_refusals(kv):
    c = case(76, [20], 4, 2)
    kc, vc, ke, ve = c["cache"]
    for cache, match in (((kc.view(torch.uint8), vc, ke, ve), "k_cache"), ((kc, vc, ke.int(), ve), "k_exp"), ((kc, vc, ke, ve[:1]), "v_exp"),
                         ((kc, vc.transpose(1, 2), ke, ve), "v_cache")):
        with pytest.raises(ValueError, match=match):
            call(kv, {**c, "cache": cache})
        x = torch.ones(2, 2, 128, dtype=BF, device="cuda")
        with pytest.raises(ValueError, match=match):
            kv.kvarn_quantize_kv(x, x, *cache)
    x = torch.ones(2, 2, 128, dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="heads"):
        kv.kvarn_quantize_kv(x[:, :1], x[:, :1], *c["cache"])
    with pytest.raises(ValueError, match="strides"):
        kv.kvarn_quantize_kv(x, x.expand(2, 2, 128).transpose(0, 1).contiguous().transpose(0, 1), *c["cache"])
    with pytest.raises(kv.KvarnError, match="workspace"):
        call(kv, c, ws=torch.empty(16, dtype=torch.uint8, device="cuda"))
