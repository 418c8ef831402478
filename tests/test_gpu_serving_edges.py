"""The serving step's calls at the ends of their ranges, on the GPU."""
import os
import subprocess
import sys

import pytest
import torch

from tests.test_gpu_serving import BF, F32, HF, _no_device_error, attn_call, attn_case, attn_check, i32, rope_call, rope_case, rope_check  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("wide", [False, True])
@pytest.mark.parametrize("dt", [HF, BF])
@pytest.mark.parametrize("out_dtype", [F32, "16"])
def test_attention_of_huge_scores(kv, dt, wide, sign, out_dtype):
    # Scores beyond 2^24 (in the log2 domain, where neighbouring fp32 numbers are 2 and more apart).  Keys differ by
    # at least 4096 * 4 in the score, so one key takes all: the output is its value and lse its score, which is
    # off by the roundings of the products with scale and log2 e, the sum with the lift and the product with
    # ln 2: four half steps, 2^-22, of itself.
    lens, hq = [40, 200], 16
    c = attn_case(60, lens, hq, 2, P=16, dt=dt, wide=wide)
    c["q"].zero_()
    step = 4.0 if dt == HF else 32.0  # neighbours of 4096 in fp16 and bf16
    c["q"][:, :, 0] = (4096 + step * torch.arange(hq, device="cuda")).to(dt)
    best = []
    for b, n in enumerate(lens):
        for t in range(n):
            c["kc"][int(c["table"][b, t // 16]), :, t % 16, 0] = sign * (4096 + step * ((37 * t) % n))
        best.append(max(range(n), key=lambda t: sign * ((37 * t) % n)))
    out, lse = attn_call(kv, c, scale=1.0, out_dtype=dt if out_dtype == "16" else F32)
    for b in range(len(lens)):
        page, off = int(c["table"][b, best[b] // 16]), best[b] % 16
        for h in range(hq):
            assert torch.equal(out[b, h], c["vc"][page, h // 8, off].to(out.dtype))
            want = float(c["q"][b, h, 0]) * float(c["kc"][page, h // 8, off, 0])
            assert abs(float(lse[b, h]) - want) <= 2.0 ** -22 * abs(want)


def _ms(f, reps=3):
    f()
    times = []
    for _ in range(reps):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        torch.cuda.synchronize()
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b))
    return min(times)


def _sparse_batch(B, live, seed=61, starts=False):
    """B sequences of which `live` ({index: length}) hold tokens; the others are empty slots of a batch of fixed size."""
    lens = [live.get(b, 0) for b in range(B)]
    c = attn_case(seed, [n for n in lens if n], 4, 2, P=16)
    idx = torch.tensor(sorted(live), device="cuda")
    q = torch.randn(B, 4, 128, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda").to(BF)
    q[idx] = c["q"]
    table = torch.full((B, c["table"].shape[1]), 2 ** 31 - 1, dtype=torch.int32, device="cuda")
    table[idx] = c["table"]
    first = None
    if starts:  # empty because everything lies before the first visible key
        first = torch.where(i32(lens) > 0, 0, 50).to(torch.int32)
        lens = [n or 50 for n in lens]
    return dict(c, q=q, table=table, lens=i32(lens), starts=first)


@pytest.mark.parametrize("starts", [False, True])
@pytest.mark.parametrize("B,live", [(40, {0: 33}), (40, {39: 100}), (300, {0: 500, 299: 3}), (2048, {5: 40, 36: 17, 37: 1, 69: 200, 1500: 700}),
                                    (2048, {i: 1 + i % 50 for i in range(0, 2048, 33)}), (600, {i: 20 for i in range(31, 600, 32)})])
def test_attention_of_mostly_empty_batches(kv, B, live, starts):
    c = _sparse_batch(B, live, starts=starts)
    attn_check(c, *attn_call(kv, c))


def test_attention_passes_over_empty_sequences_quickly(kv):
    # One by one, with a dependent load for each, they cost some 95 ns apiece; 32 at a time, and even with a load
    # from memory (600 ns) for each 32, less than 20.
    B = 30000
    ws = torch.empty(kv.kvarn_paged_attention_workspace_size(B, 4, 2), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty(B, 4, 128, device="cuda"), torch.empty(B, 4, device="cuda")
    t = {}
    for name, live in (("together", {B - 2: 64, B - 1: 64}), ("before", {0: 64, 1: 64}), ("around", {0: 64, B - 1: 64})):
        c = _sparse_batch(B, live)
        t[name] = _ms(lambda: attn_call(kv, c, ws=ws, out=out, lse=lse))
    assert t["before"] - t["together"] <= 2e-5 * B and t["around"] - t["together"] <= 2e-5 * B, t


@pytest.mark.parametrize("T", [6, 1300])
def test_rope_slots_below_minus_one_are_reported(kv, T):
    c = rope_case(62, T, 4, 2)
    c["slots"][1] = -1
    before = [c[k].clone() for k in ("qo", "kc", "vc")]
    rope_check(c, rope_call(kv, c), *before)
    assert kv.kvarn_device_error() == 0
    c = rope_case(63, T, 4, 2)
    c["slots"][1], c["slots"][4] = -2, -(2 ** 31)
    before = [c[k].clone() for k in ("qo", "kc", "vc")]
    rope_check(c, rope_call(kv, c), *before)
    assert kv.kvarn_device_error() == 32
    c["positions"][1] = c["positions"][4] = -1  # a padding row's slot is not looked at
    rope_call(kv, c)
    assert kv.kvarn_device_error() == 0


def test_attention_refuses_caps_below_the_normal_range(kv):
    # 1e-50 is no fp32 number but 0, which would mean no cap
    c = attn_case(64, [20], 4, 2)
    for cap in (1e-39, 1e-50, 5e-324):
        with pytest.raises(kv.KvarnError, match="softcap"):
            attn_call(kv, c, softcap=cap)
    for cap in (2.0 ** -126, 1e-30):  # all scores are capped to about 0: the mean of the values
        attn_check(c, *attn_call(kv, c, softcap=cap), softcap=cap)


def test_pseudo_decode_raises_when_a_step_is_refused(kv, monkeypatch):
    from bit_kv_cache_kvarn_gb300 import pseudo_decode as pd

    made = pd._PagedCache.__init__

    def short(self, *args):
        made(self, *args)
        self.n_free.fill_(2)  # pages for two of the four blocks

    monkeypatch.setattr(pd._PagedCache, "__init__", short)
    w, x = pd.make_weights(41, 1, 256, 4, 2), pd.make_input(41, 4 * 128, 256)
    try:
        with pytest.raises(RuntimeError, match="status 1"):
            pd.run(kv, None, w, x, 4, 2, quantised=False, paged=True)
    finally:
        kv.kvarn_device_error()


@pytest.mark.parametrize("dt", [HF, BF])
@pytest.mark.parametrize("wide", [False, True])
def test_attention_infinite_values_stay_in_their_channel(kv, dt, wide):
    c = attn_case(65, [40, 100], 4, 2, dt=dt, wide=wide)
    want, want_lse = attn_call(kv, c)
    c["vc"][int(c["table"][1, 3]), 1, 5, 77] = float("inf")
    out, lse = attn_call(kv, c)
    assert not torch.isfinite(out[1, 2:, 77]).any()
    out[1, 2:, 77] = want[1, 2:, 77]
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_device_error_is_cleared_by_reading(kv):
    for slot, bits in ((-2, 32), (-1, 0)):
        c = rope_case(66, 4, 2, 1)
        c["slots"][1] = slot
        rope_call(kv, c)
        assert kv.kvarn_device_error() == bits and kv.kvarn_device_error() == 0


def test_device_error_is_no_slower_for_callers_without_a_serving_step(kv):
    """In a process of its own that makes no serving call.  Four words are read and nothing is written: with
    the synchronisation no more than five copies of a number to the host, and one for the call itself."""
    code = """
import time, torch, bit_kv_cache_kvarn_gb300 as kv
kv.load()
x = torch.zeros(1, device="cuda")

def us(f):
    best = 1e9
    for _ in range(9):
        t = time.perf_counter()
        for _ in range(100):
            f()
        best = min(best, (time.perf_counter() - t) / 100 * 1e6)
    return best

item, error = us(x.item), us(kv.kvarn_device_error)
assert error <= 6 * item, (error, item)
print("quick")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "quick" in r.stdout, r.stderr[-2000:]
