"""Steps of a small server that use the calls together: tables, norm and rotation with the cache write, attention of the
step's packed rows; and the same sequences behind a shared prefix, and over 8-bit pages."""
import math
import os
import re

import numpy as np
import pytest
import torch

from oracle import serving as o
from tests.test_gpu_prompt import BF, SCALE, i32, np64

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _no_device_error(kv):
    kv.kvarn_device_error()
    yield
    assert kv.kvarn_device_error() == 0


def test_prompts_chunks_drafts_and_single_tokens_in_one_server(kv):
    B, hq, hkv, P, width, n_pages = 5, 8, 2, 16, 40, 120
    g = torch.Generator(device="cuda").manual_seed(80)
    kc, vc = (torch.full((n_pages, hkv, P, 128), math.nan, dtype=BF, device="cuda") for _ in range(2))
    table, free = torch.full((B, width), -1, dtype=torch.int32, device="cuda"), torch.arange(n_pages, dtype=torch.int32, device="cuda")
    lens, counts, n_free, status = i32([0] * B), i32([0] * B), i32([n_pages]), i32([0])
    freqs, rope_scale = kv.kvarn_rope_frequencies(128, 10000.0)
    freqs = freqs.cuda()
    c8 = [torch.full((n_pages, hkv, P, 128), 0x7f, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2)]
    e8 = [torch.full((n_pages, hkv, P), 99, dtype=torch.int8, device="cuda") for _ in range(2)]
    seen = [[[], []] for _ in range(B)]  # every sequence's rotated keys and its values, as the oracle has them
    for new in ([200, 0, 33, 1, 0], [1, 300, 4, 1, 0], [5, 1, 1, 1, 17], [1, 1, 130, 1, 1]):
        T = sum(new) + 3
        cu, pos, slots = i32([0] * (B + 1)), i32([0] * T), i32([0] * T)
        kv.kvarn_step_tables(lens, i32(new), counts, table, free, n_free, P, lens, counts, n_free, cu, pos, slots, status)
        qkv = torch.randn(T, hq + 2 * hkv, 128, generator=g, device="cuda").to(BF)
        q = torch.empty(T, hq, 128, dtype=BF, device="cuda")
        kv.kvarn_rope_qkv(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], pos, freqs, q, kc, vc, slot_map=slots, rope_scale=rope_scale)
        out, lse = torch.full((T, hq, 128), 0.75, dtype=BF, device="cuda"), torch.full((T, hq), 0.75, device="cuda")
        ws = torch.empty(kv.kvarn_prompt_attention_workspace_size(T, hq, hkv), dtype=torch.uint8, device="cuda")
        kv.kvarn_prompt_attention(q, kc, vc, table, cu, lens, out, SCALE, ws, lse=lse)
        # the step's keys and values, gathered from their slots, also go into 8-bit pages with the same table
        s = slots.long().clamp(min=0)
        k_rows, v_rows = kc[s // P, :, s % P].contiguous(), vc[s // P, :, s % P].contiguous()
        kv.kvarn_quantize_kv(k_rows, v_rows, *c8, *e8, slot_map=slots)
        last = (cu[1:] - 1).clamp(min=0).long()
        ws8 = torch.empty(kv.kvarn_paged_attention_workspace_size(B, hq, hkv), dtype=torch.uint8, device="cuda")
        out8 = torch.empty(B, hq, 128, device="cuda")
        kv.kvarn_paged_attention_q8(q[last], *c8, *e8, table, lens, out8, SCALE, ws8)
        torch.cuda.synchronize()
        assert int(status) == 0
        at = 0
        kn, vn = np64(k_rows), np64(v_rows)
        got, got_lse, qn, got8 = np64(out), np64(lse), np64(q), np64(out8)
        for b, n in enumerate(new):
            seen[b][0] += [kn[at + i] for i in range(n)]
            seen[b][1] += [vn[at + i] for i in range(n)]
            total = len(seen[b][0])
            for i in sorted({0, n // 2, n - 1}) if n else []:
                p = total - n + i
                k, v = (np.array(x[:p + 1]).repeat(hq // hkv, 1) for x in seen[b])
                sc = np.einsum("hc,thc->ht", qn[at + i], k) * SCALE
                w = np.exp(sc - sc.max(1, keepdims=True))
                want = np.einsum("ht,thc->hc", w / w.sum(1, keepdims=True), v)
                assert np.abs(got[at + i] - want).max() <= 2.0 ** -6 * np.abs(v).max()
                assert np.abs(got_lse[at + i] - sc.max(1) - np.log(w.sum(1))).max() <= 1e-3
                if i == n - 1:  # each code is off by 2^-4 of its element at most
                    assert np.linalg.norm(got8[b] - want) <= 2.0 ** -3 * np.linalg.norm(want)
            at += n
        assert torch.all(out[at:] == 0.75) and torch.all(lse[at:] == 0.75)


def test_answers_behind_a_prompt_that_they_share(kv):
    """One prompt through the prompt attention, then answers to it, a token at a time, each with pages of its own."""
    hq, hkv, P, B, n = 8, 2, 16, 6, 77
    g = torch.Generator(device="cuda").manual_seed(81)
    kc, vc = (torch.full((5 + 2 * B, hkv, P, 128), math.nan, dtype=BF, device="cuda") for _ in range(2))
    prompt = i32([[3, 1, 4, 0, 2]])
    own = torch.arange(5, 5 + 2 * B, dtype=torch.int32, device="cuda").view(B, 2)
    freqs = kv.kvarn_rope_frequencies(128, 10000.0)[0].cuda()

    def write(rows, positions, slots):
        q = torch.empty(rows.shape[0], hq, 128, dtype=BF, device="cuda")
        kv.kvarn_rope_qkv(rows[:, :hq], rows[:, hq:hq + hkv], rows[:, hq + hkv:], positions, freqs, q, kc, vc, slot_map=slots)
        return q

    t = torch.arange(n, device="cuda")
    write(torch.randn(n, hq + 2 * hkv, 128, generator=g, device="cuda").to(BF), t.int(), prompt[0][t // P] * P + (t % P).int())
    ws = torch.empty(kv.kvarn_prefix_attention_workspace_size(B, hq, hkv), dtype=torch.uint8, device="cuda")
    for i in range(20):
        rows = torch.randn(B, hq + 2 * hkv, 128, generator=g, device="cuda").to(BF)
        q = write(rows, i32([n + i] * B), own[:, i // P] * P + i % P)
        out, lse = torch.empty(B, hq, 128, dtype=BF, device="cuda"), torch.empty(B, hq, device="cuda")
        lens = i32([i + 1] * B)
        kv.kvarn_prefix_attention(q, kc, vc, prompt, i32([n]), i32([0, B]), own, lens, out, SCALE, ws, lse=lse)
        if i in (0, 15, 16, 19):
            want, want_lse, *_ = o.prefix_attention(np64(q), np64(kc), np64(vc), prompt.cpu().numpy(), [n], [0, B], own.cpu().numpy(),
                                                    [i + 1] * B, SCALE)
            assert np.abs(np64(out) - want).max() <= 2.0 ** -6 * 4 and np.abs(np64(lse) - want_lse).max() <= 1e-3


def test_the_example_of_the_documentation_runs(kv):
    with open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")) as f:
        code = next(b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "kvarn_prompt_attention" in b)
    B, Hq, Hkv, P, T = 2, 4, 2, 16, 25
    g = torch.Generator(device="cuda").manual_seed(83)
    q_out, out_rows = torch.randn(T, Hq, 128, generator=g, device="cuda").to(BF), torch.zeros(T, Hq, 128, dtype=BF, device="cuda")
    k_cache, v_cache = (torch.randn(8, Hkv, P, 128, generator=g, device="cuda").to(BF) for _ in range(2))
    k_rows, v_rows = (torch.randn(T, Hkv, 128, generator=g, device="cuda").to(BF) for _ in range(2))
    k8, v8 = (torch.zeros(8, Hkv, P, 128, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    ke, ve = (torch.zeros(8, Hkv, P, dtype=torch.int8, device="cuda") for _ in range(2))
    names = dict(kv=kv, torch=torch, B=B, Hq=Hq, Hkv=Hkv, T=T, q_out=q_out, out_rows=out_rows, k_cache=k_cache, v_cache=v_cache,
                 page_table=i32([[3, 0], [1, 2]]), cu_tokens=i32([0, 20, 25]), lens=i32([20, 30]), q_last=q_out[[19, 24]],
                 prefix_table=i32([[5, 6, 7]]), prefix_lens=i32([41]), cu_seqs=i32([0, 2]),
                 out=torch.zeros(B, Hq, 128, dtype=BF, device="cuda"), k_rows=k_rows, v_rows=v_rows, k8=k8, v8=v8, ke=ke, ve=ve,
                 slots=i32([(3, 0)[i // P] * P + i % P for i in range(20)] + [P * 2 + 9 + i for i in range(5)]))
    parts = code.partition("# k8, v8")
    exec(compile(parts[0], "README.md", "exec"), names)
    torch.cuda.synchronize()
    prefix_out = np64(names["out"])
    exec(compile(parts[1] + parts[2], "README.md", "exec"), names)
    torch.cuda.synchronize()
    table, lens = names["page_table"].cpu().numpy(), [20, 30]
    want, _, mass = o.prompt_attention(np64(q_out), np64(k_cache), np64(v_cache), table, [0, 20, 25], lens, SCALE)[:3]
    # probabilities and the output rounded once each to bf16, and 2^-8 for all that is fp32
    assert np.all(np.abs(np64(out_rows) - want) <= 2.0 ** -8 * (2 * mass + np.abs(want)))
    want, _, mass = o.prefix_attention(np64(names["q_last"]), np64(k_cache), np64(v_cache), names["prefix_table"].cpu().numpy(), [41], [0, 2],
                                       table, lens, SCALE)[:3]
    assert np.all(np.abs(prefix_out - want) <= 2.0 ** -8 * (2 * mass + np.abs(want)))
    codes = [np64(c.float()) * 2.0 ** np64(e.float())[..., None] for c, e in ((k8, ke), (v8, ve))]
    want, _, mass = o.paged_attention(np64(names["q_last"]), *codes, table, lens, SCALE)[:3]
    assert np.all(np.abs(np64(names["out"]) - want) <= 2.0 ** -8 * (mass + np.abs(want)))
