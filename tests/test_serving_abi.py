"""Host-side refusals of the serving-step calls: documented status, nothing touched, no GPU needed."""
import ctypes
import math

import numpy as np
import pytest

from oracle import serving as o
from tests.test_abi import FAKE, lib  # noqa: F401  (fixture)

INV, WS = 1, 4


def _tables(lib, B=2, max_pages=4, page=16, cap=8, rows=4, hkv=0, blocks=None, **null):
    names = ["seq_lens", "n_new", "page_counts", "page_table", "free_pages", "free_count", "kv_lens",
             "page_counts_out", "free_count_out", "cu_tokens", "positions", "slot_map", "status"]
    p = {n: null.get(n, FAKE) for n in names}
    return lib.kvarn_step_tables(B, max_pages, page, p["seq_lens"], p["n_new"], p["page_counts"], p["page_table"],
                                 p["free_pages"], p["free_count"], cap, p["kv_lens"], p["page_counts_out"],
                                 p["free_count_out"], p["cu_tokens"], p["positions"], p["slot_map"], rows, blocks, hkv,
                                 p["status"], None)


def test_step_tables_refusals(lib):
    assert _tables(lib, B=0) == 0
    for bad in (dict(B=-1), dict(B=16385), dict(page=0), dict(page=65537), dict(max_pages=0),
                dict(B=1024, max_pages=1 << 21), dict(rows=-1), dict(rows=(1 << 30) + 1), dict(cap=-1),
                dict(hkv=-1), dict(hkv=2), dict(blocks=FAKE), dict(hkv=1025, blocks=FAKE), dict(hkv=2, blocks=FAKE + 2)):
        assert _tables(lib, **bad) == INV, bad
    for name in ("seq_lens", "n_new", "page_counts", "page_table", "free_pages", "free_count", "kv_lens",
                 "page_counts_out", "free_count_out", "cu_tokens", "positions", "slot_map", "status"):
        assert _tables(lib, **{name: None}) == INV
        assert name.encode() in lib.kvarn_last_error()
        assert _tables(lib, **{name: FAKE + 2}) == INV


def _rope(lib, xt=0, ot=0, T=4, hq=4, hkv=2, q=FAKE, qs=(512, 128), k=FAKE, v=FAKE, kvs=(256, 128), pos=FAKE, freq=FAKE,
          rot=128, inter=0, scale=1.0, qw=None, kw=None, eps=1e-6, qo=FAKE + 4096, qos=(512, 128), kc=FAKE, vc=FAKE + 65536,
          pages=4, page=16, cs=(4096, 2048, 128), slots=FAKE):
    return lib.kvarn_rope_qkv(xt, ot, T, hq, hkv, q, *qs, k, v, *kvs, pos, freq, rot, inter, scale, qw, kw, eps, qo,
                              *qos, kc, vc, pages, page, *cs, slots, None)


def test_rope_refusals(lib):
    assert _rope(lib, T=0) == 0 and _rope(lib, hq=0, hkv=0) == 0
    for bad in (dict(ot=2), dict(xt=1), dict(xt=3), dict(T=-1), dict(hq=-1), dict(hkv=65536), dict(rot=8), dict(rot=144),
                dict(rot=-16), dict(inter=2), dict(scale=math.inf), dict(scale=math.nan), dict(eps=-1.0), dict(eps=math.nan),
                dict(pos=None), dict(freq=None), dict(freq=FAKE + 4), dict(q=None), dict(q=FAKE + 8), dict(qo=None),
                dict(qs=(-512, 128)), dict(qs=(512, 132)), dict(qos=(512, 132)), dict(qos=(128, 128)), dict(qos=(0, 128)),
                dict(k=None), dict(v=FAKE + 2), dict(kvs=(4, 128)), dict(kc=None), dict(vc=FAKE + 8), dict(vc=FAKE), dict(pages=0),
                dict(page=0), dict(pages=1 << 28), dict(cs=(4096, 2048, 64)), dict(cs=(2048, 2048, 128)),
                dict(cs=(0, 2048, 128)), dict(cs=(-4096, 2048, 128)), dict(cs=(4100, 2048, 128)),
                dict(cs=(1 << 41, 2048, 128)), dict(qw=FAKE + 4), dict(kw=FAKE + 8), dict(slots=FAKE + 2),
                dict(slots=None, T=65)):
        assert _rope(lib, **bad) == INV, bad
    # q_out = q only with q's type and strides
    assert _rope(lib, qo=FAKE, qos=(1024, 128)) == INV and _rope(lib, xt=2, qo=FAKE) == INV
    assert b"q_out" in lib.kvarn_last_error()


def test_python_calls_refuse_what_is_no_device_tensor(lib):
    # without a GPU the current device cannot be asked for, with one the tensors are on another device
    import torch

    import bit_kv_cache_kvarn_gb300 as kv

    t, i = torch.zeros(2, 1, 128, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    c = torch.zeros(4, 1, 16, 128, dtype=torch.bfloat16)
    with pytest.raises((ValueError, RuntimeError)):
        kv.kvarn_rope_qkv(t, None, None, i, None, t, None, None)
    with pytest.raises((ValueError, RuntimeError)):
        kv.kvarn_paged_attention(t, c, c, torch.zeros(2, 2, dtype=torch.int32), i, t, 0.1, i)
    with pytest.raises((ValueError, RuntimeError)):
        kv.kvarn_step_tables(i, i, i, torch.zeros(2, 2, dtype=torch.int32), i, i[:1], 16, i, i, i[:1], i, i, i, i[:1])


def _attn(lib, dt=0, B=2, hq=4, hkv=2, q=FAKE, qs=(512, 128), kc=FAKE, vc=FAKE, pages=4, page=16, cs=(4096, 2048, 128),
          table=FAKE, width=4, lens=FAKE, starts=None, window=0, scale=0.1, cap=0.0, slopes=None, ws=FAKE, ws_bytes=1 << 30,
          ot=2, out=FAKE, lse=None):
    return lib.kvarn_paged_attention(dt, B, hq, hkv, q, *qs, kc, vc, pages, page, *cs, table, width, lens, starts, window,
                                     scale, cap, slopes, ws, ws_bytes, ot, out, lse, None)


def test_paged_attention_refusals(lib):
    assert _attn(lib, B=0) == 0
    for bad in (dict(dt=2), dict(dt=5), dict(ot=1), dict(ot=3), dict(B=-1), dict(B=65536), dict(hq=5), dict(hkv=0),
                dict(hq=65536, hkv=1), dict(scale=math.nan), dict(cap=-1.0), dict(cap=math.inf), dict(window=-1),
                dict(page=8), dict(page=24), dict(page=0), dict(width=0), dict(width=1 << 27), dict(pages=0), dict(q=None),
                dict(q=FAKE + 8), dict(qs=(508, 128)), dict(qs=(512, -128)), dict(kc=None), dict(vc=None),
                dict(cs=(4096, 2048, 120)), dict(cs=(2048, 4096, 128), pages=3), dict(table=None), dict(table=FAKE + 1),
                dict(lens=None), dict(starts=FAKE + 2), dict(slopes=FAKE + 2), dict(out=None), dict(out=FAKE + 8),
                dict(lse=FAKE + 2), dict(ws=None), dict(ws=FAKE + 8)):
        assert _attn(lib, **bad) == INV, bad
    assert _attn(lib, ws_bytes=64) == WS
    assert b"workspace" in lib.kvarn_last_error()


def test_paged_attention_refuses_caps_without_a_reciprocal(lib):
    for cap in (2.0 ** -149, 1e-40, 2.0 ** -126 - 2.0 ** -149, -(2.0 ** -149)):
        assert _attn(lib, cap=cap) == INV, cap
        assert b"softcap" in lib.kvarn_last_error()


def test_paged_attention_workspace_size(lib):
    import bit_kv_cache_kvarn_gb300 as kv

    assert kv.kvarn_paged_attention_workspace_size(1, 5, 2) == 0
    assert kv.kvarn_paged_attention_workspace_size(-1, 4, 2) == 0
    # grows with the query heads per kv head, up to 16 of them; not with the lengths or the batch
    sizes = [kv.kvarn_paged_attention_workspace_size(1, g, 1) for g in (1, 2, 4, 8, 16, 17, 64)]
    assert sizes == sorted(sizes) and sizes[4] == sizes[5] == sizes[6] and all(s % 256 == 0 for s in sizes)
    assert kv.kvarn_paged_attention_workspace_size(300, 32, 8) == kv.kvarn_paged_attention_workspace_size(1, 4, 1)


@pytest.mark.parametrize("name,code", [("plain", 0), ("linear", 1), ("ntk", 2), ("bands", 3), ("yarn", 4)])
@pytest.mark.parametrize("rot", [16, 64, 96, 128])
def test_rope_frequencies_against_the_oracle(lib, name, code, rot):
    import bit_kv_cache_kvarn_gb300 as kv

    for base, factor, length, low, high in ((1e4, 4.0, 4096, 1.0, 32.0), (5e5, 8.0, 8192, 1.0, 4.0), (1e6, 1.0, 100, 0.5, 2.0)):
        got, scale = kv.kvarn_rope_frequencies(rot, base, code, factor, length, low, high)
        want, want_scale = o.rope_frequencies(rot, base, name, factor, length, low, high)
        # pow and log are each within an ulp or so of exact, at exponents up to about 16
        assert np.allclose(got.numpy(), want, rtol=64 * 2.0 ** -53, atol=0) and math.isclose(scale, want_scale, rel_tol=2.0 ** -23)


def test_rope_frequencies_refusals(lib):
    import bit_kv_cache_kvarn_gb300 as kv

    for bad in (dict(rot_dim=8), dict(rot_dim=136), dict(rot_dim=0), dict(base=1.0), dict(base=math.inf), dict(scaling=5),
                dict(scaling=-1), dict(scaling=1, factor=0.5), dict(scaling=3, factor=2.0),
                dict(scaling=4, factor=2.0, original_len=100.0, low=4.0, high=4.0), dict(scaling=2, factor=math.nan)):
        with pytest.raises(kv.KvarnError):
            kv.kvarn_rope_frequencies(**bad)
    out = (ctypes.c_double * 64)()
    assert lib.kvarn_rope_frequencies(None, out, ctypes.byref(ctypes.c_float())) == INV
