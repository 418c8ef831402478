"""Host-side refusals of the calls with many queries and with 8-bit caches: documented status, nothing touched, no GPU
needed."""
import math

import pytest

from tests.test_abi import FAKE, lib  # noqa: F401  (fixture)

INV, UNSUPPORTED, WS = 1, 2, 4


def _prompt(lib, dt=0, B=2, T=6, hq=4, hkv=2, q=FAKE, qs=(512, 128), kc=FAKE, vc=FAKE, pages=4, page=16, cs=(4096, 2048, 128),
            table=FAKE, width=4, cu=FAKE, lens=FAKE, starts=None, causal=1, window=0, scale=0.1, cap=0.0, slopes=None, ws=FAKE,
            ws_bytes=1 << 30, out=FAKE, lse=None):
    return lib.kvarn_prompt_attention(dt, B, T, hq, hkv, q, *qs, kc, vc, pages, page, *cs, table, width, cu, lens, starts, causal,
                                      window, scale, cap, slopes, ws, ws_bytes, out, lse, None)


def test_prompt_attention_refusals(lib):
    assert _prompt(lib, B=0) == 0 and _prompt(lib, T=0) == 0
    for bad in (dict(dt=2), dict(dt=5), dict(B=-1), dict(B=16385), dict(T=-1), dict(hq=5), dict(hkv=0), dict(hq=65536, hkv=1),
                dict(T=1 << 30, hq=4, hkv=1), dict(scale=math.nan), dict(scale=math.inf), dict(cap=-1.0), dict(cap=math.inf),
                dict(cap=1e-40), dict(window=-1), dict(causal=2), dict(causal=0, window=3), dict(causal=0, slopes=FAKE), dict(page=8),
                dict(page=24), dict(page=0), dict(width=0), dict(width=1 << 27), dict(pages=0), dict(q=None), dict(q=FAKE + 8),
                dict(qs=(508, 128)), dict(qs=(512, -128)), dict(kc=None), dict(vc=FAKE + 8), dict(cs=(4096, 2048, 120)),
                dict(cs=(2048, 4096, 128), pages=3), dict(table=None), dict(table=FAKE + 1), dict(cu=None), dict(cu=FAKE + 2),
                dict(lens=None), dict(starts=FAKE + 2), dict(slopes=FAKE + 2), dict(out=None), dict(out=FAKE + 8), dict(lse=FAKE + 2),
                dict(ws=None), dict(ws=FAKE + 8)):
        assert _prompt(lib, **bad) == INV, bad
    assert _prompt(lib, cs=(1 << 39, 2048, 128)) == UNSUPPORTED
    assert _prompt(lib, ws_bytes=64) == WS
    assert b"workspace" in lib.kvarn_last_error()


def test_prompt_attention_workspace_size(lib):
    import bit_kv_cache_kvarn_gb300 as kv

    assert kv.kvarn_prompt_attention_workspace_size(4, 5, 2) == 0 and kv.kvarn_prompt_attention_workspace_size(-1, 4, 2) == 0
    # grows with the rows up to a unit's 256, not beyond
    sizes = [kv.kvarn_prompt_attention_workspace_size(t, 8, 2) for t in (0, 1, 2, 10, 64, 65, 100000)]
    assert sizes == sorted(sizes) and sizes[4] == sizes[5] == sizes[6] and all(s % 256 == 0 for s in sizes)


def _prefix(lib, dt=0, B=4, G=2, hq=4, hkv=2, q=FAKE, qs=(512, 128), kc=FAKE, vc=FAKE, pages=4, page=16, cs=(4096, 2048, 128),
            ptable=FAKE, pwidth=4, plens=FAKE, cu=FAKE, table=FAKE, width=4, lens=FAKE, scale=0.1, cap=0.0, ws=FAKE,
            ws_bytes=1 << 30, out=FAKE, lse=None):
    return lib.kvarn_prefix_attention(dt, B, G, hq, hkv, q, *qs, kc, vc, pages, page, *cs, ptable, pwidth, plens, cu, table, width,
                                      lens, scale, cap, ws, ws_bytes, out, lse, None)


def test_prefix_attention_refusals(lib):
    assert _prefix(lib, B=0) == 0
    for bad in (dict(dt=2), dict(B=-1), dict(B=16385), dict(G=-1), dict(G=16385), dict(hq=5), dict(hkv=0), dict(scale=math.nan),
                dict(cap=-1.0), dict(cap=1e-40), dict(page=8), dict(page=24), dict(pwidth=0), dict(width=0), dict(pwidth=1 << 27),
                dict(width=1 << 27), dict(pages=0), dict(q=None), dict(q=FAKE + 8), dict(qs=(508, 128)), dict(kc=None),
                dict(vc=FAKE + 8), dict(cs=(4096, 2048, 120)), dict(ptable=None), dict(plens=None), dict(cu=None), dict(cu=FAKE + 2),
                dict(table=None), dict(lens=None), dict(out=None), dict(out=FAKE + 8), dict(lse=FAKE + 2), dict(ws=None),
                dict(ws=FAKE + 8)):
        assert _prefix(lib, **bad) == INV, bad
    assert _prefix(lib, cs=(1 << 39, 2048, 128)) == UNSUPPORTED
    assert _prefix(lib, ws_bytes=64) == WS


def test_prefix_attention_workspace_size(lib):
    import bit_kv_cache_kvarn_gb300 as kv

    assert kv.kvarn_prefix_attention_workspace_size(4, 5, 2) == 0 and kv.kvarn_prefix_attention_workspace_size(16385, 4, 2) == 0
    sizes = [kv.kvarn_prefix_attention_workspace_size(b, 8, 2) for b in (1, 2, 64, 200)]
    assert sizes == sorted(sizes) and sizes[0] > 0


def _quantize(lib, xt=0, T=4, hkv=2, k=FAKE, v=FAKE, kvs=(256, 128), kc=FAKE, vc=FAKE + 65536, pages=4, page=16,
              cs=(4096, 2048, 128), ke=FAKE, ve=FAKE + 4096, slots=FAKE):
    return lib.kvarn_quantize_kv(xt, T, hkv, k, v, *kvs, kc, vc, pages, page, *cs, ke, ve, slots, None)


def test_quantize_refusals(lib):
    assert _quantize(lib, T=0) == 0
    for bad in (dict(xt=3), dict(xt=-1), dict(T=-1), dict(hkv=0), dict(hkv=65536), dict(k=None), dict(v=FAKE + 8), dict(kvs=(4, 128)),
                dict(kvs=(-256, 128)), dict(kc=None), dict(vc=FAKE), dict(vc=FAKE + 65544), dict(pages=0), dict(page=0),
                dict(pages=1 << 28), dict(cs=(4096, 2048, 120)), dict(cs=(4096, 2048, 136)), dict(cs=(2048, 2048, 128)),
                dict(cs=(4104, 2048, 128)), dict(ke=None), dict(ve=None), dict(ve=FAKE), dict(slots=FAKE + 2), dict(slots=None, T=65),
                dict(T=1 << 30, hkv=2)):
        assert _quantize(lib, **bad) == INV, bad


def _q8(lib, dt=0, B=2, hq=4, hkv=2, q=FAKE, qs=(512, 128), kc=FAKE, vc=FAKE, ke=FAKE, ve=FAKE, pages=4, page=16,
        cs=(4096, 2048, 128), table=FAKE, width=4, lens=FAKE, starts=None, window=0, scale=0.1, cap=0.0, slopes=None, ws=FAKE,
        ws_bytes=1 << 30, ot=2, out=FAKE, lse=None):
    return lib.kvarn_paged_attention_q8(dt, B, hq, hkv, q, *qs, kc, vc, ke, ve, pages, page, *cs, table, width, lens, starts, window,
                                        scale, cap, slopes, ws, ws_bytes, ot, out, lse, None)


def test_paged_attention_q8_refusals(lib):
    assert _q8(lib, B=0) == 0
    for bad in (dict(dt=2), dict(ot=1), dict(ot=3), dict(B=-1), dict(B=65536), dict(hq=5), dict(hkv=0), dict(scale=math.nan),
                dict(cap=-1.0), dict(cap=1e-40), dict(window=-1), dict(page=8), dict(page=24), dict(width=0), dict(width=1 << 27),
                dict(pages=0), dict(q=None), dict(q=FAKE + 8), dict(qs=(508, 128)), dict(kc=None), dict(vc=FAKE + 8), dict(ke=None),
                dict(ve=FAKE + 8), dict(cs=(4096, 2048, 120)), dict(cs=(4096, 2048, 136)), dict(cs=(4104, 2048, 128)),
                dict(table=None), dict(lens=None), dict(starts=FAKE + 2), dict(slopes=FAKE + 2), dict(out=None), dict(out=FAKE + 8),
                dict(lse=FAKE + 2), dict(ws=None), dict(ws=FAKE + 8)):
        assert _q8(lib, **bad) == INV, bad
    assert _q8(lib, ws_bytes=64) == WS


def test_python_calls_refuse_what_is_no_device_tensor(lib):
    import torch

    import bit_kv_cache_kvarn_gb300 as kv

    t, i = torch.zeros(2, 1, 128, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int32)
    c, c8 = (torch.zeros(4, 1, 16, 128, dtype=d) for d in (torch.bfloat16, torch.float8_e4m3fn))
    e, table = torch.zeros(4, 1, 16, dtype=torch.int8), torch.zeros(2, 2, dtype=torch.int32)
    for call in (lambda: kv.kvarn_prompt_attention(t, c, c, table, i, i, t, 0.1, i),
                 lambda: kv.kvarn_prefix_attention(t, c, c, table, i, i, table, i, t, 0.1, i),
                 lambda: kv.kvarn_quantize_kv(t, t, c8, c8, e, e),
                 lambda: kv.kvarn_paged_attention_q8(t, c8, c8, e, e, table, i, t, 0.1, i)):
        with pytest.raises((ValueError, RuntimeError)):
            call()
