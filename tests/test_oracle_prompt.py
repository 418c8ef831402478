"""Pins of the oracle's prompt, prefix and 8-bit functions (CPU)."""
import numpy as np
import pytest
import torch

from oracle import serving as o


def dense(rng, n, hkv, P=16):
    pages = -(-n // P)
    k, v = rng.standard_normal((2, pages, hkv, P, 128))
    return k, v, np.arange(pages, dtype=np.int32)[None]


def test_prompt_attention_is_causal_attention():
    rng = np.random.default_rng(0)
    n, hq, hkv = 40, 4, 2
    k, v, table = dense(rng, n, hkv)
    q = rng.standard_normal((n, hq, 128))
    out, lse, *_ = o.prompt_attention(q, k, v, table, [0, n], [n], 0.1)
    flat = [torch.tensor(x.transpose(1, 0, 2, 3).reshape(hkv, -1, 128)[:, :n]).repeat_interleave(hq // hkv, 0) for x in (k, v)]
    want = torch.nn.functional.scaled_dot_product_attention(torch.tensor(q).transpose(0, 1), *flat, is_causal=True, scale=0.1)
    assert np.allclose(out, want.transpose(0, 1).numpy(), atol=1e-13)


@pytest.mark.parametrize("kw", [dict(), dict(softcap=3.0), dict(window=5), dict(kv_starts=[4])])
def test_prompt_attention_of_single_tokens_is_the_decode_attention(kw):
    rng = np.random.default_rng(1)
    k, v, table = dense(rng, 30, 2)
    q = rng.standard_normal((1, 4, 128))
    a = o.prompt_attention(q, k, v, table, [0, 1], [30], 0.2, **kw)
    b = o.paged_attention(q, k, v, table, [30], 0.2, **kw)
    assert np.allclose(a[0], b[0], atol=1e-13) and np.allclose(a[1], b[1], atol=1e-13)


def test_prefix_attention_is_attention_over_both_parts():
    rng = np.random.default_rng(2)
    k, v, table = dense(rng, 48, 2)
    q = rng.standard_normal((1, 4, 128))
    a = o.prefix_attention(q, k, v, table[:, :2], [32], [0, 1], table[:, 2:], [9], 0.2)
    b = o.paged_attention(q, k, v, table, [41], 0.2)
    assert np.allclose(a[0], b[0], atol=1e-13) and np.allclose(a[1], b[1], atol=1e-13)


def test_e4m3_grid_is_torchs():
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(o.e4m3_grid(), codes)


def test_quantize_row_against_torchs_cast():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((200, 128)) * np.exp(4 * rng.standard_normal((200, 1)))
    x[0], x[1, 0] = 0.0, 448.0 * 2.0 ** 9
    x = x.astype(np.float32).astype(np.float64)
    code, e = o.quantize_row(x)
    top = np.abs(x).max(-1)
    assert e[0] == -127 and np.all(top[1:] <= 448 * 2.0 ** e[1:]) and np.all(top[1:] > 448 * 2.0 ** (e[1:] - 1.0))
    cast = torch.tensor(x / 2.0 ** e[:, None].astype(float), dtype=torch.float32).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(code, cast)
    # each value is off by half a step at most
    y = x / 2.0 ** e[:, None].astype(float)
    assert np.all(np.abs(code - y) <= np.maximum(np.abs(y) * 2.0 ** -4, 2.0 ** -10))
