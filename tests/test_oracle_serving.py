"""The serving oracle against independent statements of the same mathematics (CPU)."""
import math

import numpy as np
import pytest
import torch

from oracle import serving as o


def test_plain_frequencies_and_linear_and_ntk():
    f, s = o.rope_frequencies(64, base=1e4)
    assert s == 1.0 and np.allclose(f, 1e4 ** (-np.arange(32) / 32.0), rtol=1e-14)
    g, _ = o.rope_frequencies(64, base=1e4, scaling="linear", factor=4.0)
    assert np.allclose(g, f / 4, rtol=1e-15)
    # ntk leaves the fastest pair and slows the slowest one by exactly the factor
    g, _ = o.rope_frequencies(64, base=1e4, scaling="ntk", factor=4.0)
    assert g[0] == 1.0 and math.isclose(g[-1], f[-1] / 4, rel_tol=1e-12)


def test_band_and_yarn_frequencies_keep_fast_pairs_and_stretch_slow_ones():
    f, _ = o.rope_frequencies(128, base=5e5)
    turns = 8192 * f / (2 * math.pi)
    g, s = o.rope_frequencies(128, base=5e5, scaling="bands", factor=8.0, original_len=8192, low=1.0, high=4.0)
    assert s == 1.0
    assert np.array_equal(g[turns > 4], f[turns > 4]) and np.allclose(g[turns < 1], f[turns < 1] / 8, rtol=1e-15)
    mid = (turns >= 1) & (turns <= 4)
    assert mid.any() and np.all(g[mid] <= f[mid]) and np.all(g[mid] >= f[mid] / 8)
    g, s = o.rope_frequencies(128, base=5e5, scaling="yarn", factor=8.0, original_len=8192, low=1.0, high=32.0)
    assert math.isclose(s, 0.1 * math.log(8) + 1)
    assert np.array_equal(g[turns > 40], f[turns > 40]) and np.allclose(g[turns < 0.8], f[turns < 0.8] / 8, rtol=1e-12)
    assert np.all(np.diff(g) < 0)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_pair_norms_and_scores_depend_on_distance(interleaved):
    rng = np.random.default_rng(0)
    freqs, _ = o.rope_frequencies(96)
    q, k = rng.standard_normal((1, 1, 128)), rng.standard_normal((1, 1, 128))

    def dot(a, b):
        return float((o.norm_rotate(q, [a], freqs, interleaved=interleaved)
                      * o.norm_rotate(k, [b], freqs, interleaved=interleaved)).sum())

    assert math.isclose(dot(5, 3), dot(1005, 1003), rel_tol=1e-9)
    y = o.norm_rotate(q, [77], freqs, interleaved=interleaved)
    assert np.array_equal(y[..., 96:], q[..., 96:])
    assert math.isclose(float((y ** 2).sum()), float((q ** 2).sum()), rel_tol=1e-12)
    w = rng.standard_normal(128)
    n = o.norm_rotate(q, [0], freqs, w=w, eps=0.0)
    assert np.allclose(n, torch.nn.functional.rms_norm(torch.tensor(q), (128,), torch.tensor(w), eps=0.0).numpy())


def test_tables_by_hand():
    # pages of 4: sequence 0 goes 3 -> 5 tokens (one page more), 1 is finished (gives pages 7, 8), 2
    # starts with 5 tokens (two pages), 3 idles
    table = np.array([[2, -1, -1], [7, 8, -1], [-1, -1, -1], [5, -1, -1]], dtype=np.int32)
    free = np.array([10, 11, -9, -9, -9], dtype=np.int32)
    r = o.step_tables(np.array([3, 6, 0, 2], np.int32), np.array([2, -1, 5, 0], np.int32),
                      np.array([1, 2, 0, 1], np.int32), table, free, 2, 4, 9,
                      block_table=np.full((4, 2, 3), -1, np.int32))
    assert r["status"] == 0 and r["free_count"] == 1
    assert r["page_table"].tolist() == [[2, 8, -1], [7, 8, -1], [7, 11, -1], [5, -1, -1]]
    assert r["kv_lens"].tolist() == [5, 0, 5, 2] and r["page_counts"].tolist() == [2, 0, 2, 1]
    assert r["cu_tokens"].tolist() == [0, 2, 2, 7, 7]
    assert r["positions"].tolist() == [3, 4, 0, 1, 2, 3, 4, -1, -1]
    assert r["slot_map"].tolist() == [11, 32, 28, 29, 30, 31, 44, -1, -1]
    assert r["free_pages"].tolist() == free.tolist()
    assert r["block_table"][0].tolist() == [[-1, 16, -1], [-1, 17, -1]]
    r = o.step_tables(np.array([3], np.int32), np.array([10], np.int32), np.array([1], np.int32), table[:1], free, 1, 4, 3)
    assert r["status"] == o.NO_PAGES | o.ROW_FULL | o.ROWS and r["page_table"].tolist() == table[:1].tolist()


def test_paged_attention_is_softmax_attention():
    rng = np.random.default_rng(1)
    B, hq, hkv, P, n_pages = 3, 6, 2, 16, 20
    q = rng.standard_normal((B, hq, 128))
    k, v = rng.standard_normal((n_pages, hkv, P, 128)), rng.standard_normal((n_pages, hkv, P, 128))
    table = rng.permutation(n_pages)[:B * 6].reshape(B, 6).astype(np.int32)
    lens, starts = [0, 40, 96], [0, 7, 3]
    slopes = rng.random(hq)
    out, lse, _, _ = o.paged_attention(q, k, v, table, lens, 0.09, softcap=5.0, slopes=slopes, window=60, kv_starts=starts)
    assert not out[0].any() and np.all(np.isneginf(lse[0]))
    for b in (1, 2):
        kk = torch.tensor(k[table[b]]).transpose(0, 1).reshape(hkv, -1, 128).repeat_interleave(3, 0)
        vv = torch.tensor(v[table[b]]).transpose(0, 1).reshape(hkv, -1, 128).repeat_interleave(3, 0)
        s = torch.einsum("hd,hld->hl", torch.tensor(q[b]), kk) * 0.09
        s = 5.0 * torch.tanh(s / 5.0)
        j = torch.arange(s.shape[1])
        s = s + torch.tensor(slopes)[:, None] * (j - (lens[b] - 1))
        s[:, (j >= lens[b]) | (j < starts[b]) | (j < lens[b] - 60)] = -math.inf
        assert np.allclose(out[b], torch.einsum("hl,hld->hd", torch.softmax(s, -1), vv).numpy(), rtol=1e-10)
        assert np.allclose(lse[b], torch.logsumexp(s, -1).numpy(), rtol=1e-12)
