"""fp64 CPU oracle of the serving step: rotation frequencies, norm + rotation + cache write, page tables,
and attention of one query over a paged cache.  Plain loops over the definitions."""
from __future__ import annotations

import math
from fractions import Fraction

import numpy as np


def rope_frequencies(rot_dim, base=10000.0, scaling="plain", factor=1.0, original_len=0.0, low=1.0, high=4.0):
    """(frequencies [rot_dim / 2], factor of cos and sin)."""
    if scaling == "ntk":
        base = base * factor ** (rot_dim / (rot_dim - 2))
    freqs, scale = [], 1.0
    for i in range(rot_dim // 2):
        f = base ** (-2 * i / rot_dim)
        if scaling == "linear":
            f /= factor
        elif scaling == "bands":
            turns = original_len * f / (2 * math.pi)
            if turns < low:
                f /= factor
            elif turns <= high:
                share = (turns - low) / (high - low)
                f = share * f + (1 - share) * f / factor
        elif scaling == "yarn":
            def pair(t):
                return rot_dim * math.log(original_len / (2 * math.pi * t)) / (2 * math.log(base))
            a, b = max(math.floor(pair(high)), 0), min(math.ceil(pair(low)), rot_dim - 1)
            if b <= a:
                b = a + 0.001
            stretch = min(max((i - a) / (b - a), 0.0), 1.0)
            f = (1 - stretch) * f + stretch * f / factor
        freqs.append(f)
    if scaling == "yarn":
        scale = 0.1 * math.log(factor) + 1
    return np.array(freqs), scale


def _angles(positions, f):
    """position * f modulo a turn, exactly: f as a fraction of integers, pi to 60 digits."""
    turn = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494")
    return np.array([float(Fraction(f) * int(p) % turn) for p in positions])


def norm_rotate(x, positions, freqs, w=None, eps=1e-6, scale=1.0, interleaved=False):
    """x [T, H, 128] fp64 -> the normed and rotated rows."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    if w is not None:
        y = y / np.sqrt((y * y).mean(axis=-1, keepdims=True) + eps) * np.asarray(w, dtype=np.float64)
    out = y.copy()
    half = len(freqs)
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        t = _angles(positions, float(freqs[i]))
        c, s = (scale * np.cos(t))[:, None], (scale * np.sin(t))[:, None]
        out[:, :, a] = y[:, :, a] * c - y[:, :, b] * s
        out[:, :, b] = y[:, :, b] * c + y[:, :, a] * s
    return out


NO_PAGES, ROW_FULL, ROWS, FREE_FULL, INVALID = 1, 2, 4, 8, 16


def step_tables(seq_lens, n_new, page_counts, page_table, free_pages, free_count, page_size, n_rows, block_table=None):
    """Returns a dict of the outputs; the inputs are not modified."""
    B, width = page_table.shape
    table, free = page_table.copy(), free_pages.copy()
    blocks = None if block_table is None else block_table.copy()
    out = dict(kv_lens=seq_lens.copy(), page_counts=page_counts.copy(), free_count=free_count,
               cu_tokens=np.zeros(B + 1, dtype=np.int32), positions=np.full(n_rows, -1, dtype=np.int32),
               slot_map=np.full(n_rows, -1, dtype=np.int32), page_table=table, free_pages=free, block_table=blocks,
               status=0)
    status = 0
    if not 0 <= free_count <= len(free):
        status |= INVALID
    fresh, given = [0] * B, [0] * B
    total = 0
    for b in range(B):
        length, new, held = int(seq_lens[b]), int(n_new[b]), int(page_counts[b])
        if length < 0 or not 0 <= held <= width:
            status |= INVALID
            continue
        if new < 0:
            given[b] = held
            continue
        total += new
        need = -(-(length + new) // page_size)
        if length + new > 2 ** 31 - 1:
            status |= INVALID
        if need > width:
            status |= ROW_FULL
        fresh[b] = max(0, need - held)
    left = free_count + sum(given) - sum(fresh)
    if left < 0:
        status |= NO_PAGES
    if left > len(free):
        status |= FREE_FULL
    if total > n_rows:
        status |= ROWS
    out["status"] = status
    if status:
        return out
    stack = [int(p) for p in free[:free_count]]
    for b in range(B):
        stack += [int(p) for p in page_table[b, :given[b]]]
    row = 0
    for b in range(B):
        out["cu_tokens"][b] = row
        if n_new[b] < 0:
            out["kv_lens"][b] = out["page_counts"][b] = 0
            continue
        held = int(page_counts[b])
        for i in range(held, held + fresh[b]):
            page = stack.pop()
            table[b, i] = page
            if blocks is not None:
                for h in range(blocks.shape[1]):
                    blocks[b, h, i] = page * blocks.shape[1] + h
        out["page_counts"][b] = held + fresh[b]
        for i in range(int(n_new[b])):
            pos = int(seq_lens[b]) + i
            out["positions"][row] = pos
            out["slot_map"][row] = int(table[b, pos // page_size]) * page_size + pos % page_size
            row += 1
        out["kv_lens"][b] = seq_lens[b] + n_new[b]
    out["cu_tokens"][B] = row
    out["free_count"] = len(stack)
    free[free_count:len(stack)] = stack[free_count:]
    return out


def paged_attention(q, k_cache, v_cache, page_table, kv_lens, scale, softcap=0.0, slopes=None, window=0, kv_starts=None):
    """q [B, Hq, 128], caches [pages, Hkv, P, 128] (fp64) -> out, lse and, per row, the bound's terms:
    mass = sum_j p_j |v_j| and reach = scale * max_j sum_c |q_c k_jc| over the visible keys."""
    B, hq, D = q.shape
    n_pages, hkv, P, _ = k_cache.shape
    group = hq // hkv
    out, lse = np.zeros((B, hq, D)), np.full((B, hq), -np.inf)
    mass, reach = np.zeros((B, hq, D)), np.zeros((B, hq))
    for b in range(B):
        L = min(max(int(kv_lens[b]), 0), page_table.shape[1] * P)
        lo = max(int(kv_starts[b]), 0) if kv_starts is not None else 0
        if window:
            lo = max(lo, L - window)
        if lo >= L:
            continue
        pos = np.arange(lo, L)
        pages = page_table[b, pos // P]
        known = (pages >= 0) & (pages < n_pages)
        pages = np.where(known, pages, 0)
        for h in range(hq):
            k = np.where(known[:, None], k_cache[pages, h // group, pos % P], 0.0)
            v = np.where(known[:, None], v_cache[pages, h // group, pos % P], 0.0)
            s = scale * (k @ q[b, h])
            reach[b, h] = abs(scale) * (np.abs(k) @ np.abs(q[b, h])).max()
            if softcap > 0:
                s = softcap * np.tanh(s / softcap)
            if slopes is not None:
                s = s + slopes[h] * (pos - (L - 1))
            m = s.max()
            if m == -np.inf:
                continue
            p = np.exp(s - m)
            out[b, h] = p @ v / p.sum()
            mass[b, h] = p @ np.abs(v) / p.sum()
            lse[b, h] = m + math.log(p.sum())
    return out, lse, mass, reach
