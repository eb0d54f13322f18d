"""Oracle of the serving operators around the paged cache (fp64 numpy, test infrastructure only):
page tables of a step, rotary positions, and attention with score options.

Each function states its definition once, sequentially, and shares no code with the product.
"""
from __future__ import annotations

import math

import numpy as np

from . import as_f64, gather_keys, kv_head_of

__all__ = ["step_plan", "release", "rope_rows", "visible", "attend_scored", "decode_scored",
           "prefill_scored", "rope_frequencies"]


def step_plan(cached, new, table, free, count, num_pages, total_rows, page_size=16):
    """Returns dict(cu, seq_lens, positions, slots, table, count, flags) of one step; flags is a
    set of 'length', 'no_pages', 'page'."""
    P, table = page_size, np.array(table, copy=True)
    B, cap = len(cached), table.shape[1] * P
    flags = set()
    if not 0 <= count <= len(free):
        flags.add("length")
        count = min(max(count, 0), len(free))
    cu, seq_lens = [0], []
    positions = np.zeros(total_rows, np.int32)
    slots = np.full(total_rows, -1, np.int64)
    asked = used = 0
    for b in range(B):
        c, n = int(cached[b]), int(new[b])
        ok = c >= 0 and n >= 0 and c + n <= cap
        if not ok:
            flags.add("length")
        else:
            held, need = -(-c // P), -(-(c + n) // P) - -(-c // P)
            asked += need
            if need and asked > count:
                flags.add("no_pages")
                ok = False
        n = max(n, 0)
        if ok:
            for k in range(need):
                table[b, held + k] = free[count - 1 - used]
                used += 1
                if not 0 <= table[b, held + k] < num_pages:
                    flags.add("page")
            for j in range(n):
                t, p = cu[-1] + j, c + j
                if t < total_rows:
                    page = int(table[b, p // P])
                    positions[t] = p
                    if 0 <= page < num_pages:
                        slots[t] = page * P + p % P
                    else:
                        flags.add("page")
        seq_lens.append(c + n if ok else min(max(c, 0), cap))
        cu.append(cu[-1] + n)
    if cu[-1] > total_rows:
        flags.add("length")
    return dict(cu=np.array(cu), seq_lens=np.array(seq_lens, dtype=np.int64), positions=positions,
                slots=slots, table=table, count=count - used, flags=flags)


def release(begin, end, table, free, count, num_pages):
    """Returns (table, free, count, flags)."""
    table, free = np.array(table, copy=True), np.array(free, copy=True)
    before_t, before_f, before_c = table.copy(), free.copy(), count
    flags, pages = set(), []
    for b in range(len(begin)):
        lo, hi = int(begin[b]), int(end[b])
        if lo < 0 or hi > table.shape[1]:
            flags.add("length")
            lo, hi = max(lo, 0), min(hi, table.shape[1])
        for i in range(lo, hi):
            e = int(table[b, i])
            if 0 <= e < num_pages:
                pages.append(e)
            elif e >= num_pages:
                flags.add("page")
            table[b, i] = -1
    if count + len(pages) > len(free):
        return before_t, before_f, before_c, flags | {"length"}
    free[count:count + len(pages)] = pages
    return table, free, count + len(pages), flags


def rope_rows(x, positions, inv_freq, interleaved, factor=1.0, gamma=None, eps=1e-6):
    """x [T, H, D] -> rotated (and normalised) rows in fp64. The fp64 product position * inv_freq
    carries an angle error of position * inv_freq * 2^-53 (2^-22 rad at 2^31)."""
    x = as_f64(x)
    if gamma is not None:
        x = x / np.sqrt((x * x).mean(axis=-1, keepdims=True) + eps) * np.asarray(gamma, np.float64)
    y = x.copy()
    half = len(inv_freq)
    for t, p in enumerate(positions):
        for i, f in enumerate(inv_freq):
            a = int(p) * float(f)
            c, s = factor * math.cos(a), factor * math.sin(a)
            u, w = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
            y[t, :, u] = x[t, :, u] * c - x[t, :, w] * s
            y[t, :, w] = x[t, :, w] * c + x[t, :, u] * s
    return y


def visible(i, L, prefix=0, row_start=0, window=0):
    """Boolean [L]: the keys that the row at position i of a sequence of L keys sees."""
    j = np.arange(L)
    own = (j <= i) & (j >= row_start)
    if window > 0:
        own &= i - j < window
    return own | (j < prefix)


def attend_scored(q, K, V, i, vis, scale, softcap=0.0, slope=0.0):
    """One row: (o, lse) over its visible keys; (0, -inf) when none carries weight."""
    idx = np.flatnonzero(vis)
    if len(idx) == 0:
        return np.zeros(V.shape[1]), -math.inf
    s = scale * (K[idx] @ as_f64(q))
    if softcap:
        s = softcap * np.tanh(s / softcap)
    s = s - slope * np.abs(i - idx)
    m = s.max()
    if m == -math.inf:
        return np.zeros(V.shape[1]), -math.inf
    e = np.exp(s - m)
    return (e @ V[idx]) / e.sum(), m + math.log(e.sum())


def _opts(o, b, row):
    return dict(prefix=0 if o.get("prefix") is None else int(o["prefix"][b]),
                row_start=0 if o.get("row_start") is None else int(o["row_start"][row]),
                window=int(o.get("window", 0)))


def prefill_scored(q, cu, k_pool, v_pool, table, seq_lens, scale, *, rows=None, **o):
    """q [T, Hq, D] packed by cu; options softcap, slopes [Hq], window, prefix [B], row_start [T].
    Returns fp64 (o, lse); rows limits the work (other rows NaN)."""
    T, Hq, D = q.shape
    Hkv = k_pool.shape[2]
    out, lse = np.full((T, Hq, D), np.nan), np.full((T, Hq), np.nan)
    slopes = o.get("slopes")
    for b in range(len(cu) - 1):
        n, L = int(cu[b + 1] - cu[b]), int(seq_lens[b])
        mine = [r for r in range(int(cu[b]), int(cu[b + 1])) if rows is None or r in rows]
        if not mine:
            continue
        for g in range(Hkv):
            K, V = gather_keys(k_pool, table[b], L, g), gather_keys(v_pool, table[b], L, g)
            for r in mine:
                i = L - n + r - int(cu[b])
                vis = visible(i, L, **_opts(o, b, r))
                for h in range(Hq):
                    if kv_head_of(h, Hq, Hkv) == g:
                        out[r, h], lse[r, h] = attend_scored(
                            q[r, h], K, V, i, vis, scale, o.get("softcap", 0.0),
                            0.0 if slopes is None else float(slopes[h]))
    return out, lse


def decode_scored(q, k_pool, v_pool, table, seq_lens, scale, *, rows=None, **o):
    """One query row per sequence, at its last position."""
    B = len(seq_lens)
    return prefill_scored(q, np.arange(B + 1), k_pool, v_pool, table, seq_lens, scale, rows=rows, **o)


def rope_frequencies(rot_dim, theta, kind="none", factor=1.0, original=32768, low_freq_factor=1.0,
                     high_freq_factor=4.0, beta_fast=32.0, beta_slow=1.0, attn_factor=0.0):
    """(frequencies [rot_dim / 2], factor of cos and sin), pair by pair from the definitions of the
    stretchings: by wavelength (llama3), by rotations over the original context (yarn)."""
    freqs, scale = [], 1.0
    if kind == "yarn":
        # the pair index (a real number) whose wavelength fits `turns` times into the original context
        pair = lambda turns: rot_dim / 2 * math.log(original / (2 * math.pi * turns)) / math.log(theta)
        first, last = max(0, math.floor(pair(beta_fast))), min(rot_dim - 1, math.ceil(pair(beta_slow)))
        scale = attn_factor if attn_factor > 0 else 1.0 + 0.1 * math.log(max(factor, 1.0))
    for i in range(rot_dim // 2):
        f = theta ** (-2.0 * i / rot_dim)
        if kind == "linear":
            f = f / factor
        elif kind == "ntk":
            f = (theta * factor ** (rot_dim / (rot_dim - 2))) ** (-2.0 * i / rot_dim)
        elif kind == "llama3":
            wavelength = 2 * math.pi / f
            if wavelength > original / low_freq_factor:
                f = f / factor
            elif wavelength >= original / high_freq_factor:
                kept = (original / wavelength - low_freq_factor) / (high_freq_factor - low_freq_factor)
                f = (1 - kept) * f / factor + kept * f
        elif kind == "yarn":
            if i >= last:
                f = f / factor
            elif i > first:
                divided = (i - first) / (last - first)
                f = divided * f / factor + (1 - divided) * f
        freqs.append(f)
    return np.array(freqs), scale
