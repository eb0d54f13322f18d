"""Oracle of the operators of a beam-search step over the paged cache (fp64 numpy, test infrastructure
only): the selection over beams and vocabulary, the fork of page tables, the page copies. (Attention
over shared pages has no definition of its own: it is ``oracle.decode``.)

Each function states its definition once, sequentially, and shares no code with the product.
"""
from __future__ import annotations

import math

import numpy as np

__all__ = ["select", "fork", "copy_pages"]


def select(logits, scores, k, live=None, eos=-1):
    """Returns (scores fp64, parents, tokens, live), each [N, k], and the 64-bit scores of all candidates
    per request as a list of (score, beam, token), best first."""
    N, W, V = logits.shape
    out = np.full((N, k), -np.inf), np.full((N, k), -1), np.full((N, k), -1), np.zeros((N, k), int)
    every = []
    for n in range(N):
        cand = []
        for b in range(W):
            s = float(scores[n, b])
            if not math.isfinite(s):
                continue
            if live is not None and live[n, b] == 0:
                cand.append((s, b, eos))
                continue
            x = np.asarray(logits[n, b], np.float64)
            if np.isnan(x).any() or np.isposinf(x).any() or np.isneginf(x).all():
                continue
            m = x.max()
            norm = m + math.log(math.fsum(np.exp(x - m)))
            cand += [(s - norm + x[v], b, v) for v in range(V) if x[v] > -np.inf]
        cand.sort(key=lambda c: (-c[0], c[1], c[2]))
        every.append(cand)
        for i, (s, b, v) in enumerate(cand[:k]):
            ended = live is not None and live[n, b] == 0
            out[0][n, i], out[1][n, i], out[2][n, i] = s, b, v
            out[3][n, i] = 0 if ended or v == eos else 1
    return out, every


def fork(parents, lens, table, free, count, num_pages, page_size=16):
    """Returns dict(lens, table, free, count, copies, shared, flags) of one fork; flags is a set of
    'length', 'no_pages', 'page'."""
    P = page_size
    parents, lens = np.asarray(parents), [int(x) for x in lens]
    G, W = parents.shape
    table, free = np.array(table, copy=True), np.array(free, copy=True)
    cap = table.shape[1] * P
    flags = set()
    if not 0 <= count <= len(free):
        flags.add("length")
        count = min(max(count, 0), len(free))
    none = [(-1, -1, 0)] * (G * W)
    same = dict(lens=list(lens), table=table.copy(), free=free.copy(), count=count, copies=none, shared=[0] * G)
    if any(not -1 <= p < W for p in parents.ravel()) or any(not 0 <= n <= cap for n in lens):
        return dict(same, flags=flags | {"length"})
    pages = lambda n: -(-n // P)
    new_lens, copies, shared, freed = [0] * (G * W), list(none), [0] * G, []
    held, given = [[] for _ in range(G * W)], []   # pages of every new row; rows that get a page of their own
    for g in range(G):
        rows = range(g * W, g * W + W)
        for b in rows:
            p = parents[g, b - g * W]
            if p >= 0:
                new_lens[b] = lens[g * W + p]
                held[b] = [int(e) for e in table[g * W + p, :pages(new_lens[b])]]
        for b in rows:
            if new_lens[b] % P == 0:
                continue
            at = len(held[b]) - 1
            page = held[b][at]
            if not 0 <= page < num_pages:
                flags.add("page")
                continue
            others = [o for o in rows if o != b and len(held[o]) > at and held[o][at] == page]
            if any(o < b or new_lens[o] >= P * (at + 1) for o in others):
                given.append((b, page))
        live = [b for b in rows if new_lens[b] > 0]
        while live and all(shared[g] < new_lens[b] // P for b in live):
            here = {held[b][shared[g]] for b in live}
            if len(here) > 1 or min(here) < 0:
                break
            shared[g] += 1
        kept = {(j, e) for b in rows for j, e in enumerate(held[b])}
        for j in range(table.shape[1]):
            for r in rows:
                if j >= pages(lens[r]):
                    continue
                e = int(table[r, j])
                if (j, e) in kept:
                    continue
                if e >= num_pages:
                    flags.add("page")
                elif e >= 0:
                    kept.add((j, e))
                    freed.append(e)
    if len(given) > count:
        flags.add("no_pages")
    if count - len(given) + len(freed) > len(free):
        flags.add("length")
    if len(given) > count or count - len(given) + len(freed) > len(free):
        return dict(same, flags=flags)
    for b, page in given:
        count -= 1
        fresh = int(free[count])
        held[b][-1] = fresh
        if 0 <= fresh < num_pages:
            copies[b] = (page, fresh, new_lens[b] % P)
        else:
            flags.add("page")
    for e in freed:
        free[count] = e
        count += 1
    for b in range(G * W):
        table[b, :pages(lens[b])] = -1
        table[b, :len(held[b])] = held[b]
    return dict(lens=new_lens, table=table, free=free, count=count, copies=copies, shared=shared, flags=flags)


def copy_pages(copies, pool):
    """pool [num_pages, 16, ...] after the copies."""
    out = np.array(pool, copy=True)
    for src, dst, n in copies:
        if n > 0:
            out[dst, :n] = pool[src, :n]
    return out
