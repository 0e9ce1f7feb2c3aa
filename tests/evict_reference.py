"""Plain restatement of the eviction calls on host arrays, one (sequence, KV
head) and one slot at a time: which tokens stay, and where their rows go."""
from __future__ import annotations

import numpy as np


def slot_positions(positions, recorded, length, n):
    """Position of each of the first n slots."""
    return np.array([int(positions[i]) if i < recorded else int(length) - n + i
                     for i in range(n)], dtype=np.int64)


def select_row(weights, positions, recorded, length, n, budget, sink, recent):
    """source [budget] of one (sequence, KV head) with n tokens."""
    source = np.full(budget, -1, dtype=np.int32)
    new = min(n, budget)
    source[:new] = np.arange(new)
    if n <= budget:
        return source
    pos = slot_positions(positions, recorded, length, n)

    def claim(i):                     # ascending order of claims, best last
        w = float(weights[i])
        held = pos[i] < sink or pos[i] >= int(length) - recent
        return (held, w == w, w if w == w else 0.0, -i)

    kept = set(sorted(range(n), key=claim)[n - budget:])
    tail = [i for i in range(budget, n) if i in kept]
    holes = [i for i in range(budget) if i not in kept]
    assert len(tail) == len(holes)
    for i, j in zip(holes, tail):
        source[i] = j
    return source


def select(weights, positions, recorded, seq_lens, context_lens, budget, sink, recent):
    S, Hk, W = weights.shape
    source = np.stack([np.stack([
        select_row(weights[s, h], positions[s, h], int(recorded[s]), int(seq_lens[s]),
                   int(context_lens[s]), budget, sink, recent) for h in range(Hk)])
        for s in range(S)])
    return source, np.minimum(context_lens, budget).astype(np.int32)


def compact(key_cache, value_cache, weights, positions, source, new_lens, tables, context_lens,
            recorded, seq_lens):
    """Edits copies of the caches, weights and positions; returns them."""
    kc, vc, w, p = (x.copy() for x in (key_cache, value_cache, weights, positions))
    bs = key_cache.shape[1]
    S, Hk, _ = weights.shape
    for s in range(S):
        n = int(context_lens[s])
        for h in range(Hk):
            pos = slot_positions(positions[s, h], int(recorded[s]), int(seq_lens[s]), n)
            for i in range(int(new_lens[s])):
                j = int(source[s, h, i])
                p[s, h, i] = pos[j]
                w[s, h, i] = weights[s, h, j]
                if i != j:
                    a, b = tables[s, j // bs], tables[s, i // bs]
                    kc[b, i % bs, h] = key_cache[a, j % bs, h]
                    vc[b, i % bs, h] = value_cache[a, j % bs, h]
    return kc, vc, w, p
