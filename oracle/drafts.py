"""CPU oracle of decoding with drafted tokens -- TEST INFRASTRUCTURE ONLY (see the package docstring).

Trees are given by parents, attention by who sees whom; verification runs in Python's whole numbers, the move as
reads of all rows before the writes.  The pages have no counterpart: these are the definitions themselves.
"""
from __future__ import annotations

import numpy as np

from . import attention

ONE = 1 << 60


def ancestors(parents) -> np.ndarray:
    """seen[i, j]: node j is i or one of its ancestors, by walking up from each node."""
    n = len(parents)
    seen = np.zeros((n, n), dtype=bool)
    for i in range(n):
        j = i
        while j >= 0:
            seen[i, j] = True
            j = parents[j]
    return seen


def tree_attention(q, k_cache, v_cache, block_tables, context_lens, query_start, seen, scale):
    """float64 [total_q, H, D]; seen: one [n_s, n_s] truth table per sequence.  Rows of q in no sequence stay NaN."""
    T, H, D = q.shape
    group = H // k_cache.shape[1]
    out = np.full((T, H, D), np.nan)
    for s, ctx in enumerate(context_lens):
        q0, n = int(query_start[s]), int(query_start[s + 1] - query_start[s])
        if n == 0:
            continue
        keys = attention.gather_sequence(k_cache, block_tables[s], ctx)
        values = attention.gather_sequence(v_cache, block_tables[s], ctx)
        for i in range(n):
            live = np.concatenate([np.ones(int(ctx) - n, dtype=bool), seen[s][i]])
            out[q0 + i] = attention.contiguous_attention(q[q0 + i], np.repeat(keys[live], group, axis=1),
                                                         np.repeat(values[live], group, axis=1), scale)
    return out


def _whole(x) -> list:
    """floor(x 2^60) of fp32 numbers, exactly: the product with a power of two is."""
    return [int(v * float(ONE)) for v in np.asarray(x, dtype=np.float64).tolist()]


def verify(target, draft, tokens, parents, uniforms, max_path):
    """One sequence's (path, next token) from its rows, by the rule's own words."""
    at, path = 0, [0]
    left, mass, taken = _whole(target[0]), ONE, 0
    j = 1
    while j < len(tokens) and len(path) < max_path:
        if parents[j] == at:
            x, u = int(tokens[j]), _whole([uniforms[j]])[0]
            q = None if draft is None else _whole(draft[at])
            threshold = (mass * (ONE if q is None else q[x]) >> 60) * u >> 60
            if threshold < left[x]:
                path.append(j)
                at, left, mass, taken = j, _whole(target[j]), ONE, 0
            elif q is None:
                mass = max(mass - left[x], 0)
                left[x] = 0
            else:
                taken += mass
                left = [max(p - (taken * d >> 60), 0) for p, d in zip(_whole(target[at]), q)]
                mass = sum(left)
        j += 1
    # where the path is full the last node's children are not tried, and its row is untouched
    if sum(left) == 0:
        left = _whole(target[at])
    aim, upto = sum(left) * _whole([uniforms[0]])[0] >> 60, 0
    for i, r in enumerate(left):
        upto += r
        if upto > aim:
            return path, i
    return path, -1


def move_accepted(k_caches, v_caches, slots, query_start, path, path_len):
    """In place: all of a sequence's source rows are read, then written."""
    B = k_caches[0].shape[2]
    for s, kept in enumerate(path_len):
        q0 = int(query_start[s])
        for pools in (k_caches, v_caches):
            for pool in pools:
                rows = [pool[slots[q0 + path[s][i]] // B, :, slots[q0 + path[s][i]] % B].copy() for i in range(1, kept)]
                for i, row in enumerate(rows, 1):
                    pool[slots[q0 + i] // B, :, slots[q0 + i] % B] = row
