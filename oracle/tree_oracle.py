"""Plain definitions of a drafted tree's verification: masks and positions,
the greedy walk, the rows' move, and which cache rows a node attends.

TEST INFRASTRUCTURE: imported only by tests/.  It shares no code with the CUDA
path; trees are walked node by node in Python.

Pins (tests/test_tree_operators.py): a tree drawn by hand.
"""
from __future__ import annotations

import numpy as np


def ancestors(parent, j):
    """Node j's own index and its ancestors', upwards."""
    line = []
    while j >= 0:
        line.append(j)
        j = int(parent[j])
    return line


def tree_maps(parents, row_start, prefix, T, max_nodes):
    """(masks uint64 [T, W], positions int32 [T])."""
    W = -(-max_nodes // 64)
    masks = np.zeros((T, W), dtype=np.uint64)
    positions = np.zeros(T, dtype=np.int32)
    for b in range(len(row_start) - 1):
        parent = parents[row_start[b]:row_start[b + 1]]
        for j in range(len(parent)):
            line = ancestors(parent, j)
            t = row_start[b] + j
            for m in line:
                masks[t, m // 64] |= np.uint64(1) << np.uint64(m % 64)
            positions[t] = prefix[b] + len(line) - 1
    return masks, positions


def tree_accept(parents, tokens, targets, row_start, T):
    """(accepted [B], rows [T], next_tokens [B])."""
    accepted, rows, nexts = [], [], []
    for b in range(len(row_start) - 1):
        t0, n = int(row_start[b]), int(row_start[b + 1] - row_start[b])
        line = []
        if n > 0:
            line = [0]
            while True:
                u = line[-1]
                fits = [c for c in range(u + 1, n) if parents[t0 + c] == u
                        and tokens[t0 + c] == targets[t0 + u]]
                if not fits:
                    break
                line.append(fits[0])
        accepted.append(len(line))
        rows += [t0 + j for j in line]
        nexts.append(int(targets[t0 + line[-1]]) if line else -1)
    rows += [-1] * (T - len(rows))
    return (np.array(accepted, dtype=np.int32), np.array(rows, dtype=np.int32),
            np.array(nexts, dtype=np.int32))


def random_tree(rng, n, shape="bushy"):
    """Parents of n nodes: a chain, a star, or each on one of the few before."""
    if shape == "chain":
        return np.arange(n) - 1
    if shape == "star":
        return np.where(np.arange(n) > 0, 0, -1)
    if shape == "roots":  # every node follows the prefix
        return np.full(n, -1)
    return np.array([-1 if j == 0 else rng.integers(max(0, j - 5), j) for j in range(n)])


def prefix_keys(ctx, D, rank, bs, I, tables, b):
    """(pool, slot) of the positions 0..ctx-1 of request b, on `rank` or all."""
    keys = []
    for p in range(ctx):
        d = (p // I) % D
        if rank >= 0 and d != rank:
            continue
        lp = (p // (I * D)) * I + p % I
        keys.append((d, int(tables[d][b][lp // bs]) * bs + lp % bs))
    return keys


def draft_key(slots, row):
    """(pool, slot) of a drafted node: the lowest pool that holds it, or None.
    `slots`: pool -> its draft slots, of the pools attended."""
    for d in sorted(slots):
        if slots[d][row] >= 0:
            return d, int(slots[d][row])
    return None
