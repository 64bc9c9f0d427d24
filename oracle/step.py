"""Oracle of a step that verifies drafted tokens: the plan of its index arrays, the masks of its
trees, the commit of accepted rows, and its attention in fp64.

TEST INFRASTRUCTURE: see the package docstring. Plain Python and numpy loops from the
definitions, sharing no code with the kernels.
"""
import math

import numpy as np


def plan(lens, new, tables, held, free_list, free, bs, num_blocks, N, keep=None, bad=()):
    """Returns (tables, held, free_list, free, missing, row_starts, positions, slots); lists and arrays are copied.
    What a stack place or table entry held stays where nothing is written; entries that a sequence wanted and did not
    get are -1. Sequences `bad` have numbers out of range:
    their blocks stay and their rows have no slot."""
    B, mbps = tables.shape
    tables, stack = tables.copy(), list(free_list[:free])
    need = [max(-(-(lens[b] + new[b]) // bs), 0 if keep is None else keep[b]) for b in range(B)]
    for b in bad:
        need[b] = held[b]
    for b in range(B):
        for k in range(need[b], held[b]):
            stack.append(tables[b, k])
    room, wanted, missing, taken, short = len(stack), 0, 0, 0, set()
    for b in range(B):
        take = max(0, need[b] - held[b])
        wanted += take
        if take and wanted > room:
            short.add(b)
            missing += take
            tables[b, held[b]:need[b]] = -1
            continue
        for k in range(held[b], held[b] + take):
            tables[b, k] = stack[room - 1 - taken]
            taken += 1
    left = room - taken
    out_list = np.array(free_list).copy()
    out_list[free:left] = stack[free:left]
    starts = np.concatenate([[0], np.cumsum(np.maximum(new, 0))])
    positions, slots = np.zeros(N, np.int64), np.full(N, -1, np.int64)
    for b in range(B):
        for i in range(min(new[b], N - starts[b])):
            at = lens[b] + i
            positions[starts[b] + i] = at
            if b not in short and b not in bad:
                slots[starts[b] + i] = int(tables[b, at // bs]) * bs + at % bs
    held_out = [held[b] if b in short else need[b] for b in range(B)]
    return tables, np.array(held_out), out_list, left, missing, starts, positions, slots


def ancestors(parents, starts):
    """For each packed row the set of rows of its tree that it sees (itself among them)."""
    out = []
    for b in range(len(starts) - 1):
        for i in range(starts[b + 1] - starts[b]):
            seen, at = set(), i
            while at >= 0:
                seen.add(at)
                at = parents[starts[b] + at]
            out.append(seen)
    return out


def words(seen, n):
    """Sets of rows as int64 mask words [len(seen), n]."""
    out = np.zeros((len(seen), n), np.uint64)
    for i, s in enumerate(seen):
        for j in s:
            out[i, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    return out.view(np.int64)


def commit(pool, table, length, path):
    """pool [num_blocks, Hkv, bs, d] with the accepted rows of one sequence moved."""
    pool, bs = pool.copy(), pool.shape[2]
    rows = [pool[table[(length + x) // bs], :, (length + x) % bs].copy() for x in path]
    for j, r in enumerate(rows):
        pool[table[(length + j) // bs], :, (length + j) % bs] = r
    return pool


def attend(q, k, v, hist, seen, scale, window=0, softcap=0.0, sinks=None, slopes=None):
    """q [n, H, dk] of one sequence's drafted rows, k [Hkv, hist + n, dk], v [.., dv]; seen[i]: the drafted rows
    that row i sees. A drafted row stands at position hist + (rows that it sees, at least 1) - 1. Keys that a row does not see
    take no part, whatever they hold. Returns the output, sum_j w_j |v_j| and the largest scale * sum |q_i k_ji|."""
    n, H, _ = q.shape
    dv = v.shape[2]
    out, size, reach = np.zeros((n, H, dv)), np.zeros((n, H, dv)), np.zeros((n, H, 1))
    G = H // k.shape[0]
    at = [hist + max(len(s), 1) - 1 for s in seen]
    for i in range(n):
        keys = [(j, j) for j in range(hist)] + [(hist + j, at[j]) for j in sorted(seen[i])]
        if window > 0:
            keys = [(j, p) for j, p in keys if p > at[i] - window]
        if not keys:
            continue
        idx = np.array([j for j, _ in keys])
        pos = np.array([p for _, p in keys], np.float64)
        for h in range(H):
            kh, vh = k[h // G][idx], v[h // G][idx]
            with np.errstate(invalid="ignore", over="ignore"):
                s = scale * (kh @ q[i, h])
                far = scale * (np.abs(kh) @ np.abs(q[i, h]))
                reach[i, h, 0] = far[s != -math.inf].max(initial=0.0)  # (a key that scores -infinity weighs zero, exactly)
                if softcap > 0:
                    s = softcap * np.tanh(s / softcap)
                if slopes is not None:
                    s = s + slopes[h] * (pos - at[i])
                m = max(s.max(), -math.inf if sinks is None else sinks[h])
                if m == -math.inf:
                    continue
                w = np.exp(s - m)
                den = w.sum() + (0.0 if sinks is None else np.exp(sinks[h] - m))
                w, vh = w[w != 0], vh[w != 0]
                out[i, h] = w @ vh / den
                size[i, h] = w @ np.abs(vh) / den
    return out, size, reach
