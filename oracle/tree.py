"""Reference definitions in fp64 (numpy) of rotary positions with several axes and of trees of drafted tokens:
their plan, attention over a paged 4-bit cache, what is accepted, and the move of cached rows.

Written from the definitions, one request, one node and one row at a time; shares no code with the CUDA
library."""
from __future__ import annotations

import math

import numpy as np

from .kv import dequantise, unblock


def rope_axes(x, positions, turns, axes, interleaved=False, inverse=False, mscale=1.0):
    """x [..., N, d] fp64 at positions [A][N]; pair i turns by positions[axes[i]] times turns[i] (integers, units
    of 2^-64 turn; the exact product reduced modulo one turn with Python integers)."""
    y = np.array(x, dtype=np.float64)
    half = len(turns)
    for i, t in enumerate(turns):
        axis = int(axes[i])
        row = positions[axis if axis < len(positions) else 0]
        part = np.array([(int(p) * int(t)) % (1 << 64) / 2.0 ** 64 for p in row])
        angle = 2 * math.pi * np.where(part >= 0.5, part - 1, part) * (-1 if inverse else 1)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        u, v = np.array(x[..., a], dtype=np.float64), np.array(x[..., b], dtype=np.float64)
        y[..., a] = mscale * (u * np.cos(angle) - v * np.sin(angle))
        y[..., b] = mscale * (v * np.cos(angle) + u * np.sin(angle))
    return y


def way_up(parents, i):
    """Node i and the nodes above it, from i up; a parent that is no smaller number >= 0 ends the way."""
    out = [i]
    while 0 <= parents[out[-1]] < out[-1]:
        out.append(parents[out[-1]])
    return out


def tree_plan(parents, q_offsets, lens, words):
    """Positions [T] and truth values [T, 32 words]; zeros past the last request."""
    T = len(parents)
    positions, seen = np.zeros(T, dtype=np.int64), np.zeros((T, 32 * words), dtype=bool)
    for b in range(len(lens)):
        first, last = min(q_offsets[b], T), min(q_offsets[b + 1], T)
        mine = parents[first:last]
        for i in range(last - first):
            way = way_up(mine, i)
            positions[first + i] = lens[b] + len(way) - 1
            for j in way:
                if j < 32 * words:
                    seen[first + i, j] = True
    return positions, seen


def bits(seen):
    """Truth values [T, 32 words] as int32 words [T, words]."""
    word = (seen.reshape(seen.shape[0], -1, 32).astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1)
    return word.astype(np.uint32).view(np.int32)


def tree_accept(parents, tokens, choices, lens, new_lens, q_offsets, slots, table, queue, state, page, words):
    """One request after the other, walking down from node 0; returns new copies (lens, counts, path, next,
    sources, state, queue)."""
    T, queue = len(parents), list(queue)
    head, free = state
    out, counts, nexts = [], [], []
    path, sources, back = [-1] * T, [-1] * T, []
    for b in range(len(lens)):
        first, last = min(q_offsets[b], T), min(q_offsets[b + 1], T)
        n = min(last - first, 32 * words)
        at, way = 0, []
        while new_lens[b] > lens[b] and n > 0:
            way.append(at)
            children = [j for j in range(at + 1, n)
                        if parents[first + j] == at and tokens[first + j] == choices[first + at]]
            if not children:
                break
            at = children[0]
        for i, node in enumerate(way):
            path[first + i], sources[first + i] = node, slots[first + node]
        counts.append(len(way))
        nexts.append(choices[first + way[-1]] if way else -1)
        out.append(min(lens[b], new_lens[b]) + len(way))
        have, keep = math.ceil(max(new_lens[b], 0) / page), math.ceil(max(out[b], 0) / page)
        back += list(table[b][keep:have])
    back = back[:len(queue) - free]  # what the ring has no room for is lost
    for i, p in enumerate(back):
        queue[(head + free + i) % len(queue)] = p
    return out, counts, path, nexts, sources, [head, free + len(back)], queue


def kv4_move(cache, sources, slots, q_offsets, counts, d):
    """A copy of the cache's bytes [P, H, 2, :] with the rows moved."""
    old, new = cache, cache.copy()
    page = cache.shape[3] * 16 // (9 * d)
    for b in range(len(counts)):
        for i in range(q_offsets[b], q_offsets[b] + min(counts[b], q_offsets[b + 1] - q_offsets[b])):
            (p, r), (q, s) = divmod(int(sources[i]), page), divmod(int(slots[i]), page)
            if not (0 <= p < len(cache) and 0 <= q < len(cache)):
                continue
            for at, size in ((0, d // 2), (page * d // 2, d // 16)):
                new[q, :, :, at + s * size:at + (s + 1) * size] = old[p, :, :, at + r * size:at + (r + 1) * size]
    return new


def kv4_tree_attention(q, cache, table, lens, q_offsets, seen, d, scale, k_descale=1.0, v_descale=1.0):
    """q [T, Hq, d] fp64, cache bytes [P, Hkv, 2, :], seen [T, bits] truth values; returns O, LSE and for
    tolerances, per row, the sums of p |v| and of |v| and the largest sum |q k| of a key it sees.  Rows past the
    last request keep NaN; a request that reaches past the T rows keeps its nodes' places."""
    T, Hq, _ = q.shape
    P, Hkv = cache.shape[:2]
    page, group = cache.shape[3] * 16 // (9 * d), Hq // Hkv
    o, lse = np.full((T, Hq, d), np.nan), np.full((T, Hq), np.nan)
    mass, total, dot = np.zeros((T, Hq, d)), np.zeros((T, Hq, d)), np.zeros((T, Hq))
    for b in range(len(lens)):
        n = min(max(int(lens[b]), 0), table.shape[1] * page)
        nodes = int(q_offsets[b + 1]) - int(q_offsets[b])
        there = np.zeros(n, dtype=bool)
        kv = np.zeros((2, Hkv, n, d))
        for j0 in range(0, n, page):
            p, m = int(table[b, j0 // page]), min(page, n - j0)
            if 0 <= p < P:
                there[j0:j0 + m] = True
                for h in range(Hkv):
                    for x, ds in ((0, k_descale), (1, v_descale)):
                        kv[x, h, j0:j0 + m] = dequantise(*unblock(cache[p, h, x], page, d), ds)[:m]
        for i in range(min(nodes, T - int(q_offsets[b]))):
            t = int(q_offsets[b]) + i
            node = np.arange(n) - (n - nodes)
            sees = there & ((node < 0) | seen[t][np.clip(node, 0, seen.shape[1] - 1)] & (node < seen.shape[1]))
            for r in range(Hq):
                if not sees.any():
                    o[t, r], lse[t, r] = 0.0, -np.inf
                    continue
                k, v = kv[0, r // group, sees], kv[1, r // group, sees]
                x = scale * (k @ q[t, r])
                e = np.exp(x - x.max())
                lse[t, r] = x.max() + math.log(e.sum())
                p = e / e.sum()
                o[t, r] = p @ v
                mass[t, r], total[t, r] = p @ np.abs(v), np.abs(v).sum(0)
                dot[t, r] = (np.abs(k) @ np.abs(q[t, r])).max()
    return o, lse, mass, total, dot
