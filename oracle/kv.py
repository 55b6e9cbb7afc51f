"""Reference definitions in fp64 (numpy) of the operators around attention: rotary positions, page
planning, the 4-bit cache's quantiser and attention over a paged cache.

Written from the definitions, one request and one row at a time, on values decoded from their bit
fields; shares no code, header or constant with the CUDA library."""
from __future__ import annotations

import math

import numpy as np

GROUP = 16


# --------------------------------------------------------------------------------- rotary positions
def rope(x, positions, turns, interleaved=False, inverse=False, mscale=1.0):
    """x [..., N, d] fp64 at positions [N]; turns: integers, units of 2^-64 turn.  The angle is the
    exact product reduced modulo one turn with Python integers."""
    x = np.asarray(x, dtype=np.float64)
    y = x.copy()
    half = len(turns)
    angle = np.empty((len(positions), half))
    for n, p in enumerate(positions):
        for i, t in enumerate(turns):
            frac = (int(p) * int(t)) % (1 << 64)
            if frac >= 1 << 63:
                frac -= 1 << 64
            angle[n, i] = 2 * math.pi * (frac / 2.0 ** 64)
    if inverse:
        angle = -angle
    first = slice(0, 2 * half, 2) if interleaved else slice(0, half)
    second = slice(1, 2 * half, 2) if interleaved else slice(half, 2 * half)
    a, b = x[..., first], x[..., second]
    y[..., first] = mscale * (a * np.cos(angle) - b * np.sin(angle))
    y[..., second] = mscale * (b * np.cos(angle) + a * np.sin(angle))
    return y


# --------------------------------------------------------------------------------- page planning
def page_plan(lens, new_lens, table, queue, state, page, num_tokens):
    """One request after the other; returns new copies (lens, q_offsets, positions, slots, state,
    table, queue)."""
    lens, table, queue = [int(x) for x in lens], [list(r) for r in table], list(queue)
    head, count = state
    cap, width = len(queue), len(table[0])
    used, wanted, back = 0, 0, []
    out, offsets, positions, slots = [], [0], [], []
    for b, (n, add) in enumerate(zip(lens, new_lens)):
        have = math.ceil(n / page)
        if add < 0:
            back += table[b][:have]
            out.append(0)
            offsets.append(offsets[-1])
            continue
        want = math.ceil((n + add) / page)
        need = want - have if want <= width else 0
        wanted += need
        ok = want <= width and (need == 0 or wanted <= count)
        if ok:
            for i in range(have, want):
                table[b][i] = queue[(head + used) % cap]
                used += 1
        out.append(n + add if ok else n)
        offsets.append(offsets[-1] + add)
        for p in range(n, n + add):
            positions.append(p)
            slot = table[b][p // page] * page + p % page if ok else -1
            slots.append(slot if 0 <= slot < 2 ** 31 else -1)
    back = back[:cap - count]  # what the ring has no room for is lost
    for i, p in enumerate(back):
        queue[(head + count + i) % cap] = p
    pad = num_tokens - len(positions)
    return (out, offsets, (positions + [0] * pad)[:num_tokens], (slots + [-1] * pad)[:num_tokens],
            [(head + used) % cap, count - used + len(back)], table, queue)


# --------------------------------------------------------------------------------- the 4-bit cache
def _grid(exponent_bits, mantissa_bits, bias, codes):
    """The non-negative values of a small float format, by code."""
    out = []
    for c in range(codes):
        e, m = c >> mantissa_bits, c & ((1 << mantissa_bits) - 1)
        f = m / 2.0 ** mantissa_bits
        out.append(f * 2.0 ** (1 - bias) if e == 0 else (1 + f) * 2.0 ** (e - bias))
    return np.array(out)


E2M1 = _grid(2, 1, 1, 8)      # 0 .. 6
E4M3 = _grid(4, 3, 7, 127)    # 0 .. 448 (code 127 is NaN)


def nearest(x, grid):
    """Code of the grid value nearest to each x >= 0; ties to the even code; saturating."""
    x = np.asarray(x, dtype=np.float64)
    hi = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo = hi - 1
    down, up = x - grid[lo], grid[hi] - x
    return np.where((down < up) | ((down == up) & (lo % 2 == 0)), lo, hi)


def quantise(x, descale=1.0):
    """x [..., d] -> codes (0 .. 15) [..., d], scale codes [..., d / 16]."""
    x = np.asarray(x, dtype=np.float64)
    bad = ~np.isfinite(x).all(-1)
    g = np.where(bad[..., None], 0.0, x).reshape(*x.shape[:-1], -1, GROUP) / descale
    s8 = nearest(np.abs(g).max(-1) / 6, E4M3)
    s = E4M3[s8][..., None]
    with np.errstate(divide="ignore", invalid="ignore"):
        t = np.where(s > 0, np.abs(g) / s, 0.0)
    code = nearest(t, E2M1) | (np.signbit(g) & (s > 0)).astype(np.int64) << 3
    return (code.reshape(x.shape).astype(np.uint8),
            np.where(bad[..., None], 127, s8).astype(np.uint8))


def dequantise(code, s8, descale=1.0):
    v = np.where(code >= 8, -E2M1[code & 7], E2M1[code & 7])
    s = np.append(E4M3, np.nan)[np.asarray(s8) & 127]
    return v * np.repeat(s, GROUP, axis=-1) * descale


def block(code, s8):
    """Bytes of one (page, head) block from the codes and scales of its rows."""
    packed = (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8)
    return np.concatenate([packed.reshape(-1), s8.astype(np.uint8).reshape(-1)])


def unblock(raw, page, d):
    """Codes and scales [page, ...] of one block's bytes."""
    packed = raw[:page * d // 2].reshape(page, d // 2)
    code = np.empty((page, d), dtype=np.uint8)
    code[:, 0::2], code[:, 1::2] = packed & 15, packed >> 4
    return code, raw[page * d // 2:].reshape(page, d // GROUP)


# --------------------------------------------------------------------------------- attention
def kv4_attention(q, cache, table, lens, q_offsets, d, scale, causal, k_descale=1.0, v_descale=1.0):
    """q [T, Hq, d] fp64, cache bytes [P, Hkv, 2, :]; returns O [T, Hq, d], LSE [T, Hq], and for
    tolerances, per row, the sums of p |v| and of |v| and the largest sum |q k| of a visible key.
    Rows past the last request keep NaN; of a request that reaches past the T rows there are the first are
    computed, at the places in the cache that they have among all of its rows."""
    T, Hq, _ = q.shape
    P, Hkv = cache.shape[:2]
    page = cache.shape[3] * 16 // (9 * d)
    o, lse = np.full((T, Hq, d), np.nan), np.full((T, Hq), np.nan)
    mass, total, dot = np.zeros((T, Hq, d)), np.zeros((T, Hq, d)), np.zeros((T, Hq))
    for b in range(len(lens)):
        n = min(max(int(lens[b]), 0), table.shape[1] * page)
        rows = int(q_offsets[b + 1]) - int(q_offsets[b])
        for h in range(Hkv):
            k, v = np.zeros((n, d)), np.zeros((n, d))
            there = np.zeros(n, dtype=bool)
            for j0 in range(0, n, page):
                p = int(table[b, j0 // page])
                if not 0 <= p < P:
                    continue
                m = min(page, n - j0)
                there[j0:j0 + m] = True
                for dst, kv, ds in ((k, 0, k_descale), (v, 1, v_descale)):
                    dst[j0:j0 + m] = dequantise(*unblock(cache[p, h, kv], page, d), ds)[:m]
            for i in range(min(rows, T - int(q_offsets[b]))):
                t = int(q_offsets[b]) + i
                seen = there & (np.arange(n) <= (n - rows + i if causal else n))
                for g in range(Hq // Hkv):
                    r = h * (Hq // Hkv) + g
                    if not seen.any():
                        o[t, r], lse[t, r] = 0.0, -np.inf
                        continue
                    x = scale * (k[seen] @ q[t, r])
                    top = x.max()
                    e = np.exp(x - top)
                    lse[t, r] = top + math.log(e.sum())
                    p = e / e.sum()
                    o[t, r] = p @ v[seen]
                    mass[t, r], total[t, r] = p @ np.abs(v[seen]), np.abs(v[seen]).sum(0)
                    dot[t, r] = (np.abs(k[seen]) @ np.abs(q[t, r])).max()
    return o, lse, mass, total, dot
