"""The step around the cache in plain numpy, 64-bit: slots from request lengths, rotary
positions, attention over packed prompts.

"LLM inference tutorial" section 4.2 (append_token: a new block at every multiple of the block
size), 4.4 (MHA/GQA forward), 1.2 (prefill)."""
from __future__ import annotations

import numpy as np


def slots(tables, ctx, new, free, free_start, block_size, num_tokens, num_blocks,
          row_per_sequence=False, first_block_held=False):
    """(tables, slot_mapping, positions, query_start, context_out, free_next, flags), one token at
    a time.  ``flags``: the names of the status bits."""
    tables, ctx = np.array(tables), [int(c) for c in ctx]
    new = [1] * len(ctx) if new is None else [int(n) for n in new]
    mb, flags = tables.shape[1], set()
    slot = np.full(num_tokens, -1, dtype=np.int64)
    pos = np.zeros(num_tokens, dtype=np.int32)
    rows = [1 if row_per_sequence else max(n, 0) for n in new]
    good = [c >= 0 and n >= 0 and c + n <= mb * block_size and (n <= 1 or not row_per_sequence)
            for c, n in zip(ctx, new)]
    if not all(good):
        flags.add("context")
    held = [max(-(-c // block_size), 1 if first_block_held else 0) for c in ctx]
    need = [max(-(-(c + n) // block_size) - h, 0) if ok else 0
            for c, n, h, ok in zip(ctx, new, held, good)]
    few = sum(need) > 0 and not 0 <= free_start <= len(free) - sum(need)
    if few:
        flags.add("free")
    if sum(rows) > num_tokens:
        flags.add("context")
    if few or sum(rows) > num_tokens:
        return (tables, slot, pos, np.zeros(len(ctx) + 1, dtype=np.int32),
                np.array(ctx, dtype=np.int32), free_start, flags)
    at, row, start, out = free_start, 0, [0], []
    for s, (c, n, ok) in enumerate(zip(ctx, new, good)):
        for i in range(n if ok else 0):
            p = c + i
            if p // block_size >= held[s] and p % block_size == 0:
                tables[s, p // block_size] = free[at]
                at += 1
            b = int(tables[s, p // block_size])
            if 0 <= b < num_blocks:
                slot[row + i] = b * block_size + p % block_size
            else:
                flags.add("block")
            pos[row + i] = p
        row += rows[s]
        start.append(row)
        out.append(c + n if ok else c)
    return (tables, slot, pos, np.array(start, dtype=np.int32), np.array(out, dtype=np.int32), at,
            flags)


def rotary(x, positions, inv_freq, axes=None, adjacent=False, scale=1.0):
    """float64 rows ``[T, H, D]`` turned; ``positions`` ``[T]`` or ``[axes, T]``."""
    y = np.array(x, dtype=np.float64)
    positions = np.asarray(positions, dtype=np.float64).reshape(-1, y.shape[0])
    half = len(inv_freq)
    for i, f in enumerate(np.asarray(inv_freq, dtype=np.float64)):
        angle = positions[0 if axes is None else axes[i]] * f
        c, s = scale * np.cos(angle)[:, None], scale * np.sin(angle)[:, None]
        a, b = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
        u, w = y[:, :, a].copy(), y[:, :, b].copy()
        y[:, :, a], y[:, :, b] = u * c - w * s, w * c + u * s
    return y


def packed(q, k, v, q_start, k_start, scale, causal=True, window=0, sinks=0):
    """float64 ``(out, A, reach, seen)`` of packed rows ``[T, Hq, D]``, ``[N, Hkv, D]``: the attention,
    ``A`` = sum p |v|, ``reach`` = max over visible keys of sum |q_d k_d| and the number of visible
    keys.  Rows outside every sequence are NaN."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    group, scale = q.shape[1] // k.shape[1], float(np.float32(scale))
    out, mag = np.full(q.shape, np.nan), np.zeros(q.shape)
    reach, seen = np.zeros(q.shape[:2]), np.zeros(q.shape[0], dtype=np.int64)
    for s in range(len(q_start) - 1):
        a, b, c0, c1 = (int(x) for x in (q_start[s], q_start[s + 1], k_start[s], k_start[s + 1]))
        n, c = b - a, c1 - c0
        j = np.arange(c)
        for i in range(n):
            p = c - n + i
            vis = np.ones(c, dtype=bool)
            if causal:
                vis = j <= p
                if window:
                    vis &= (j > p - window) | (j < sinks)
            rows = c0 + j[vis]
            seen[a + i] = rows.size
            if rows.size == 0:
                out[a + i] = 0.0
                continue
            for h in range(q.shape[1]):
                z = k[rows, h // group] @ q[a + i, h] * scale
                w = np.exp(z - z.max())
                w /= w.sum()
                out[a + i, h] = w @ v[rows, h // group]
                mag[a + i, h] = w @ np.abs(v[rows, h // group])
                reach[a + i, h] = (np.abs(k[rows, h // group]) @ np.abs(q[a + i, h])).max()
    return out, mag, reach, seen
