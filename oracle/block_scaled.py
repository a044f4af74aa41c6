"""Oracle for the 8-bit cache with one scale per (block, KV head), and for
attention with a sliding window and sinks (plain definitions, numpy).

TEST INFRASTRUCTURE ONLY (see ``oracle/__init__``).

``quantize_and_cache`` restates the call's rule block by block in IEEE float32:
scale ``max(a / qmax, 2^-64)`` for a block that the call begins, the stored scale
times the least sufficient power of two for one that already holds tokens, whose
codes then move to the new scale.  ``attend`` gathers the tokens a query sees and
applies softmax in float64.
"""
from __future__ import annotations

import numpy as np

from . import attention as OA
from . import fp8

QMAX = {"fp8_e4m3": np.float32(448), "int8": np.float32(127)}
MIN_SCALE = np.float32(2.0 ** -64)


def code_values(codes, kv_dtype) -> np.ndarray:
    """8-bit codes -> float32, exactly."""
    if kv_dtype == "fp8_e4m3":
        return fp8.decode(codes).astype(np.float32)
    return np.asarray(codes, dtype=np.int8).astype(np.float32)


def encode(x_f32, kv_dtype) -> np.ndarray:
    """float32 quotients -> codes: half to even, saturating."""
    if kv_dtype == "fp8_e4m3":
        return fp8.encode_f32(np.asarray(x_f32, dtype=np.float32))
    q = np.where(np.isnan(x_f32), np.float32(0), np.asarray(x_f32, dtype=np.float32))
    return np.clip(np.rint(q), -128, 127).astype(np.int8)


def grown_scale(s0, a, qmax):
    """(scale, k): the least k >= 0 with a <= qmax * s0 * 2^k."""
    k = 0
    s = np.float32(s0)
    with np.errstate(over="ignore"):
        while a > np.float32(qmax * s):
            s = np.float32(s * np.float32(2))
            k += 1
    return s, k


def quantize_and_cache(k_new, v_new, query_start, block_tables, context_lens, k_cache, v_cache,
                       k_scales, v_scales, src_dtype, kv_dtype):
    """In place; rows ``[T, Hkv, D]`` in the source storage type, caches
    ``[NB, bs, Hkv, D]`` codes, scales ``[NB, >= Hkv]`` float32."""
    bs, hkv = k_cache.shape[1], k_cache.shape[2]
    qmax = QMAX[kv_dtype]
    for s in range(len(context_lens)):
        q0, q1 = int(query_start[s]), int(query_start[s + 1])
        pos, end, row = int(context_lens[s]) - (q1 - q0), int(context_lens[s]), q0
        while pos < end:
            b, off = int(block_tables[s][pos // bs]), pos % bs
            m = min(bs - off, end - pos)
            for new, cache, scales in ((k_new, k_cache, k_scales), (v_new, v_cache, v_scales)):
                for h in range(hkv):
                    x = OA.to_f64(new[row:row + m, h], src_dtype).astype(np.float32)
                    fin = np.abs(x[np.isfinite(x)])
                    a = fin.max() if fin.size else np.float32(0)
                    s0 = scales[b, h]
                    if off == 0 or not (s0 >= MIN_SCALE) or np.isinf(s0):
                        sc = max(np.float32(a / qmax), MIN_SCALE)
                    else:
                        sc, k = grown_scale(s0, a, qmax)
                        if k:
                            old = code_values(cache[b, :off, h], kv_dtype)
                            cache[b, :off, h] = encode(np.ldexp(old, -k).astype(np.float32), kv_dtype)
                    scales[b, h] = sc
                    with np.errstate(over="ignore", invalid="ignore"):
                        cache[b, off:off + m, h] = encode((x / sc).astype(np.float32), kv_dtype)
            pos, row = pos + m, row + m


def gather(cache, scales, table, first, n, kv_dtype) -> np.ndarray:
    """Positions first .. first + n - 1 as float32 ``[n, Hkv, D]``: code * scale, one
    float32 product (scales ``[NB, >= Hkv]``, ``[Hkv]``, or None for f32 / bf16 caches)."""
    bs, hkv, d = cache.shape[1:]
    out = np.zeros((n, hkv, d), dtype=np.float32)
    for i in range(n):
        b, off = int(table[(first + i) // bs]), (first + i) % bs
        if kv_dtype in ("f32", "bf16"):
            out[i] = OA.to_f64(cache[b, off], kv_dtype).astype(np.float32)
        else:
            s = scales if scales.ndim == 1 else scales[b, :hkv]
            out[i] = code_values(cache[b, off], kv_dtype) * s[:, None].astype(np.float32)
    return out


def visible(pos, window, sinks) -> np.ndarray:
    """Tokens the query at position ``pos`` sees."""
    t = np.arange(pos + 1)
    if window == 0:
        return t
    return t[(t > pos - window) | (t < sinks)]


def attend(q, positions, K, V, scale, window, sinks):
    """``q [n, Hq, D]`` float64 at ``positions``; ``K``, ``V [L, Hkv, D]`` float64.
    Returns ``out`` and ``A = sum p |v|`` (for error bounds), each ``[n, Hq, D]``, and the
    largest ``sum_d |q_d k_d|`` of each (query, head)."""
    n, hq, d = q.shape
    g = hq // K.shape[1]
    out, mag = np.zeros((n, hq, d)), np.zeros((n, hq, d))
    reach = np.zeros((n, hq))
    for i, pos in enumerate(positions):
        t = visible(int(pos), window, sinks)
        for h in range(hq):
            k, v = K[t, h // g], V[t, h // g]
            z = float(np.float32(scale)) * (k @ q[i, h])
            p = np.exp(z - z.max())
            p /= p.sum()
            out[i, h], mag[i, h] = p @ v, p @ np.abs(v)
            reach[i, h] = (np.abs(k) @ np.abs(q[i, h])).max()
    return out, mag, reach
