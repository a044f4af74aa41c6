"""The step around the cache without a GPU: refusals of its calls (every argument is checked
before a launch), the frequencies of rotary positions, and pins of the oracle."""
import ctypes as C
import math
import os
import subprocess

import numpy as np
import pytest
import torch

from oracle import block_scaled as OB
from oracle import step as OS
from oracle import pool as OP

OK, INVALID, UNSUPPORTED = 0, 1, 5
PTR = C.c_void_p(1 << 20)      # aligned, never dereferenced: the calls below are refused first


def at(n):
    return C.c_void_p((1 << 20) + n)


def slots(lib, **kw):
    a = dict(bt=at(0), ctx=at(0x100), new=at(0x200), free=at(0x300), fs=at(0x400), S=2, T=8, F=5, nb=10, bs=16,
             mb=4, per_row=0, held=0, slots=at(0x500), pos=at(0x600), qs=at(0x700), co=at(0x800), fn=at(0x900),
             status=None)
    a.update(kw)
    return lib.library().slots_from_lengths(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(S=-1), INVALID), (dict(T=-1), INVALID), (dict(F=-1), INVALID), (dict(nb=0), INVALID),
    (dict(bs=0), INVALID), (dict(mb=0), INVALID), (dict(per_row=2), INVALID), (dict(held=-1), INVALID),
    (dict(per_row=1, T=1), INVALID), (dict(mb=1 << 28), INVALID), (dict(nb=1 << 31), UNSUPPORTED),
    (dict(bt=None), INVALID), (dict(ctx=None), INVALID), (dict(free=None), INVALID),
    (dict(slots=None), INVALID), (dict(slots=C.c_void_p(4)), INVALID), (dict(ctx=C.c_void_p(2)), INVALID),
    (dict(fn=C.c_void_p(1)), INVALID), (dict(qs=C.c_void_p(6)), INVALID)])
def test_slots_refusals(lib, kw, want):
    assert slots(lib, **kw) == want


@pytest.mark.parametrize("kw", [
    dict(co=at(0x200)), dict(co=at(0x104)), dict(co=at(0xFC)), dict(co=at(0x400)), dict(fn=at(0x104)),
    dict(fn=at(0x200)), dict(fn=at(0x310)), dict(bt=at(0xE4)), dict(bt=at(0x30C)), dict(slots=at(0x1C8)),
    dict(pos=at(0x51C)), dict(qs=at(0xF8)), dict(qs=at(0x804)), dict(co=at(0x700)), dict(fn=at(0x61C)),
    dict(status=at(0x104)), dict(status=at(0x01C)), dict(status=at(0x800)), dict(pos=at(0x200), new=at(0x21C))])
def test_slots_outputs_overlap_nothing(lib, kw):
    """8 bytes of lengths, 32 of tables, positions and 64 of slots: by one element, from either side."""
    assert slots(lib, **kw) == INVALID


def rotary(lib, **kw):
    a = dict(q=PTR, k=PTR, v=PTR, q_out=PTR, k_out=PTR, num_tokens=4, num_q_heads=4, num_kv_heads=2,
             head_dim=64, src_dtype=1, turns=PTR, positions=PTR, rotary_dim=64, num_axes=1, adjacent=0,
             scale=1.0, slot_mapping=PTR, k_cache=PTR, v_cache=PTR, block_size=16, num_blocks=4, cache_dtype=1)
    a.update(kw)
    for n in ("q", "k", "v", "q_out", "k_out"):
        a.setdefault(f"{n}_token_stride", 1024)
        a.setdefault(f"{n}_head_stride", 64)
    a = {n: v.value if isinstance(v, C.c_void_p) else v for n, v in a.items()}
    return lib.library().rotary_and_cache(C.byref(lib._RotaryArgs(**a)), None)


@pytest.mark.parametrize("kw,want", [
    (dict(num_tokens=-1), INVALID), (dict(num_kv_heads=0), INVALID), (dict(num_q_heads=-1), INVALID),
    (dict(head_dim=0), INVALID), (dict(rotary_dim=66), INVALID), (dict(rotary_dim=7), INVALID),
    (dict(rotary_dim=-2), INVALID), (dict(num_axes=0), INVALID), (dict(adjacent=2), INVALID),
    (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID), (dict(src_dtype=2), UNSUPPORTED),
    (dict(cache_dtype=0), UNSUPPORTED), (dict(src_dtype=0, cache_dtype=1), UNSUPPORTED),
    (dict(cache_dtype=2), INVALID), (dict(cache_dtype=3, k_scale=PTR), INVALID),
    (dict(block_size=0), INVALID), (dict(num_blocks=0), INVALID), (dict(num_blocks=1 << 62), UNSUPPORTED),
    (dict(k=None), INVALID), (dict(q=None), INVALID), (dict(q_out=None), INVALID), (dict(v=None), INVALID),
    (dict(v_cache=None), INVALID), (dict(slot_mapping=None), INVALID), (dict(turns=None), INVALID),
    (dict(positions=None), INVALID), (dict(k_cache=None, k_out=None), INVALID),
    (dict(q=C.c_void_p(1 + (1 << 20))), INVALID), (dict(k_cache=C.c_void_p(8 + (1 << 20))), INVALID),
    (dict(turns=C.c_void_p(4 + (1 << 20))), INVALID), (dict(slot_mapping=C.c_void_p(4)), INVALID),
    (dict(positions=C.c_void_p(2)), INVALID), (dict(num_tokens=0), OK)])
def test_rotary_refusals(lib, kw, want):
    assert rotary(lib, **kw) == want
    assert lib.library().rotary_and_cache(None, None) == INVALID


def apart(**kw):
    """Arguments whose arrays lie apart: 4 tokens of 4 + 2 + 2 heads of 64 in one projection's bf16 rows."""
    a = dict(q=at(0), k=at(512), v=at(768), q_out=at(0x10000), k_out=at(0x20000), turns=at(0x30000),
             positions=at(0x31000), slot_mapping=at(0x32000), k_cache=at(0x40000), v_cache=at(0x50000),
             axis=at(0x33000), q_token_stride=512, k_token_stride=512, v_token_stride=512,
             q_out_token_stride=256, k_out_token_stride=128)
    return {**a, **kw}


@pytest.mark.parametrize("kw", [
    dict(q_out=at(2)), dict(q_out=at(512)), dict(q_out=at(512 - 126)), dict(q_out=at(768)), dict(k_out=at(768)),
    dict(q_out=at(0), q_out_token_stride=520), dict(q_out=at(0)), dict(k_out=at(0)), dict(k_out=at(512)),
    dict(k_out=at(512 + 128), k_out_token_stride=512), dict(k_out=at(512 - 2), k_out_token_stride=512),
    dict(q_out=at(1024 - 128), q_out_token_stride=512), dict(q_out=at(0x10000), k_out=at(0x10000 + 2048 - 2)),
    dict(v_cache=at(0x40000)), dict(v_cache=at(0x40000 + 16 * 4 * 256 - 16)), dict(k_cache=at(0x10000 - 0x3FF0)),
    dict(q_out=at(0x40000 - 2046)), dict(k_out=at(0x50000 + 16 * 4 * 256 - 2)), dict(k=at(0x40000)),
    dict(q_out=at(0x30000 - 2046)), dict(q_out=at(0x30000 + 32 * 8 - 4)), dict(q_out=at(0x31000 + 12)),
    dict(k_out=at(0x32000 + 28)), dict(q_out=at(0x33000 + 32 * 4 - 4)), dict(device_status=at(0x40004)),
    dict(cache_dtype=2, k_scale=at(0x34000), v_scale=at(0x35000), k_out=at(0x34004)),
    dict(cache_dtype=2, k_scale=at(0x34000), v_scale=at(0x50000)), dict(src_dtype=0, cache_dtype=0, q_out=at(0x20000 - 4092))])
def test_rotary_outputs_overlap_nothing(lib, kw):
    """By one element or aligned unit, from either side; in place only where it is the same rows."""
    assert rotary(lib, **apart(**kw)) == INVALID


def test_rotary_cache_bytes(lib):
    assert rotary(lib, **apart(num_blocks=1 << 52, num_kv_heads=1 << 20)) == UNSUPPORTED


def test_rows_that_meet(tmp_path):
    """The check of strided rows against every byte of them, and its answer where strides are huge."""
    src = tmp_path / "meet.cpp"
    src.write_text('''
#include "ranges.cuh"
extern "C" int meets(const long long* x, const long long* y, int budget) {
  auto of = [](const long long* a) {
    return pkv::Rows(reinterpret_cast<const void*>(a[0]), a[1], a[2], a[3], a[4], a[5]);
  };
  return pkv::meet(of(x), of(y), budget);
}
''')
    so = tmp_path / "meet.so"
    csrc = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_295_gb300", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-shared", "-fPIC", f"-I{csrc}", str(src), "-o", str(so)],
                   check=True)
    fn = C.CDLL(str(so)).meets

    def meets(x, y, budget=4096):
        return fn((C.c_longlong * 6)(*x), (C.c_longlong * 6)(*y), budget)

    rng = np.random.default_rng(0)
    seen = [0, 0]
    for trial in range(6000):
        sets = []
        for _ in range(2):
            rows, heads, n = (int(z) for z in rng.integers(1, (6, 5, 9)))
            ts, hs = (int(z) for z in rng.integers(-40, 120, 2))
            if trial % 2 and sets:
                ts, hs = sets[0][3:5]
            sets.append((int(rng.integers(2000, 2300)), rows, heads, ts, hs, n))
        byte = [{b + i * ts + j * hs + e for i in range(r) for j in range(h) for e in range(n)}
                for b, r, h, ts, hs, n in sets]
        want = int(bool(byte[0] & byte[1]))
        assert meets(*sets) == want, sets
        assert meets(*sets, 1) >= want
        seen[want] += 1
    assert min(seen) > 1000
    far = (4096, 2 ** 31 - 1, 2 ** 20, 2 ** 62, 2 ** 62 - 1, 4096)
    assert meets(far, (4096 + 4095, 1, 1, 0, 0, 1)) and not meets(far, (4096 + 4096, 1, 1, 0, 0, 1))
    qkv = 10240 * 2       # 8,192 tokens of 32 + 4 + 4 heads of 256 bytes, and the three parts of each head
    parts = [(1 << 30, 8192, 32, qkv // 2, 256, 256), ((1 << 30) + 8192, 8192, 4, qkv // 2, 256, 256)]
    assert not meets(*parts, 8) and meets(parts[0], ((1 << 30) + 8191, *parts[1][1:]), 8)
    parts = [((1 << 30) + 256 * i, 8192, 32, 32 * 768, 768, 256) for i in range(3)]
    assert not meets(parts[0], parts[1], 8) and not meets(parts[2], parts[0], 8)
    assert meets(parts[0], (parts[1][0] - 1, *parts[1][1:]), 8)
    for none in ((0, 4, 4, 64, 64, 64), (4096, 0, 4, 64, 64, 64), (4096, 4, 4, 64, 64, 0)):
        assert not meets(none, (4096, 4, 4, 64, 64, 64))


def packed(lib, **kw):
    a = dict(q=at(0), k=at(0x10000), v=at(0x20000), out=at(0x30000), query_start=at(0x40000), key_start=at(0x50000),
             num_seqs=2, num_tokens=8, num_keys=8, num_q_heads=4, num_kv_heads=2, head_dim=64, scale=0.1, causal=1, window=0, sinks=0,
             q_dtype=1, kv_dtype=1, out_dtype=1)
    for n in ("q", "k", "v"):
        a[f"{n}_token_stride"], a[f"{n}_head_stride"] = 256, 64
    a.update(kw)
    a = {n: v.value if isinstance(v, C.c_void_p) else v for n, v in a.items()}
    return lib.library().packed_attention_prefill(C.byref(lib._PackedPrefillArgs(**a)), None)


@pytest.mark.parametrize("kw,want", [
    (dict(num_seqs=-1), INVALID), (dict(num_tokens=-1), INVALID), (dict(num_keys=-1), INVALID),
    (dict(num_q_heads=5), INVALID), (dict(num_kv_heads=0), INVALID), (dict(head_dim=0), INVALID),
    (dict(causal=2), INVALID), (dict(window=-1), INVALID), (dict(window=5, causal=0), INVALID),
    (dict(sinks=3), INVALID), (dict(scale=math.nan), INVALID), (dict(q_dtype=0), UNSUPPORTED),
    (dict(kv_dtype=2), UNSUPPORTED), (dict(out_dtype=2), UNSUPPORTED), (dict(head_dim=136), UNSUPPORTED),
    (dict(head_dim=68), UNSUPPORTED), (dict(num_q_heads=258), UNSUPPORTED),
    (dict(q_token_stride=0), INVALID), (dict(k_head_stride=-64), INVALID), (dict(v_token_stride=260), INVALID),
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(out=None), INVALID),
    (dict(query_start=None), INVALID), (dict(key_start=None, num_keys=9), INVALID),
    (dict(q=C.c_void_p(8)), INVALID), (dict(out=C.c_void_p(8)), INVALID), (dict(key_start=C.c_void_p(2)), INVALID),
    (dict(num_seqs=0), OK), (dict(num_tokens=0), OK)])
def test_packed_refusals(lib, kw, want):
    assert packed(lib, **kw) == want
    assert lib.library().packed_attention_prefill(None, None) == INVALID


def test_status_words_off_their_boundary(lib):
    """Four bytes that are flagged atomically: refused where they begin between two words."""
    assert slots(lib, status=at(0xA02)) == INVALID
    assert rotary(lib, **apart(device_status=at(0x36001))) == INVALID
    assert packed(lib, device_status=at(0x60002)) == INVALID


def test_packed_check(lib):
    """The check alone answers as the call does, without a launch: these arguments are taken."""
    a = dict(q=at(0), k=at(0x10000), v=at(0x20000), out=at(0x30000), query_start=at(0x100000), num_seqs=2,
             num_tokens=8, num_keys=8, num_q_heads=4, num_kv_heads=2, head_dim=64, scale=0.1, causal=1, q_dtype=1,
             kv_dtype=1, out_dtype=1)
    for n in ("q", "k", "v"):
        a[f"{n}_token_stride"], a[f"{n}_head_stride"] = 256, 64

    def check(**kw):
        b = {n: v.value if isinstance(v, C.c_void_p) else v for n, v in {**a, **kw}.items()}
        return lib.library().packed_attention_prefill_check(C.byref(lib._PackedPrefillArgs(**b)))

    for kw in ({}, dict(out_dtype=0), dict(window=2 ** 31 - 1, sinks=2 ** 31 - 1), dict(causal=0),
               dict(key_start=at(0x110000), num_keys=3), dict(num_seqs=0, q=None), dict(num_q_heads=256)):
        assert check(**kw) == OK, kw
    for parts in (0, 1, 2):
        assert check(weight_parts=parts) == OK
    assert check(weight_parts=2, out_dtype=0) == OK and check(weight_parts=1, out_dtype=0) == UNSUPPORTED
    assert check(weight_parts=3) == INVALID and check(weight_parts=-1) == INVALID
    # as the C compiler lays the arguments out
    assert lib._PackedPrefillArgs.device_status.offset == 152 and C.sizeof(lib._PackedPrefillArgs) == 168
    no = dict(q_token_stride=0, q_head_stride=0, k_token_stride=0, k_head_stride=0, v_token_stride=0, v_head_stride=3)
    assert check(num_tokens=0, num_keys=0, **no) == OK      # no rows: whatever their strides are
    assert check(key_start=at(0x110000), num_keys=0, k_head_stride=0, v_token_stride=-1, k=None, v=None) == OK
    for n, status in ((0x60000, OK), (0x31000, OK), (0x60002, INVALID), (0x30FFC, INVALID), (0x2FFFC, INVALID)):
        assert check(context_lens=at(n)) == status
    for kw in (dict(window=-1), dict(sinks=1), dict(out=at(0)), dict(v=at(8)), dict(num_keys=9),
               dict(v_token_stride=260), dict(window=4, causal=0)):
        assert check(**kw) == INVALID, kw
    for kw in (dict(num_q_heads=258), dict(head_dim=136), dict(out_dtype=2), dict(num_tokens=2 ** 30 + 1),
               dict(num_seqs=2 ** 24, num_q_heads=128, num_kv_heads=64)):
        assert check(**kw) == UNSUPPORTED, kw
    assert lib.library().packed_attention_prefill_check(None) == INVALID


@pytest.mark.parametrize("kw", [
    dict(out=at(0)), dict(out=at(0x10000)), dict(out=at(0x20000 - 0xFF0)), dict(out=at(0x20000 + 7 * 512 + 240)),
    dict(out=at(0x40000 - 0xFF0)), dict(key_start=at(0x30FFC)),
    dict(out=at(0x10000), num_tokens=1, num_keys=1)])
def test_packed_output_overlaps_no_input(lib, kw):
    """Rows of 4 heads (512 bytes) for q and of 2 (256 of 512) for k and v, 4,096 bytes of output."""
    assert packed(lib, **kw) == INVALID


def test_python_refusals(lib):
    S, T = 2, 4
    i32 = dict(dtype=torch.int32)
    bt, ctx, free = torch.zeros((S, 3), **i32), torch.ones(S, **i32), torch.arange(4, **i32)

    def sl(**kw):
        a = dict(block_tables=bt, context_lens=ctx, new_lens=ctx, free_blocks=free, num_blocks=8, block_size=16,
                 num_tokens=T)
        a.update(kw)
        lib.slots_from_lengths(**a)

    for kw in (dict(), dict(context_lens=ctx.long()), dict(new_lens=ctx[:1]), dict(block_tables=bt[:1]),
               dict(free_blocks=free.float()), dict(free_start=free), dict(num_tokens=None),
               dict(num_tokens=-1), dict(context_lens=None), dict(block_size="x"), dict(num_blocks=1.5)):
        with pytest.raises(ValueError):      # the first: no CPU path
            sl(**kw)
    q, k = torch.zeros((T, 4, 64)), torch.zeros((T, 2, 64))
    plan = lib.Rotary(64, device="cpu")

    def ro(**kw):
        a = dict(q=q, k=k, v=k, positions=torch.zeros(T, **i32), rotary=plan)
        a.update(kw)
        lib.rotary_and_cache(**a)

    for kw in (dict(), dict(q=q.half(), k=k.half()), dict(k=None), dict(k=k[0]), dict(q=q[0]), dict(positions=None)):
        with pytest.raises(ValueError):
            ro(**kw)

    def pa(**kw):
        a = dict(q=q.bfloat16(), k=k.bfloat16(), v=k.bfloat16(), query_start=torch.zeros(S + 1, **i32), scale=0.1)
        a.update(kw)
        lib.packed_attention_prefill(**a)

    for kw in (dict(), dict(q=q), dict(k=None), dict(query_start=torch.zeros(0, **i32)), dict(scale="x"),
               dict(window="x"), dict(out_dtype="bf16"), dict(v=k)):
        with pytest.raises((ValueError, TypeError)):
            pa(**kw)


def test_rotary_plan_refusals(lib):
    for kw in (dict(rotary_dim=7), dict(rotary_dim=-2), dict(rotary_dim=8, sections=[1, 2]),
               dict(rotary_dim=8, sections=[5, -1]), dict(rotary_dim=8, sections=[4], axes=[0] * 4),
               dict(rotary_dim=8, axes=[0, 1]), dict(rotary_dim=4, axes=[0, -1]),
               dict(rotary_dim=8, inv_freq=[1.0, 2.0])):
        with pytest.raises(ValueError):
            lib.Rotary(device="cpu", **kw)
    with pytest.raises(lib.PagedKVError):
        lib.Rotary(4, inv_freq=[1.0, math.inf], device="cpu")
    p = lib.Rotary(8, sections=[1, 0, 3], device="cpu")
    assert p.num_axes == 3 and p.axis.tolist() == [0, 2, 2, 2]
    p = lib.Rotary(4, axes=[1, 0], inv_freq=torch.tensor([1.0, 0.5]), device="cpu")
    assert p.num_axes == 2 and p.axis.tolist() == [1, 0]
    assert lib.Rotary(0, device="cpu").turns.numel() == 0


def test_rotary_turns(lib):
    """position * turns modulo 2^64 is the angle modulo one turn: to 2^-52 of the frequency's
    turns times the position (a double's rounding of the quotient and of 2 pi), any sign."""
    freq = np.concatenate([10000.0 ** (-np.arange(64) / 64), [0.0, -0.3, 7.5, 2 * math.pi, 1e-30, -1e-30]])
    turns = np.empty(freq.size, dtype=np.uint64)
    assert lib.library().rotary_turns(lib._np_ptr(freq), freq.size, lib._np_ptr(turns)) == OK
    from fractions import Fraction
    # 2 pi to 60 digits
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459")
    for f, t in zip(freq.tolist(), turns.tolist()):
        for pos in (0, 1, -1, 77, 1000003, -123456, 2 ** 31 - 1, -2 ** 31):
            got = Fraction(pos * t % 2 ** 64, 2 ** 64)
            off = (got - pos * Fraction(f) / two_pi) % 1
            off = min(off, 1 - off)
            # half a step of a double in the quotient, one in 2 pi, and the cut to 2^-64
            assert off <= abs(pos) * (abs(Fraction(f)) / two_pi * Fraction(3, 2 ** 53) + Fraction(2, 2 ** 64)
                                      + Fraction(1, 2 ** 53) * (1 if f < 0 else 0)), (f, pos)


def test_oracle_slots_are_the_pools():
    """The same blocks and slots as the pool's appends, sequence after sequence."""
    rng = np.random.default_rng(5)
    for bs in (1, 3, 16):
        pool = OP.Pool(1, 1, 16, bs, 2, 200, initial_free_order=rng.permutation(200).tolist())
        for s in range(4):
            pool.seq_create(s)
            pool.seq_append_tokens(s, int(rng.integers(0, 3 * bs + 1)))
        tables, lens = pool.padded_tables(range(4), 60)
        new = rng.integers(0, 4 * bs + 2, 4)
        free = list(pool.free)
        t, slot, pos, start, out, at, flags = OS.slots(tables, lens, new, free, 0, bs, int(new.sum()) + 2, 200,
                                                       first_block_held=True)
        want = [x for s in range(4) for x in pool.seq_append_tokens(s, int(new[s]))]
        assert slot.tolist() == want + [-1, -1] and not flags
        assert (t == np.asarray(pool.padded_tables(range(4), 60)[0])).all()
        assert list(pool.free) == free[at:]
        assert out.tolist() == [pool.lens[s] for s in range(4)] and start.tolist() == [0, *np.cumsum(new)]


def test_oracle_rotary():
    """Turning keeps lengths, turns add up, and several axes at one position are one axis."""
    rng = np.random.default_rng(2)
    x, freq = rng.standard_normal((5, 3, 12)), 100.0 ** (-np.arange(4) / 4)
    pos = rng.integers(0, 1000, 5)
    for adjacent in (False, True):
        y = OS.rotary(x, pos, freq, adjacent=adjacent)
        assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
        assert np.array_equal(y[..., 8:], x[..., 8:])
        assert np.allclose(OS.rotary(y, -pos, freq, adjacent=adjacent), x)
        three = OS.rotary(x, np.stack([pos] * 3), freq, axes=[0, 2, 1, 2], adjacent=adjacent)
        assert np.array_equal(three, y)
    z = OS.rotary(np.ones((1, 1, 2)), [1], [math.pi / 2])
    assert np.allclose(z, [[[-1.0, 1.0]]])


def test_oracle_packed_is_the_windowed_one():
    rng = np.random.default_rng(3)
    q, k, v = (rng.standard_normal((9, h, 8)) for h in (4, 2, 2))
    for window, sinks in ((0, 0), (3, 1)):
        out, mag, reach, seen = OS.packed(q, k, v, [0, 4, 4, 9], [0, 4, 4, 9], 0.3, True, window, sinks)
        for a, b in ((0, 4), (4, 9)):
            o, m, r = OB.attend(q[a:b], np.arange(b - a), k[a:b], v[a:b], 0.3, window, sinks)
            assert np.allclose(out[a:b], o) and np.allclose(mag[a:b], m) and np.allclose(reach[a:b], r)
    out, _, _, seen = OS.packed(q[:4], k, v, [0, 4], [0, 2], 0.3)      # two queries before every key
    assert seen.tolist() == [0, 0, 1, 2] and (out[:2] == 0).all() and np.allclose(out[2], v[0].repeat(2, 0))
