"""Rotary positions with the append, against float64."""
import numpy as np
import pytest

from oracle import step as OS
from tests import gpu_cases as GC

pytestmark = pytest.mark.gpu


def bound(x, plan, y, adjacent, scale):
    """Elementwise bound on the float32 result.  cos and sin are off by less than 2^-23 (one unit of
    their last place), times the factor by 2^-24 more; the two products and their sum by 2^-24 of each
    product: 2^-22 together and rounded up to 2^-21."""
    half = plan.rotary_dim // 2
    e = np.zeros(y.shape)
    a, b = (np.s_[..., 0:2 * half:2], np.s_[..., 1:2 * half:2]) if adjacent else \
        (np.s_[..., :half], np.s_[..., half:2 * half])
    both = abs(scale) * (np.abs(x[a]) + np.abs(x[b])) * 2.0 ** -21
    e[a], e[b] = both, both
    return e


def rounded(y, e, dtype):
    import torch
    return e + (np.abs(y) + e) * (2.0 ** -8 if dtype == torch.bfloat16 else 2.0 ** -24)


def f64(t):
    return t.double().cpu().numpy()


def run(lib, seed, T, hq, hkv, dim, rot, dtype, kv="", axes=1, adjacent=False, scale=1.0, far=5000, keep_k=False,
        layout="fused", place=False, bs=16, sections=None):
    """One call on random rows, checked whole: q, k, both caches, rows that are not appended."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rng = np.random.default_rng(seed)

    def rows(h):
        return torch.randn((T, h, dim), generator=gen, device="cuda").to(dtype)

    if layout == "fused":            # parts of one projection's rows
        qkv = rows(hq + 2 * hkv)
        q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    elif layout == "odd":            # rows that begin on no 16-byte boundary
        flat = torch.randn(T * (hq + 2 * hkv) * (dim + 1) + 1, generator=gen, device="cuda").to(dtype)
        all_ = flat[1:].view(T, hq + 2 * hkv, dim + 1)[..., :dim]
        q, k, v = all_[:, :hq], all_[:, hq:hq + hkv], all_[:, hq + hkv:]
    else:
        q, k, v = rows(hq), rows(hkv), rows(hkv)
    half = rot // 2
    freq = 10000.0 ** (-np.arange(half) / max(half, 1))
    ax = None if axes == 1 else rng.integers(0, axes, half)
    if ax is not None and half:
        ax[-1] = axes - 1
    plan = lib.Rotary(rot, axes=ax, adjacent=adjacent, scale=scale)
    num_axes = plan.num_axes
    pos = rng.integers(-far // 4, far, (num_axes, T)).astype(np.int32)
    pd = torch.from_numpy(pos if num_axes > 1 else pos[0]).cuda()
    x = {n: f64(t) for n, t in (("q", q), ("k", k), ("v", v))}
    want, err = {}, {}
    for n in ("q", "k"):
        want[n] = OS.rotary(x[n], pos, freq, ax, adjacent, scale)
        err[n] = bound(x[n], plan, want[n], adjacent, scale)
    want["v"], err["v"] = x["v"], np.zeros(x["v"].shape)
    kw, cache = {}, {}
    nb = -(-T // bs) + 2
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if kv:
        slots = rng.permutation(nb * bs)[:T].astype(np.int64)
        slots[::5] = -1 - slots[::5]          # every fifth token is not appended
        types = {"same": dtype, "fp8": torch.float8_e4m3fn, "int8": torch.int8}
        for n in ("k", "v"):
            c = torch.randn((nb, bs, hkv, dim), generator=gen, device="cuda") * 30
            cache[n] = c.to(types[kv])
        before = {n: c.clone() for n, c in cache.items()}
        kw = dict(slot_mapping=torch.from_numpy(slots).cuda(), k_cache=cache["k"], v_cache=cache["v"])
        if kv != "same":
            sc = {n: (rng.uniform(0.5, 2.0, hkv) * 2.5 / (448 if kv == "fp8" else 127)).astype(np.float32)
                  for n in ("k", "v")}
            kw.update(k_scale=torch.from_numpy(sc["k"]).cuda(), v_scale=torch.from_numpy(sc["v"]).cuda())
    if place:
        kw.update(q_out=q, k_out=k)
    v_before = v.clone()
    got_q, got_k = lib.rotary_and_cache(q, k, v, pd, plan, keep_k=keep_k, device_status=status, **kw)
    assert int(status.item()) == 0
    if place:
        assert got_q is q and got_k is k or got_q.data_ptr() == q.data_ptr()
    assert torch.equal(v, v_before)
    assert (np.abs(f64(got_q) - want["q"]) <= rounded(want["q"], err["q"], dtype)).all()
    if not kv or keep_k or place:
        assert (np.abs(f64(got_k) - want["k"]) <= rounded(want["k"], err["k"], dtype)).all()
    else:
        assert got_k is None
    if not place:
        assert np.array_equal(f64(q), x["q"]) and np.array_equal(f64(k), x["k"])
    for n, c in cache.items():
        bits = (lambda t: t.view(torch.uint8) if t.element_size() == 1 else t)
        flat, old = bits(c).flatten(0, 1), bits(before[n]).flatten(0, 1)
        rest = np.ones(nb * bs, dtype=bool)
        rest[slots[slots >= 0]] = False
        at = torch.from_numpy(np.flatnonzero(rest)).cuda()
        assert torch.equal(flat[at], old[at])
        there = slots >= 0
        val = c.flatten(0, 1) if kv != "fp8" else c.float().flatten(0, 1)
        val = f64(val[torch.from_numpy(slots[there]).cuda()])
        y, e = want[n][there], err[n][there]
        if kv == "same":
            assert (np.abs(val - y) <= rounded(y, e, dtype)).all()
            continue
        s = sc[n].astype(np.float64)[None, :, None]
        z, e = y / s, e / s + np.abs(y / s) * 2.0 ** -23
        if kv == "fp8":     # half a step: 2^-4 of the value, or of the smallest normal's 2^-6 2^-3
            top, step = 448.0, np.maximum((np.abs(z) + e) * 2.0 ** -4, 2.0 ** -10)
        else:
            top, step = 127.0, 0.5
            z = np.maximum(z, -128.0)
        assert (np.abs(val - np.clip(z, -128.0 if kv == "int8" else -top, top)) <= step + e).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("dim,rot", [(64, 64), (128, 128), (128, 32), (80, 80), (80, 16), (256, 64), (96, 48),
                                     (8, 4), (6, 2), (7, 6), (64, 0), (128, 6), (72, 72), (1024, 512), (2056, 16)])
def test_rows(lib, dtype, adjacent, dim, rot):
    """Whole and part-rotated heads, sizes that 16-byte loads do not divide, without a cache."""
    import torch
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    run(lib, dim + rot, 11, 3, 2, dim, rot, dt, adjacent=adjacent)
    run(lib, dim + rot, 2, 1, 1, dim, rot, dt, adjacent=adjacent, layout="odd")


@pytest.mark.parametrize("kv", ["same", "fp8", "int8"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["fused", "odd"])
def test_append(lib, kv, dtype, layout):
    import torch
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    for T, hq, hkv, dim, rot, axes, adj in ((1, 4, 1, 128, 128, 1, False), (37, 8, 2, 128, 128, 3, False),
                                            (200, 3, 3, 80, 32, 2, True), (5, 7, 1, 64, 64, 1, True),
                                            (9, 40, 5, 96, 96, 3, False), (3, 2, 2, 48, 20, 1, False)):
        run(lib, T, T, hq, hkv, dim, rot, dt, kv=kv, axes=axes, adjacent=adj, layout=layout)
        run(lib, T, T, hq, hkv, dim, rot, dt, kv=kv, axes=axes, adjacent=adj, keep_k=True, scale=1.25,
            layout="own" if layout == "fused" else layout, bs=3)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_in_place(lib, dtype):
    import torch
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    for dim, rot, adj, layout in ((128, 128, False, "fused"), (80, 32, True, "fused"), (128, 128, False, "odd"),
                                  (64, 24, False, "own")):
        run(lib, 5, 67, 6, 2, dim, rot, dt, adjacent=adj, layout=layout, place=True)
        run(lib, 6, 67, 6, 2, dim, rot, dt, kv="same", adjacent=adj, layout=layout, place=True)


def test_far_positions(lib):
    """The largest and smallest positions: 2^31 times half a step of the frequency's turns (2^-53,
    twice: the quotient and 2 pi) is 2^-20 of a turn; up to a million nothing shows."""
    import torch
    run(lib, 1, 300, 2, 1, 128, 128, torch.float32, far=10 ** 6)
    plan = lib.Rotary(64)
    q = torch.randn((4, 1, 64), device="cuda")
    pos = np.array([2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, -1], dtype=np.int32)
    got, _ = lib.rotary_and_cache(q, q, None, torch.from_numpy(pos).cuda(), plan)
    want = OS.rotary(f64(q), pos, 10000.0 ** (-np.arange(32) / 32))
    x = np.abs(f64(q))
    size = x[..., :32] + x[..., 32:]
    e = np.concatenate([size, size], -1) * (2.0 ** -21 + np.abs(pos.astype(float))[:, None, None] * 2.0 ** -51)
    assert (np.abs(f64(got) - want) <= e).all()


def test_many_rows(lib):
    """Grids larger than a wave, more heads than a CTA's threads, few tokens with many heads."""
    import torch
    for T, hq, hkv in ((3000, 8, 2), (2, 512, 64), (1, 33, 1)):
        run(lib, T, T, hq, hkv, 128, 128, torch.bfloat16, kv="same", keep_k=True)


def test_only_k_and_no_tokens(lib):
    import torch
    plan = lib.Rotary(64)
    k = torch.randn((5, 2, 64), device="cuda")
    pos = torch.arange(5, dtype=torch.int32, device="cuda")
    q, out = lib.rotary_and_cache(None, k, None, pos, plan)
    assert q is None
    same, _ = lib.rotary_and_cache(k, k, None, pos, plan)
    assert torch.equal(out, same)
    q, out = lib.rotary_and_cache(k[:0], k[:0], None, pos[:0], plan)
    assert q.shape == out.shape == (0, 2, 64)


@pytest.mark.parametrize("odd", [False, True])
def test_bad_slots(lib, odd):
    """A slot past the cache is flagged and skipped; the other tokens are appended."""
    import torch
    plan = lib.Rotary(64)
    flat = torch.randn((6, 2, 65), device="cuda")
    k = flat[..., 1:] if odd else flat[..., :64].contiguous()
    pos = torch.arange(6, dtype=torch.int32, device="cuda")
    caches = [torch.zeros((2, 4, 2, 64), device="cuda") for _ in range(2)]
    slots = torch.tensor([0, 8, 2 ** 40, -1, -2 ** 50, 7], device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    q, kk = lib.rotary_and_cache(k, k, k, pos, plan, slots, *caches, keep_k=True, device_status=status)
    assert int(status.item()) == lib.DEV_BAD_SLOT
    assert torch.equal(caches[0].flatten(0, 1)[[0, 7]], kk[[0, 5]])
    assert torch.equal(caches[1].flatten(0, 1)[[0, 7]], k[[0, 5]])
    assert (caches[0].flatten(0, 1)[1:7] == 0).all() and (caches[1].flatten(0, 1)[1:7] == 0).all()


def test_values_that_are_not_finite(lib):
    """Infinities and NaN stay in their pair (and out of dims that do not turn)."""
    import torch
    plan = lib.Rotary(32)
    for view in (np.s_[..., :64], np.s_[..., 1:]):
        k = torch.randn((3, 1, 65), device="cuda")[view]
        clean, _ = lib.rotary_and_cache(k, k, None, torch.arange(3, dtype=torch.int32, device="cuda"), plan)
        k = k.clone() if view[1].start is None else k
        k[1, 0, 3], k[1, 0, 40], k[2, 0, 63] = float("nan"), float("inf"), float("-inf")
        got, _ = lib.rotary_and_cache(k, k, None, torch.arange(3, dtype=torch.int32, device="cuda"), plan)
        hit = torch.zeros_like(got, dtype=torch.bool)
        hit[1, 0, 3] = hit[1, 0, 19] = hit[1, 0, 40] = hit[2, 0, 63] = True
        assert torch.equal(got[~hit], clean[~hit])
        assert got[1, 0, [3, 19]].isnan().all() and got[1, 0, 40] == float("inf") and got[2, 0, 63] == -float("inf")


def test_refusals(lib):
    import torch
    plan, three = lib.Rotary(64), lib.Rotary(64, sections=[8, 12, 12])
    q = torch.zeros((4, 4, 64), device="cuda", dtype=torch.bfloat16)
    k = torch.zeros((4, 2, 64), device="cuda", dtype=torch.bfloat16)
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    caches = [torch.zeros((2, 4, 2, 64), device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    codes = [torch.zeros((2, 4, 2, 64), device="cuda", dtype=torch.int8) for _ in range(2)]
    slots = torch.arange(4, device="cuda")
    sc = torch.ones(2, device="cuda")

    def call(**kw):
        a = dict(q=q, k=k, v=k, positions=pos, rotary=plan, slot_mapping=slots, k_cache=caches[0],
                 v_cache=caches[1])
        a.update(kw)
        return lib.rotary_and_cache(a.pop("q"), a.pop("k"), a.pop("v"), a.pop("positions"), a.pop("rotary"), **a)

    call()
    for kw in (dict(q=q[:3]), dict(q=q.float()), dict(v=None), dict(v=k[:, :1]), dict(positions=pos.long()),
               dict(positions=pos[:3]), dict(rotary=three), dict(rotary=lib.Rotary(128)),
               dict(rotary=lib.Rotary(64, device="cpu")), dict(slot_mapping=None), dict(slot_mapping=pos),
               dict(slot_mapping=slots[:3]), dict(v_cache=None), dict(k_cache=None), dict(k_cache=codes[0], v_cache=codes[1]),
               dict(k_cache=codes[0], v_cache=codes[1], k_scale=torch.ones((2, 4), device="cuda"),
                    v_scale=torch.ones((2, 4), device="cuda")),
               dict(q=q.transpose(1, 2)[:, :, :4].transpose(1, 2)[..., ::2]), dict(q_out=torch.empty_like(q)[:2]),
               dict(k_out=torch.empty((4, 1, 64), device="cuda", dtype=torch.bfloat16).expand(4, 2, 64)),
               dict(q=q.cpu()), dict(device_status=sc)):
        with pytest.raises((ValueError, lib.PagedKVError)):
            call(**kw)
    with pytest.raises(lib.PagedKVError):
        call(q=q.float(), k=k.float(), v=k.float())       # float32 rows into a bfloat16 cache


def test_captured_and_on_another_stream(lib):
    import torch
    plan = lib.Rotary(128, sections=[16, 24, 24])
    q = torch.randn((40, 8, 128), device="cuda").bfloat16()
    pos = torch.arange(120, dtype=torch.int32, device="cuda").view(3, 40)
    want, _ = lib.rotary_and_cache(q, q, None, pos, plan)
    s, out = torch.cuda.Stream(), torch.empty_like(q)
    torch.cuda.synchronize()
    got, _ = lib.rotary_and_cache(q, q, None, pos, plan, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        lib.rotary_and_cache(q, q, None, pos, plan, q_out=out, k_out=out.clone())
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_outputs_that_overlap_themselves(lib):
    """Rows and heads of an output lie apart, whichever of the two is the outer one."""
    import torch
    plan = lib.Rotary(64)
    q = torch.randn((4, 3, 64), device="cuda").bfloat16()
    pos = torch.arange(4, dtype=torch.int32, device="cuda")
    want, _ = lib.rotary_and_cache(q, q, None, pos, plan)
    room = torch.empty(4096, device="cuda", dtype=torch.bfloat16)
    for strides in ((64, 64, 1), (128, 64, 1), (184, 64, 1), (64, 248, 1), (32, 512, 1), (0, 64, 1), (192, 0, 1)):
        bad = room.as_strided((4, 3, 64), strides)
        for kw in (dict(q_out=bad), dict(k_out=bad)):
            with pytest.raises(ValueError):
                lib.rotary_and_cache(q, q, None, pos, plan, **kw)
    for strides in ((192, 64, 1), (64, 256, 1), (200, 64, 1), (72, 284, 1)):
        out = room.as_strided((4, 3, 64), strides)
        assert lib.rotary_and_cache(q, q, None, pos, plan, q_out=out)[0] is not None
        assert torch.equal(out, want)


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_slots_past_32_bits(lib, kv):
    """The last blocks of a cache of more than 2^32 elements, and rows of a source far apart."""
    import torch
    bs, hkv, dim = 16, 8, 128
    nb = 2 ** 32 // (bs * hkv * dim) + 3 if kv == "int8" else 2 ** 31 // (bs * hkv * dim) + 3
    dt = torch.int8 if kv == "int8" else torch.bfloat16
    k_cache, v_cache = (torch.empty((nb, bs, hkv, dim), device="cuda", dtype=dt) for _ in range(2))
    small = [torch.empty((3, bs, hkv, dim), device="cuda", dtype=dt) for _ in range(2)]
    room = torch.empty((3, 2 ** 30), device="cuda", dtype=torch.bfloat16)
    x = room[:, -(2 + 2 * hkv) * dim:].view(3, -1, dim)
    x.copy_(torch.randn(x.shape, device="cuda"))
    q, k, v = x[:, :2], x[:, 2:2 + hkv], x[:, 2 + hkv:]
    plan, pos = lib.Rotary(dim), torch.tensor([5, 77, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    kw = dict(keep_k=True)
    if kv == "int8":
        kw.update(k_scale=torch.full((hkv,), 0.03, device="cuda"), v_scale=torch.full((hkv,), 0.03, device="cuda"))
    slots = torch.tensor([(nb - 1) * bs + 15, (nb - 2) * bs, (nb - 3) * bs + 7], device="cuda")
    a = lib.rotary_and_cache(q, k, v, pos, plan, slots, k_cache, v_cache, **kw)
    b = lib.rotary_and_cache(q.contiguous(), k.contiguous(), v.contiguous(), pos, plan, slots - (nb - 3) * bs, *small, **kw)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for big, few in ((k_cache, small[0]), (v_cache, small[1])):
        at = slots - (nb - 3) * bs
        assert torch.equal(big[-3:].view(-1, hkv, dim)[at], few.view(-1, hkv, dim)[at])


@pytest.mark.parametrize("kv", ["", "same", "fp8", "int8"])
@pytest.mark.parametrize("dim,rot", [(80, 40), (20, 8), (36, 28), (84, 84), (100, 48), (60, 0), (6, 4), (512, 8)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("adjacent", [False, True])
def test_halves_of_few_dims(lib, kv, dim, rot, dtype, adjacent):
    """Halves, heads and strides that are multiples of 8 bytes, or of less, and not of 16."""
    import torch
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    run(lib, dim + rot, 19, 5, 3, dim, rot, dt, kv, adjacent=adjacent, keep_k=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_outputs_that_overlap_inputs(lib, dtype):
    """Rows turned in place, parts of one projection's rows between others and parts of each head are taken; an
    output over another input, a cache or the other output is refused and nothing is written."""
    import torch
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    T, D, plan = 9, 64, lib.Rotary(64)
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    slots = torch.arange(T, device="cuda")
    pool = torch.zeros((2, 3, 4, 2, D), device="cuda", dtype=dt)

    def call(q, k, v, **kw):
        return lib.rotary_and_cache(q, k, v, pos, plan, slots, pool[0], pool[1], **kw)

    def views(layout):
        x = torch.randn((T, 2, 3, D) if layout == "heads" else (T, 6, D), device="cuda").to(dt)
        if layout == "heads":        # q, k and v of a head side by side
            return x, x[:, :, 0], x[:, :, 1], x[:, :, 2]
        return x, x[:, :2], x[:, 2:4], x[:, 4:]

    for layout in ("heads", "rows"):
        x, q, k, v = views(layout)
        want = call(q, k, v, keep_k=True)
        caches = pool.clone()
        for places in (dict(q_out=q, k_out=k), dict(q_out=q), dict(k_out=k)):
            y = x.clone()
            q2, k2, v2 = (y[:, :, i] for i in range(3)) if layout == "heads" else (y[:, :2], y[:, 2:4], y[:, 4:])
            pool.zero_()
            got = call(q2, k2, v2, keep_k=True, **{n: q2 if n == "q_out" else k2 for n in places})
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            assert torch.equal(v2, v) and torch.equal(pool, caches)
        # the rows of this step within those of a longer one
        room = torch.zeros((T, 12, D), device="cuda", dtype=dt)
        got = call(room[:, 2:4].copy_(q), room[:, 6:8].copy_(k), room[:, 10:12].copy_(v), q_out=room[:, :2],
                   k_out=room[:, 8:10])
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])

        x, q, k, v = views(layout)
        before, pool_before = x.clone(), pool.clone()
        own = torch.empty((T, 2, D), device="cuda", dtype=dt)
        for kw in (dict(q_out=k), dict(q_out=v), dict(k_out=q), dict(k_out=v), dict(q_out=own, k_out=own),
                   dict(k_out=pool[0].view(-1, 2, D)[:T]), dict(q_out=pool[1].view(-1, 2, D)[1:T + 1])):
            with pytest.raises((ValueError, lib.PagedKVError)):
                call(q, k, v, **kw)
        with pytest.raises((ValueError, lib.PagedKVError)):
            lib.rotary_and_cache(q, k, v, pos, plan, slots, pool[0], pool[0])
        torch.cuda.synchronize()
        assert torch.equal(x, before) and torch.equal(pool, pool_before)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "int8"])
def test_only_k_into_a_cache(lib, kv):
    """Without q the caches and the turned k are what they are with it; one token of any token stride too."""
    import torch
    T, D, plan = 21, 80, lib.Rotary(40)
    dt = {"bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn, "int8": torch.int8}[kv]
    x = torch.randn((T, 8, D), device="cuda").bfloat16()
    q, k, v = x[:, :4], x[:, 4:6], x[:, 6:]
    pos, slots = torch.arange(T, dtype=torch.int32, device="cuda") * 977, torch.randperm(32, device="cuda")[:T]
    sc = {} if kv == "bf16" else {n: torch.tensor([0.02, 0.05], device="cuda") for n in ("k_scale", "v_scale")}

    def call(q, k, v, pos, slots):
        caches = [torch.zeros((2, 16, 2, D), device="cuda").to(dt) for _ in range(2)]
        got = lib.rotary_and_cache(q, k, v, pos, plan, slots, *caches, keep_k=True, **sc)
        return (*got, *(c.view(torch.uint8) for c in caches))

    want = call(q, k, v, pos, slots)
    got = call(None, k, v, pos, slots)
    assert got[0] is None and all(torch.equal(a, b) for a, b in zip(got[1:], want[1:]))
    for t in (0, 20):
        a = call(q[t:t + 1], k[t:t + 1], v[t:t + 1], pos[t:t + 1], slots[t:t + 1])
        far = [y[t:t + 1].as_strided((1, y.shape[1], D), (7, D, 1)) for y in (q, k, v)]
        b = call(*far, pos[t:t + 1], slots[t:t + 1])
        assert all(torch.equal(c, d) for c, d in zip(a, b))
        assert torch.equal(a[0], want[0][t:t + 1]) and torch.equal(a[1], want[1][t:t + 1])
