"""Attention over packed prompts on the GPU, against float64."""
import time
import types

import numpy as np
import pytest

from oracle import step as OS
from tests import paged_cases as PC

pytestmark = pytest.mark.gpu

BF16 = types.SimpleNamespace(kv="bf16")


def starts(lens, gap=0):
    """Packed row starts; ``gap`` rows of nobody before the first and behind the last."""
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32) + gap


def inputs(seed, T, N, hq, hkv, dim, layout="own", k_size=1.0):
    """bf16 rows on the GPU; "fused": parts of one projection's rows (T = N)."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(seed)
    if layout == "fused":
        x = torch.randn((T, hq + 2 * hkv, dim), generator=gen, device="cuda")
        x[:, hq:hq + hkv] *= k_size
        x = x.bfloat16()
        return x[:, :hq], x[:, hq:hq + hkv], x[:, hq + hkv:]
    if layout == "heads":     # heads outside, tokens inside
        return tuple((s * torch.randn((h, n, dim), generator=gen, device="cuda")).bfloat16().transpose(0, 1)
                     for n, h, s in ((T, hq, 1.0), (N, hkv, k_size), (N, hkv, 1.0)))
    return tuple((s * torch.randn((n, h, dim), generator=gen, device="cuda")).bfloat16()
                 for n, h, s in ((T, hq, 1.0), (N, hkv, k_size), (N, hkv, 1.0)))


def check(lib, q, k, v, qs, ks, scale, out_type="bf16", causal=True, window=0, sinks=0, **kw):
    """One call, checked whole; rows outside every sequence keep what they held."""
    import torch
    dt = torch.bfloat16 if out_type == "bf16" else torch.float32
    out = torch.full(q.shape, 77.0, dtype=dt, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = lib.packed_attention_prefill(
        q, k, v, torch.from_numpy(qs).cuda(), scale, key_start=None if ks is None else torch.from_numpy(ks).cuda(),
        causal=causal, window=window, sinks=sinks, out=out, device_status=status, **kw)
    assert got is out or got.data_ptr() == out.data_ptr()
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    x = [t.double().cpu().numpy() for t in (q, k, v)]
    want, mag, reach, seen = OS.packed(*x, qs, qs if ks is None else ks, scale, causal, window, sinks)
    y = out.double().cpu().numpy()
    inside = ~np.isnan(want[:, 0, 0]) if want.size else np.zeros(0, dtype=bool)
    assert (y[~inside] == 77.0).all()
    e = PC.attention_bound(BF16, x[0], want, mag, reach, scale, False, out_type == "bf16",
                           out_type == "f32", int(seen.max(initial=1)))
    assert (np.abs(y - want)[inside] <= e[inside]).all(), np.nanmax((np.abs(y - want) / e)[inside])
    return out


@pytest.mark.parametrize("dim", [8, 16, 40, 64, 72, 80, 96, 112, 128])
@pytest.mark.parametrize("out_type", ["bf16", "f32"])
def test_dims(lib, dim, out_type):
    lens = [130, 1, 0, 257, 33]
    q, k, v = inputs(dim, sum(lens), sum(lens), 4, 2, dim, "fused")
    for causal in (True, False):
        check(lib, q, k, v, starts(lens), None, dim ** -0.5, out_type, causal)


@pytest.mark.parametrize("group,hkv", [(1, 3), (2, 2), (3, 1), (5, 2), (7, 1), (8, 2), (16, 1), (31, 1), (40, 1),
                                       (64, 2), (100, 1), (128, 1)])
def test_groups(lib, group, hkv):
    lens = [max(1, 150 // group), 1, 300 // group + 2]
    q, k, v = inputs(group, sum(lens), sum(lens), group * hkv, hkv, 64)
    check(lib, q, k, v, starts(lens), None, 0.125, "f32")


@pytest.mark.parametrize("n", [1, 2, 63, 64, 65, 127, 128, 129, 255, 256, 257, 383, 384, 385, 511, 513])
@pytest.mark.parametrize("causal", [False, True])
def test_lengths(lib, n, causal):
    """Sequences that end at, before and behind a tile's and a pair's end, next to others."""
    q, k, v = inputs(n, n + 9, n + 9, 2, 1, 128, "heads")
    check(lib, q, k, v, starts([4, n, 5]), None, 0.09, "bf16", causal)
    check(lib, q, k, v, starts([n, 9]), None, 0.09, "f32", causal)


@pytest.mark.parametrize("keys", [1, 2, 130])
def test_one_query(lib, keys):
    """A single row of q, as a decode step over packed keys has it."""
    q, k, v = inputs(keys, 1, keys, 6, 2, 128)
    for out_type in ("bf16", "f32"):
        check(lib, q, k, v, starts([1]), starts([keys]), 0.09, out_type)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (17, 4), (100, 0), (128, 129), (200, 300), (5000, 2)])
@pytest.mark.parametrize("dim", [64, 128])
def test_windows(lib, window, sinks, dim):
    lens = [700, 3, 129, 400]
    q, k, v = inputs(window, sum(lens), sum(lens), 3, 1, dim)
    check(lib, q, k, v, starts(lens), None, 0.1, "f32", window=window, sinks=sinks)
    more = [x + y for x, y in zip(lens, (260, 128, 0, 1))]
    q, k, v = inputs(window, sum(lens), sum(more), 4, 2, dim)
    check(lib, q, k, v, starts(lens), starts(more), 0.1, "bf16", window=window, sinks=sinks)


@pytest.mark.parametrize("window,group", [(1, 8), (40, 8), (64, 16), (65, 16), (300, 3), (10 ** 9, 8)])
def test_every_item_under_a_window(lib, window, group):
    """Lists that grow up to the window and stay there, in sequences of all lengths: every row is written once."""
    lens, ahead = [900, 5, 333, 0, 64, 600, 1], [0, 200, 17, 9, 70, 900, 0]
    for more in (None, [x + y for x, y in zip(lens, ahead)]):
        q, k, v = inputs(group, sum(lens), sum(more or lens), 2 * group, 2, 64)
        check(lib, q, k, v, starts(lens), None if more is None else starts(more), 0.1, "bf16", window=window, sinks=3)


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 200, 2 ** 30 + 3])
@pytest.mark.parametrize("sinks", [0, 4, 2 ** 31 - 1])
@pytest.mark.parametrize("group", [1, 8])
def test_largest_windows_over_fewer_keys_than_queries(lib, window, sinks, group):
    """A window that hides nothing, where position - window of the first queries is below -2^31."""
    lens, keys = [10, 300, 5, 400, 64], [5, 150, 5, 1, 500]
    q, k, v = inputs(group, sum(lens), sum(keys), 2 * group, 2, 64)
    for out_type in ("bf16", "f32"):
        check(lib, q, k, v, starts(lens), starts(keys), 0.1, out_type, window=window, sinks=sinks)


def test_many_sequences_under_a_window(lib):
    rng = np.random.default_rng(4)
    lens = rng.integers(0, 4, 1500)
    lens[rng.integers(0, 1500, 5)] = 140
    q, k, v = inputs(4, int(lens.sum()), int(lens.sum()), 32, 1, 64)
    check(lib, q, k, v, starts(lens), None, 0.125, "bf16", window=20, sinks=1)


@pytest.mark.parametrize("causal", [False, True])
def test_other_key_lengths(lib, causal):
    """More keys than queries, fewer (rows that see nothing), none at all."""
    lens, keys = [50, 200, 1, 300, 7, 20, 0], [300, 60, 500, 0, 1, 20, 40]
    q, k, v = inputs(5, sum(lens), sum(keys), 4, 2, 80)
    for out_type in ("bf16", "f32"):
        out = check(lib, q, k, v, starts(lens), starts(keys), 0.1, out_type, causal)
        assert (out[251:551] == 0).all()
        if causal:
            assert (out[50:190] == 0).all() and (out[551:557] == 0).all()
    q, k, v = inputs(6, 30, 0, 4, 2, 64)
    assert (check(lib, q, k, v, starts([30]), starts([0]), 0.1, "bf16", causal) == 0).all()


@pytest.mark.parametrize("out_type", ["bf16", "f32"])
def test_neighbours_have_no_influence(lib, out_type):
    """NaN and infinities in other sequences, before the first and behind the last."""
    import torch
    lens = [70, 130, 1, 300]
    qs = starts(lens, 40)
    q, k, v = inputs(7, 600, 600, 4, 2, 128, "fused")
    clean = check(lib, q, k, v, qs, None, 0.09, out_type)
    for bad in (float("nan"), float("inf"), -float("inf")):
        for x in (q, k, v):
            y = [t.clone() for t in (q, k, v)]
            z = y[0 if x is q else 1 if x is k else 2]
            z[:40] = bad
            z[qs[-1]:] = bad
            z[qs[1]:qs[2]] = bad          # sequence 1
            out = torch.full(q.shape, 77.0, dtype=clean.dtype, device="cuda")
            lib.packed_attention_prefill(*y, torch.from_numpy(qs).cuda(), 0.09, out=out)
            keep = torch.ones(600, dtype=torch.bool, device="cuda")
            keep[qs[1]:qs[2]] = False
            assert torch.equal(out[keep], clean[keep])


def test_hidden_rows(lib):
    """Keys that causality or the window hides from a whole query tile: whatever they hold."""
    import torch
    q, k, v = inputs(8, 640, 640, 1, 1, 64)
    a = lib.packed_attention_prefill(q, k, v, torch.tensor([0, 640], dtype=torch.int32, device="cuda"), 0.1)
    k[512:], v[512:] = float("nan"), float("nan")
    b = lib.packed_attention_prefill(q, k, v, torch.tensor([0, 640], dtype=torch.int32, device="cuda"), 0.1)
    assert torch.equal(a[:512], b[:512]) and b[600:].isnan().all()
    # hidden keys (not values) of the same tile: no influence either
    q, k, v = inputs(9, 100, 100, 1, 1, 64)
    a = lib.packed_attention_prefill(q, k, v, torch.tensor([0, 100], dtype=torch.int32, device="cuda"), 0.1)
    k[60:] = float("inf")
    b = lib.packed_attention_prefill(q, k, v, torch.tensor([0, 100], dtype=torch.int32, device="cuda"), 0.1)
    assert torch.equal(a[:60], b[:60])


@pytest.mark.parametrize("scale", [0.0, -0.1, 3.0, -2.0, 1e-30])
def test_scales(lib, scale):
    """Negative, zero, tiny and large factors."""
    for size in (1.0, 6.0):
        q, k, v = inputs(10, 500, 500, 2, 1, 128, k_size=size)
        check(lib, q, k, v, starts([500]), None, scale, "f32")
        check(lib, q, k, v, starts([500]), None, scale, "bf16", causal=False)


def test_rising_logits(lib):
    """Every key tile's logits are far above the one before: the reference moves each time."""
    import torch
    q, k, v = inputs(11, 700, 700, 2, 1, 64)
    q[:] = q.abs()
    k[:] = (k.float().abs() * (torch.arange(700, device="cuda") // 100 + 1).view(-1, 1, 1)).bfloat16()
    check(lib, q, k, v, starts([700]), None, 1.0, "f32", causal=False)
    check(lib, q, k, v, starts([700]), None, 1.0, "bf16", causal=False)
    k[:] = k.flip(0)
    check(lib, q, k, v, starts([700]), None, 1.0, "f32")


@pytest.mark.parametrize("seqs", [300, 1024, 1025, 2300])
def test_many_sequences(lib, seqs):
    """More sequences than are ordered together; most of them short, some without a row."""
    rng = np.random.default_rng(seqs)
    lens = rng.integers(0, 4, seqs)
    lens[rng.integers(0, seqs, 5)] = 140
    T = int(lens.sum())
    q, k, v = inputs(seqs, T, T, 2, 1, 64)
    check(lib, q, k, v, starts(lens), None, 0.125, "bf16")


@pytest.mark.parametrize("out_type", ["bf16", "f32"])
def test_more_items_than_ctas(lib, out_type):
    """Several items per CTA, of one key tile to many, both query tiles and one; twice the same bits."""
    import torch
    lens = [1, 400, 129, 257, 20, 128, 700, 1, 64, 300]
    q, k, v = inputs(12, sum(lens), sum(lens), 64, 32, 64, "fused")
    qs = torch.from_numpy(starts(lens)).cuda()
    dt = torch.bfloat16 if out_type == "bf16" else torch.float32
    a = lib.packed_attention_prefill(q, k, v, qs, 0.125, out_dtype=dt)
    for _ in range(3):
        assert torch.equal(a, lib.packed_attention_prefill(q, k, v, qs, 0.125, out_dtype=dt))
    for h in (0, 17, 63):     # a head among the others and alone
        one = check(lib, q[:, h:h + 1], k[:, h // 2:h // 2 + 1], v[:, h // 2:h // 2 + 1], starts(lens), None, 0.125,
                    out_type)
        # (grouped heads share a query tile: another order of nothing, the same numbers)
        assert torch.equal(one[:, 0], a[:, h])


def long_reference(q, k, v, scale, causal):
    """float64 on the GPU, one sequence, one head."""
    import torch
    q, k, v = (x.double() for x in (q, k, v))
    z = q @ k.t() * float(np.float32(scale))
    if causal:
        n, c = z.shape
        z += torch.triu(torch.full((n, c), -torch.inf, dtype=torch.float64, device="cuda"), c - n + 1)
    return torch.softmax(z, -1) @ v


@pytest.mark.parametrize("keys", [3000, 20000])
@pytest.mark.parametrize("dim", [64, 128])
def test_long_float32(lib, keys, dim):
    """The tensor cores cut each sum in O towards zero, up to 2^-23 of it.  Over 16 key tiles, 8 k-steps each
    for two parts of the weights, that is 256 cuts: half of the most on average, of an O that is
    on average half its last size, 256 2^-25 = 2^-17.  The weights' second part is off by 2^-17 at most.
    Together they stay under 1.2e-5 of the norm, however many keys there are."""
    import torch
    q, k, v = inputs(13, 260, keys, 1, 1, dim)
    for causal in (True, False):
        want = long_reference(q[:, 0], k[:, 0], v[:, 0], 0.1, causal)
        got = lib.packed_attention_prefill(q, k, v, torch.tensor([0, 260], dtype=torch.int32, device="cuda"), 0.1,
                                           key_start=torch.tensor([0, keys], dtype=torch.int32, device="cuda"),
                                           causal=causal)
        assert ((got[:, 0].double() - want).norm() / want.norm()).item() <= 1.2e-5


def test_flags(lib):
    import torch
    q, k, v = inputs(14, 100, 100, 2, 1, 64)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call(qs, ks=None):
        out = torch.full(q.shape, 5.0, device="cuda")
        status.zero_()
        lib.packed_attention_prefill(q, k, v, torch.tensor(qs, dtype=torch.int32, device="cuda"), 0.125,
                                     key_start=None if ks is None else torch.tensor(ks, dtype=torch.int32, device="cuda"),
                                     out=out, device_status=status)
        torch.cuda.synchronize()
        return out, int(status.item())

    good, st = call([0, 30, 100])
    assert st == 0
    for qs, ks, whole in (([0, 30, 101], None, 30), ([0, 30, 10], None, 30), ([0, 30, 100], [0, 30, 200], 30),
                          ([0, 30, 100], [0, 30, 20], 30), ([0, 30, 2 ** 31 - 1], None, 30)):
        out, st = call(qs, ks)
        assert st == lib.DEV_BAD_CONTEXT
        assert torch.equal(out[:whole], good[:whole]) and (out[whole:] == 5.0).all()
    out, st = call([-1, 30, 100])
    assert st == lib.DEV_BAD_CONTEXT and torch.equal(out[30:], good[30:]) and (out[:30] == 5.0).all()


def test_streams_graphs_and_refusals(lib):
    """Two calls at once on two streams, a captured one, replayed on new inputs; arguments refused."""
    import torch
    lens = [300, 1, 200]
    a, b = inputs(15, 501, 501, 8, 2, 128), inputs(16, 501, 501, 8, 2, 128, "fused")
    qs = torch.from_numpy(starts(lens)).cuda()
    want = [lib.packed_attention_prefill(*x, qs, 0.09, out_dtype=torch.bfloat16) for x in (a, b)]
    s = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = [lib.packed_attention_prefill(*x, qs, 0.09, out_dtype=torch.bfloat16, stream=t)
               for x, t in zip((a, b), s)]
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    g, out = torch.cuda.CUDAGraph(), torch.empty_like(want[0])
    hold = [x.clone() for x in a]
    with torch.cuda.graph(g, stream=s[0]):
        lib.packed_attention_prefill(*hold, qs, 0.09, out=out)
    for x, y in ((a, want[0]), (b, want[1])):
        for h, t in zip(hold, x):
            h.copy_(t)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, y)
    q, k, v = a

    def call(**kw):
        x = dict(q=q, k=k, v=v, query_start=qs, scale=0.09)
        x.update(kw)
        return lib.packed_attention_prefill(x.pop("q"), x.pop("k"), x.pop("v"), x.pop("query_start"), x.pop("scale"), **x)

    for kw in (dict(k=k[:-1]), dict(k=k.float()), dict(v=v[:, :1]), dict(q=q[:, :7]), dict(query_start=qs.long()),
               dict(key_start=qs[:-1]), dict(q=q[..., ::2], k=k[..., ::2], v=v[..., ::2]),
               dict(k=k[:, :1].expand(501, 2, 128)), dict(q=q.cpu()), dict(out=out.double()),
               dict(out=out.transpose(0, 1)), dict(out_dtype=torch.float16), dict(window=-1), dict(sinks=4),
               dict(window=8, causal=False), dict(scale=float("inf"))):
        with pytest.raises((ValueError, lib.PagedKVError)):
            call(**kw)
    # rows that begin on no 16-byte boundary
    with pytest.raises((ValueError, lib.PagedKVError)):
        call(q=torch.zeros(501 * 8 * 128 + 1, device="cuda", dtype=torch.bfloat16)[1:].view(501, 8, 128))


@pytest.mark.parametrize("out_type", ["bf16", "f32"])
def test_waits_run_out_and_the_next_call_is_clean(lib, out_type):
    """The first V tile's copies never complete: the call flags it and returns, nothing hangs."""
    import torch
    lens = [50, 300]
    q, k, v = inputs(17, 350, 350, 4, 2, 64)
    qs = torch.from_numpy(starts(lens)).cuda()
    dt = torch.bfloat16 if out_type == "bf16" else torch.float32
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        status.zero_()
        torch.cuda.synchronize()
        t0 = time.monotonic()
        out = lib.packed_attention_prefill(q, k, v, qs, 0.125, out_dtype=dt, device_status=status)
        torch.cuda.synchronize()
        return out, int(status.item()), time.monotonic() - t0

    want, st, _ = call()
    assert st == 0
    lib.stall_decode_for_test(16)
    try:
        _, st, waited = call()
        assert st & lib.DEV_TIMEOUT, st
        assert 1.5 <= waited < 30.0, waited
    finally:
        lib.stall_decode_for_test(0)
    out, st, _ = call()
    assert st == 0 and torch.equal(out, want)


def test_rows_past_32_bits(lib):
    """Rows and heads whose elements lie past 2^32 bytes, and past 2^31 elements."""
    import torch
    lens = [5, 2]
    q, k, v = inputs(21, 7, 7, 4, 2, 64)
    want = check(lib, q, k, v, starts(lens), None, 0.125, "f32")
    far = []
    for x in (q, k, v):
        y = torch.empty((7, 2 ** 29), device="cuda", dtype=torch.bfloat16)[:, -x[0].numel():].view(x.shape)
        y.copy_(x)
        far.append(y)
    qs = torch.from_numpy(starts(lens)).cuda()
    assert torch.equal(lib.packed_attention_prefill(*far, qs, 0.125), want)
    del far, y
    # an output of more than 2^32 bytes: its last rows
    T = 2 ** 32 // (2 * 32 * 128) + 40
    q = torch.empty((T, 32, 128), device="cuda", dtype=torch.bfloat16)
    a, k, v = inputs(22, 50, 50, 32, 1, 128)
    q[-50:] = a
    out = torch.empty_like(q)
    lib.packed_attention_prefill(q, k, v, torch.tensor([T - 50, T], dtype=torch.int32, device="cuda"), 0.09, out=out,
                                 key_start=torch.tensor([0, 50], dtype=torch.int32, device="cuda"))
    alone = lib.packed_attention_prefill(a, k, v, torch.tensor([0, 50], dtype=torch.int32, device="cuda"), 0.09,
                                         out_dtype=torch.bfloat16)
    assert torch.equal(out[-50:], alone)


@pytest.mark.parametrize("dim,group,hkv", [(128, 4, 2), (64, 8, 1), (80, 1, 3), (40, 3, 2), (128, 1, 2)])
@pytest.mark.parametrize("kw", [{}, {"causal": False}, {"window": 150, "sinks": 3}])
def test_bf16_outputs_are_the_float32_ones_rounded(lib, dim, group, hkv, kw):
    """The same weights in two parts and the same sums (lists of up to seven key tiles: a float32 output takes
    them in one go too), so the same float32 numbers, rounded once; with logits from small to large."""
    import torch
    lens, ahead = [130, 1, 600, 257, 33], [0, 200, 250, 0, 7]
    keys = [x + y for x, y in zip(lens, ahead)]
    for size in (0.2, 1.0, 5.0):
        q, k, v = inputs(dim, sum(lens), sum(keys), group * hkv, hkv, dim, k_size=size)
        qs, ks = (torch.from_numpy(starts(x)).cuda() for x in (lens, keys))

        def call(dt, **more):
            return lib.packed_attention_prefill(q, k, v, qs, dim ** -0.5, key_start=ks, out_dtype=dt, **kw, **more)

        want = call(torch.float32)
        assert torch.equal(call(torch.bfloat16), want.bfloat16())
        assert torch.equal(call(torch.bfloat16, weight_parts=2), want.bfloat16())


@pytest.mark.parametrize("dim", [64, 128])
def test_one_weight_part(lib, dim):
    """Asked for: weights off by up to 2^-8 of each, as the bound without a second part has it; a float32 output does
    not take it."""
    import torch
    lens = [300, 1, 129]
    q, k, v = inputs(3, sum(lens), sum(lens), 6, 2, dim, "fused")
    one = check(lib, q, k, v, starts(lens), None, dim ** -0.5, "bf16", weight_parts=1)
    two = check(lib, q, k, v, starts(lens), None, dim ** -0.5, "bf16")
    assert not torch.equal(one, two)
    qs = torch.from_numpy(starts(lens)).cuda()
    for kw in (dict(weight_parts=1), dict(weight_parts=0), dict(weight_parts=3, out_dtype=torch.bfloat16),
               dict(weight_parts="x"), dict(weight_parts=-1)):
        with pytest.raises((ValueError, lib.PagedKVError)):
            lib.packed_attention_prefill(q, k, v, qs, 0.1, **kw)


@pytest.mark.parametrize("dim,keys", [(64, 20000), (128, 9000), (128, 130000)])
def test_sums_of_one_sign(lib, dim, keys):
    """Values of one sign, so that O grows evenly while the tensor cores cut each of its sums.  A cut takes half a
    step of the sum on average, and the steps are 2^-23 of their sum's binade: over a sum that grows from 0 they
    average 1/3 to 3/8 of 2^-23 of its last size.  In the 8 key tiles that O is left in the tensor cores for there are 128
    cuts (8 of 16 keys a tile, two weight parts): 128 2^-24 3/8 = 2.9e-6 of every output, however many keys there are.
    The sums in float32 (156 to 1,016 tiles, 20 to 130 parts, both to nearest) add 2^-25 times the root of their number
    over 3 at most, 0.6e-6.  The weights' parts are rounded to nearest and average out.  4e-6 leaves room for what is
    cut of single products; twice as many sums, at 5.1e-6, do not pass."""
    import torch
    q, k, v = inputs(23, 130, keys, 2, 1, dim)
    v = (1 + v.float().abs() / 8).bfloat16()
    for causal in (True, False):
        got = lib.packed_attention_prefill(q, k, v, torch.tensor([0, 130], dtype=torch.int32, device="cuda"), 0.1,
                                           key_start=torch.tensor([0, keys], dtype=torch.int32, device="cuda"),
                                           causal=causal)
        for h in range(2):
            want = long_reference(q[:, h], k[:, 0], v[:, 0], 0.1, causal)
            assert ((got[:, h].double() - want).norm() / want.norm()).item() <= 4e-6


@pytest.mark.parametrize("group,dim", [(8, 64), (3, 128), (1, 128), (100, 64)])
@pytest.mark.parametrize("out_type", ["bf16", "f32"])
def test_values_that_are_not_finite(lib, group, dim, out_type):
    """A NaN or an infinity in V reaches the queries of those groups of 2 (128 / group) that see a key of its 128,
    and one in K those that see it: no others, whatever order the tiles are worked on."""
    import torch
    lens, window, sinks = [20, 520, 33], 64, 3
    q, k, v = inputs(group, sum(lens), sum(lens), group, 1, dim)
    qs, dt = torch.from_numpy(starts(lens)).cuda(), torch.bfloat16 if out_type == "bf16" else torch.float32
    i, per = np.arange(520), 2 * (128 // group)

    def call(k, v, **kw):
        return lib.packed_attention_prefill(q, k, v, qs, 0.1, out_dtype=dt, **kw)

    for kw in ({}, dict(window=window), dict(window=window, sinks=sinks)):
        sees = i <= i[:, None]
        if kw:
            sees &= (i > i[:, None] - window) | (i < kw.get("sinks", 0))
        clean = call(k, v, **kw)
        for at in (0, 100, 127, 128, 300, 519):
            for bad in (float("nan"), float("inf")):
                kb, vb = k.clone(), v.clone()
                kb[20 + at] = bad
                got = call(kb, v, **kw)
                hit = torch.zeros(sum(lens), dtype=torch.bool, device="cuda")
                hit[20:540] = torch.from_numpy(sees[:, at]).cuda()
                assert torch.equal(got[~hit], clean[~hit]) and not torch.equal(got[hit], clean[hit])
                vb[20 + at] = bad
                got = call(k, vb, **kw)
                tile = sees[:, at // 128 * 128:at // 128 * 128 + 128].any(1)
                near = np.array([tile[n // per * per:n // per * per + per].any() for n in i])
                assert not got[hit].isfinite().any()
                hit[20:540] = torch.from_numpy(near).cuda()
                assert torch.equal(got[~hit], clean[~hit])


@pytest.mark.parametrize("keys", [20000, 130000])
def test_long_bf16(lib, keys):
    """A bf16 output over long lists: its own rounding (2^-8 of a value at most) and the cut sums, which the tensor
    cores keep to the end.  A key adds a sum of two parts; cut by half a step of a sum that averages half of the last
    one, and of 16 products with two more bits each, keys / 16 4 2^-24 / 2 at most on average."""
    import torch
    q, k, v = inputs(24, 200, keys, 1, 1, 128)
    for one_sign in (False, True):
        if one_sign:
            v = (1 + v.float().abs() / 8).bfloat16()
        want = long_reference(q[:, 0], k[:, 0], v[:, 0], 0.1, True)
        got = lib.packed_attention_prefill(q, k, v, torch.tensor([0, 200], dtype=torch.int32, device="cuda"), 0.1,
                                           key_start=torch.tensor([0, keys], dtype=torch.int32, device="cuda"),
                                           out_dtype=torch.bfloat16)
        own = (want.bfloat16().double() - want).norm() / want.norm()
        more = (got[:, 0].double() - want).norm() / want.norm()
        assert more.item() <= own.item() + keys / 16 * 4 * 2.0 ** -25


def gpu_reference(q, k, v, qs, ks, scale, causal=True, window=0, sinks=0):
    """float64 on the GPU: (out, A = sum p |v|, the most of sum |q k| over visible keys), by sequence and head."""
    import torch
    out, mag = (torch.zeros(q.shape, dtype=torch.float64, device="cuda") for _ in range(2))
    reach = torch.zeros(q.shape[:2], dtype=torch.float64, device="cuda")
    group = q.shape[1] // k.shape[1]
    for a, b, c0, c1 in zip(qs[:-1], qs[1:], ks[:-1], ks[1:]):
        n, c = int(b - a), int(c1 - c0)
        place = torch.arange(c - n, c, device="cuda")[:, None]
        j = torch.arange(c, device="cuda")
        sees = torch.ones((n, c), dtype=torch.bool, device="cuda")
        if causal:
            sees = j <= place
            if window:
                sees &= (j > place - window) | (j < sinks)
        for h in range(q.shape[1]):
            x, y, w = (z.double() for z in (q[a:b, h], k[c0:c1, h // group], v[c0:c1, h // group]))
            z = (x @ y.t() * float(np.float32(scale))).masked_fill(~sees, -torch.inf)
            p = torch.softmax(z, -1).nan_to_num(0.0)      # rows that see nothing
            out[a:b, h], mag[a:b, h] = p @ w, p @ w.abs()
            reach[a:b, h] = (x.abs() @ y.abs().t()).masked_fill(~sees, 0.0).amax(-1)
    return out, mag, reach


def check_parts(lib, q, k, v, lens, keys, scale, **kw):
    """Every element of a float32 output of long lists, and the same call's again."""
    import torch
    qs, ks = starts(lens), starts(keys)
    args = (q, k, v, torch.from_numpy(qs).cuda(), scale)
    out = torch.full(q.shape, 77.0, device="cuda")
    lib.packed_attention_prefill(*args, key_start=torch.from_numpy(ks).cuda(), out=out, **kw)
    want, mag, reach = (x.cpu().numpy() for x in gpu_reference(q, k, v, qs, ks, scale, **kw))
    # the bound's sums are a float32 step for each 16 keys: a list's parts are as exact as one list of 1,024 keys and a step
    # for each part more
    e = PC.attention_bound(BF16, None, want, mag, reach, scale, False, False, True, 1024 + max(keys) // 64)
    y = out.double().cpu().numpy()
    assert (np.abs(y - want) <= e).all(), (np.abs(y - want) / e).max()
    again = lib.packed_attention_prefill(*args, key_start=torch.from_numpy(ks).cuda(), **kw)
    assert torch.equal(out, again)
    return out


@pytest.mark.parametrize("keys", [1024, 1025, 1152, 2048, 2049, 2176, 3200, 4097])
@pytest.mark.parametrize("causal", [True, False])
def test_parts_that_end_at_a_tile(lib, keys, causal):
    """Lists that fill parts of 8 key tiles, or one key or tile more; a pair whose first tile ends there and
    whose second goes on."""
    for n in (129, 256):
        q, k, v = inputs(keys + n, n, keys, 2, 1, 64)
        check_parts(lib, q, k, v, [n], [keys], 0.125, causal=causal)


@pytest.mark.parametrize("group,hkv,dim", [(3, 2, 128), (8, 1, 64), (1, 2, 80), (40, 1, 128), (128, 1, 64)])
@pytest.mark.parametrize("kw", [{}, {"window": 2500, "sinks": 200}, {"window": 1100}, {"causal": False}])
def test_parts_of_grouped_heads(lib, group, hkv, dim, kw):
    """Several parts to a list under grouped heads, windows (whose lists skip key tiles) and sinks of more than a tile;
    sequences of one part beside them, and rows that see nothing."""
    lens, keys = [70, 3, 130, 1, 40], [4300, 3, 2700, 1500, 10]
    q, k, v = inputs(group, sum(lens), sum(keys), group * hkv, hkv, dim)
    check_parts(lib, q, k, v, lens, keys, dim ** -0.5, **kw)


@pytest.mark.parametrize("order", ["rising", "falling", "both"])
@pytest.mark.parametrize("kw", [{}, {"causal": False}, {"window": 1500, "sinks": 129}])
def test_parts_whose_references_move(lib, order, kw):
    """Logits that grow or shrink by far more than 2^24 from part to part: what earlier parts left is scaled, or
    what later ones add vanishes; rows of either kind beside rows whose logits stay."""
    import torch
    n, keys = 300, 4600
    q, k, v = inputs(31, n, keys, 2, 1, 64)
    step = 1 + (torch.arange(keys, device="cuda") // 512).double()
    if order == "falling":
        step = step.flip(0)
    if order == "both":
        step = torch.minimum(step, step.flip(0)) ** 2
    k[:, 0, :32] = (k[:, 0, :32].double().abs() * step[:, None] / 2).bfloat16()
    q[:, 0, :32] = q[:, 0, :32].abs()
    q[:, 1, :32] *= 0.01                              # the other head's logits hardly move
    q[1::3, 0, :32] *= -1                             # rows whose logits go the other way
    check_parts(lib, q, k, v, [n], [keys], 1.0, **kw)


def test_more_items_of_several_parts_than_ctas(lib):
    """Items of two to five parts, three and more to a CTA, in sequences of all lengths."""
    lens, ahead = [1500, 40, 700, 3, 260], [300, 2100, 1500, 4500, 0]
    q, k, v = inputs(32, sum(lens), sum(lens) + sum(ahead), 32, 16, 64)
    check_parts(lib, q, k, v, lens, [x + y for x, y in zip(lens, ahead)], 0.125)


def test_a_first_part_that_is_masked_whole(lib):
    """Sinks and a window far behind them: rows of an early position see keys of a later part alone, or of the first
    one alone."""
    lens, keys = [1300, 900], [1300, 4000]
    q, k, v = inputs(33, sum(lens), sum(keys), 8, 1, 64)
    for kw in (dict(window=1, sinks=1100), dict(window=1030, sinks=1), dict(window=1500, sinks=0),
               dict(window=300, sinks=1030)):
        check_parts(lib, q, k, v, lens, keys, 0.125, **kw)


@pytest.mark.parametrize("out_type", ["bf16", "f32"])
def test_strides_of_no_rows(lib, out_type):
    """Rows of an empty tensor may have any strides: no tokens, and queries over no keys."""
    import torch
    i32 = dict(dtype=torch.int32, device="cuda")
    dt = torch.bfloat16 if out_type == "bf16" else torch.float32
    room = torch.empty(4096, dtype=torch.bfloat16, device="cuda")
    for strides in ((0, 0, 0), (0, 0, 1), (5, 3, 1), (512, 64, 1)):
        def none(heads):
            return room.as_strided((0, heads, 64), strides)

        for seqs in (0, 1, 3):
            got = lib.packed_attention_prefill(none(4), none(2), none(2), torch.zeros(seqs + 1, **i32), 0.1, out_dtype=dt)
            assert got.shape == (0, 4, 64) and got.dtype == dt
        q = torch.ones((5, 4, 64), dtype=torch.bfloat16, device="cuda")
        got = lib.packed_attention_prefill(q, none(2), none(2), torch.tensor([0, 2, 5], **i32), 0.1,
                                           key_start=torch.zeros(3, **i32), out_dtype=dt)
        assert got.shape == (5, 4, 64) and not got.any()
