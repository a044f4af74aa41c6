"""Attention with a sliding window and sinks on the GPU, against the numpy definition."""
import numpy as np
import pytest

from oracle import block_scaled as OB
from tests import gpu_cases as GC
from tests import paged_cases as PC
from tests.test_gpu_block_scaled import check_decode, decode

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kv,d", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("fp8_e4m3", 128),
                                  ("int8", 128)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (33, 0), (64, 129), (300, 16),
                                          (5000, 4)])
def test_decode(lib, kv, d, window, sinks):
    """Contexts below, at and above the window; windows and sinks that begin inside blocks,
    meet, overlap or cover everything."""
    lens = [1, 17, window + sinks + 1 if window < 400 else 40, 513, 0, 350]
    for bs, hq, hkv in ((16, 8, 2), (64, 3, 1), (8, 12, 1)):
        case = PC.make(7 * bs + window, kv, lens, hkv, d, bs)
        check_decode(lib, case, hq, 8, out="f32", window=window, sinks=sinks)


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3", "int8"])
@pytest.mark.parametrize("q_type", ["bf16", "f32"])
def test_decode_split(lib, kv, q_type):
    """Several partitions of the visible tokens; out in bf16 too."""
    for bs, window, sinks in ((16, 500, 70), (256, 900, 300), (8, 65, 1)):
        case = PC.make(bs, kv, [2100, 64, 571, 1300, 1], 2, 128, bs)
        for part in (0, 64, 192):
            check_decode(lib, case, 16, 9, q_type=q_type, out="f32", window=window, sinks=sinks,
                         partition=part)
        check_decode(lib, case, 8, 10, q_type=q_type, out="bf16", window=window, sinks=sinks)


@pytest.mark.parametrize("kv,d", [("bf16", 64), ("bf16", 128), ("bf16", 256), ("fp8_e4m3", 128)])
def test_decode_clusters(lib, kv, d):
    """Two to eight partitions merged within a cluster, sequences with fewer than the most, and
    more partitions than a cluster takes."""
    case = PC.make(17, kv, [1, 64, 130, 520, 0, 300], 2, d, 16)
    for part, parts in ((64, 9), (128, 5), (192, 3), (320, 2), (576, 1)):
        scratch = lib.workspace_bytes(6, 20, 2, d, 520, part, window=0)
        assert (scratch > 0) == (parts > 8)
        check_decode(lib, case, 20, 18, out="f32", window=10 ** 6, partition=part)
    check_decode(lib, case, 6, 19, out="bf16", window=200, sinks=30, partition=64)


def test_decode_over_one_wave(lib):
    """480 sequences and heads of about 1,100 visible tokens: the automatic partition takes
    more than one wave of CTAs, with a last partition shorter than the others."""
    rng = np.random.default_rng(3)
    case = PC.make(23, "bf16", [int(n) for n in rng.integers(900, 1400, 60)], 8, 64, 16)
    assert lib.workspace_bytes(60, 16, 8, 64, 1400, 0, window=1024, sinks=4) > 0
    check_decode(lib, case, 16, 24, out="f32", window=1024, sinks=4)
    check_decode(lib, case, 16, 25, out="bf16")


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3", "int8"])
def test_hidden_blocks_are_not_read(lib, kv):
    """Table entries of blocks without a visible token may be anything, and hidden rows NaN."""
    import torch
    bs, window, sinks = 16, 40, 20
    case = PC.make(3, kv, [400, 200, 61], 2, 128, bs)
    if kv != "int8":
        for s, n in enumerate(case.lens):     # poison every hidden token
            for t in range(sinks, max(sinks, n - window)):
                for c in (case.k, case.v):
                    c[case.tables[s][t // bs], t % bs] = GC.POISON[kv][1]
    check_decode(lib, case, 4, 4, out="f32", window=window, sinks=sinks)
    q = PC.bf16_bits(np.random.default_rng(1).standard_normal((3, 4, 128)))
    a = decode(lib, case, q, "bf16", 0.1, "f32", window=window, sinks=sinks)
    for s, n in enumerate(case.lens):
        for b in range(-(-n // bs)):
            if (b * bs >= sinks) and (b + 1) * bs <= n - window:
                case.tables[s][b] = -5 if b % 2 else 10 ** 8
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    b = decode(lib, case, q, "bf16", 0.1, "f32", status=status, window=window, sinks=sinks)
    assert int(status.item()) == 0
    assert np.array_equal(a, b)


def test_window_over_everything_equals_plain_decode(lib):
    """A window that covers every context gives the plain call's result within the sum of
    both bounds (the chunks are the same, the exponent's argument is rounded once more)."""
    case = PC.make(5, "bf16", [700, 33, 1], 2, 128, 16)
    check_decode(lib, case, 8, 6, out="f32", window=4096, sinks=0)


def test_flags(lib):
    import torch
    case = PC.make(6, "bf16", [100, 50, 20], 2, 128, 16)
    q = PC.bf16_bits(np.random.default_rng(1).standard_normal((3, 4, 128)))
    ok = decode(lib, case, q, "bf16", 0.1, "f32", window=30, sinks=4)
    case.tables[0, 5] = 10 ** 7           # visible (tokens 80..95)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = decode(lib, case, q, "bf16", 0.1, "f32", status=status, window=30, sinks=4)
    assert int(status.item()) == lib.DEV_BAD_BLOCK
    assert np.array_equal(got[1:], ok[1:])
    case = PC.make(6, "bf16", [100, 50, 20], 2, 128, 16)
    d = case.device()
    d["lens"][1] = 10 ** 6
    d["lens"][2] = -3
    status.zero_()
    out = lib.paged_attention_decode(GC.to_torch(q, "bf16"), d["k"], d["v"], d["tables"], d["lens"],
                                     0.1, 100, window=30, sinks=4, device_status=status)
    assert int(status.item()) & lib.DEV_BAD_CONTEXT
    assert np.array_equal(out[0].cpu().numpy(), ok[0].astype(np.float32))
    assert (out[2] == 0).all()


def test_two_graphs_share_a_workspace(lib):
    """Two captured calls on one stream with the same scratch, replayed in any order."""
    import torch
    case = PC.make(8, "bf16", [900, 500], 2, 128, 16)
    d = case.device()
    need = lib.workspace_bytes(2, 8, 2, 128, 900, 64, window=0)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    qs = [torch.randn((2, 8, 128), device="cuda").to(torch.bfloat16) for _ in range(2)]
    outs = [torch.zeros((2, 8, 128), device="cuda") for _ in range(2)]
    wins = [(300, 4), (700, 0)]

    def call(i, out):
        return lib.paged_attention_decode(qs[i], d["k"], d["v"], d["tables"], d["lens"], 0.1, 900,
                                          out=out, workspace=ws, partition=64, window=wins[i][0],
                                          sinks=wins[i][1])
    want = [call(i, None).clone() for i in range(2)]
    graphs = []
    for i in range(2):
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(i, outs[i])
        graphs.append(g)
    for i in (0, 1, 1, 0, 0):
        outs[i].zero_()
        graphs[i].replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))


# ---- prefill ------------------------------------------------------------------
def prefill(lib, case, new, q, scale, out="f32", status=None, causal=True, window=0, sinks=0, **kw):
    import torch
    d = case.device()
    start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    r = lib.paged_attention_prefill(
        GC.to_torch(q, "bf16"), start, d["k"], d["v"], d["tables"], d["lens"], scale, max(new),
        max(case.lens), causal=causal, k_scale=d.get("ks"), v_scale=d.get("vs"), window=window,
        sinks=sinks, out_dtype=torch.bfloat16 if out == "bf16" else torch.float32,
        device_status=status, **kw)
    return r.float().cpu().numpy().astype(np.float64)


def check_prefill(lib, case, new, hq, seed, out="f32", window=0, sinks=0, scale=None, causal=True,
                  sample=9):
    """Every chunk's first, last and some other rows against the definition."""
    import torch
    hkv, d = case.k.shape[2:]
    scale = d ** -0.5 if scale is None else scale
    q = PC.bf16_bits(np.random.default_rng(seed).standard_normal((sum(new), hq, d)))
    q64 = GC.OA.to_f64(q, "bf16")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = prefill(lib, case, new, q, scale, out, status, causal, window, sinks)
    assert int(status.item()) == 0
    rng = np.random.default_rng(seed + 1)
    row = worst = 0
    for s, (c, n) in enumerate(zip(case.lens, new)):
        if n == 0:
            continue
        pick = np.unique(np.r_[0, n - 1, rng.integers(0, n, sample)])
        K, V = case.values(s)
        pos = c - n + pick if causal else np.full(pick.shape, c - 1)
        x = q64[row + pick]
        o, mag, reach = OB.attend(x, pos, K, V, scale, window, sinks)
        lim = PC.attention_bound(case, x, o, mag, reach, scale, False, out == "bf16",
                                 case.kv == "bf16" and out == "f32",
                                 min(c, window + sinks) if window else c)
        worst = max(worst, float((np.abs(got[row + pick] - o) / lim).max()))
        row += n
    assert worst <= 1.0, worst
    return got


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3", "int8"])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 0), (33, 4), (100, 64), (200, 129),
                                          (300, 16), (5000, 4)])
def test_prefill(lib, kv, window, sinks):
    """Chunks of one token to several query tiles, with and without a prefix; windows below
    and above the chunk's and the tile's length; group sizes that do and do not divide 128."""
    for bs, hq, hkv in ((16, 2, 2), (64, 8, 1), (8, 6, 2)):
        lens = [1, 300, 641, 130, 700]
        new = [1, 300, 130, 0, 257]
        case = PC.make(11 * bs + window, kv, lens, hkv, 128, bs, stride=hkv + 1)
        check_prefill(lib, case, new, hq, 12, window=window, sinks=sinks)


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3", "int8"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("bs,hq,hkv", [(16, 4, 4), (128, 16, 1), (32, 3, 1), (256, 5, 1)])
def test_prefill_block_scales_and_outputs(lib, kv, out, bs, hq, hkv):
    """The whole context and windows, causal or (without a window) not, either output type,
    scales of blocks that differ a lot, negative and zero logit scales."""
    lens, new = [257, 64, 500], [257, 3, 140]
    case = PC.make(bs, kv, lens, hkv, 128, bs, spread=1.5)
    if kv != "bf16":
        case.ks = np.minimum(case.ks, np.float32(8.0 / OB.QMAX[kv]))
    check_prefill(lib, case, new, hq, 13, out=out)
    check_prefill(lib, case, new, hq, 14, out=out, causal=False)
    check_prefill(lib, case, new, hq, 15, out=out, window=77, sinks=3, scale=-0.1)
    check_prefill(lib, case, new, hq, 16, out=out, window=70, sinks=0, scale=0.0)
    if kv != "bf16":   # one scale per head
        case = PC.make(bs, kv, lens, hkv, 128, bs, scales="head")
        check_prefill(lib, case, new, hq, 17, out=out, window=90, sinks=70)


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
def test_prefill_hidden_blocks_are_not_read(lib, kv):
    """Hidden rows hold NaN and hidden blocks' table entries anything."""
    import torch
    bs, window, sinks = 16, 90, 20
    lens, new = [700, 400, 333], [200, 1, 130]
    case = PC.make(3, kv, lens, 2, 128, bs)
    for s, (c, n) in enumerate(zip(lens, new)):
        low = c - n - window + 1
        for t in range(sinks, max(sinks, low)):
            for x in (case.k, case.v):
                x[case.tables[s][t // bs], t % bs] = GC.POISON[kv][1]
        for b in range(-(-c // bs)):
            if b * bs >= sinks and (b + 1) * bs <= low:
                case.tables[s][b] = -5 if b % 2 else 10 ** 8
    real = case.tables.copy()
    case.tables = np.where((real < 0) | (real >= case.k.shape[0]), 0, real).astype(np.int32)
    hold = case.values
    kept = case.tables
    case.tables = real
    case.values = lambda s, *a: _values_with(case, kept, hold, s)
    check_prefill(lib, case, new, 4, 5, window=window, sinks=sinks)


def _values_with(case, tables, values, s):
    """The sequence's rows with the hidden blocks' entries replaced and their NaN as 0."""
    real, case.tables = case.tables, tables
    K, V = values(s)
    case.tables = real
    return np.nan_to_num(K), np.nan_to_num(V)


def test_prefill_flags(lib):
    import torch
    case = PC.make(6, "bf16", [100, 50, 20], 2, 128, 16)
    new = [30, 50, 20]
    q = PC.bf16_bits(np.random.default_rng(1).standard_normal((100, 4, 128)))
    ok = prefill(lib, case, new, q, 0.1, window=30, sinks=4)
    case.lens = [100, 49, 20]              # shorter than its chunk: rows of 0
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = prefill(lib, case, new, q, 0.1, status=status, window=30, sinks=4)
    assert int(status.item()) == lib.DEV_BAD_CONTEXT
    assert (got[30:80] == 0).all() and np.array_equal(got[:30], ok[:30]) and np.array_equal(got[80:], ok[80:])
    case = PC.make(6, "bf16", [100, 50, 20], 2, 128, 16)
    case.tables[0, 4] = 10 ** 7            # tokens 64..79, inside the first chunk's windows
    status.zero_()
    got = prefill(lib, case, new, q, 0.1, status=status, window=30, sinks=4)
    assert int(status.item()) == lib.DEV_BAD_BLOCK and np.array_equal(got[30:], ok[30:])


def test_prefill_equals_decode_rows(lib):
    """The last token of each chunk is the decode query of that context."""
    for kv in ("bf16", "fp8_e4m3"):
        case = PC.make(21, kv, [300, 77, 1], 2, 128, 16)
        new = [40, 77, 1]
        q = PC.bf16_bits(np.random.default_rng(2).standard_normal((sum(new), 8, 128)))
        last = np.cumsum(new) - 1
        for w, s in ((50, 4), (1000, 0)):
            a = prefill(lib, case, new, q, 0.09, out="bf16", window=w, sinks=s)[last]
            b = decode(lib, case, q[last], "bf16", 0.09, "bf16", window=w, sinks=s)
            # both round to bf16 (two half steps); weights: one bf16 in prefill, else fp16 or finer
            A = max(float(np.abs(case.values(i)[1]).max()) for i in range(3))
            assert np.abs(a - b).max() <= (2 * 2.0 ** -8 + 2 * 2.0 ** -8 + 2 * 2.0 ** -11) * A


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3", "int8"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
def test_prefill_long(lib, kv, out):
    """Many key tiles per CTA and more CTAs than SMs, whole and cut tiles in turn."""
    case = PC.make(31, kv, [2500, 1111, 3000], 4, 128, 32)
    new = [700, 1111, 65]
    check_prefill(lib, case, new, 16, 32, out=out, window=1500, sinks=200)
    check_prefill(lib, case, new, 16, 33, out=out, window=4000 if kv == "bf16" else 0)


def test_prefill_repeats_itself(lib):
    """The same call again and again, beside others: the same bits."""
    import torch
    for kv in ("bf16", "int8"):
        case = PC.make(41, kv, [900, 500, 77], 2, 128, 16)
        new = [900, 123, 77]
        q = PC.bf16_bits(np.random.default_rng(5).standard_normal((sum(new), 8, 128)))
        first = prefill(lib, case, new, q, 0.09, window=200, sinks=5)
        for _ in range(5):
            prefill(lib, case, new, q, 0.09, out="bf16", window=600)
            assert np.array_equal(prefill(lib, case, new, q, 0.09, window=200, sinks=5), first)


def _fill(case, s, K=None, V=None):
    """Puts rows ``[n, Hkv, D]`` in storage at positions 0 .. n - 1 of sequence s."""
    for cache, rows in ((case.k, K), (case.v, V)):
        for t in range(0 if rows is None else len(rows)):
            cache[case.tables[s][t // case.bs], t % case.bs] = rows[t]


def test_prefill_weights_keep_their_bits_in_bf16_outputs(lib):
    """bf16 caches and outputs: the weights are two bf16 parts as with a float32 output.

    The values are +u and -u in turn and the weights nearly equal, so a result is a small
    difference of large terms: the bound on sum p |v| has 2^-16, which one bf16 value (2^-8)
    exceeds."""
    n = 200
    case = PC.make(51, "bf16", [n], 2, 128, 16)
    rng = np.random.default_rng(52)
    u = np.abs(rng.standard_normal((2, 128))) + 0.5
    _fill(case, 0, V=PC.bf16_bits(np.where(np.arange(n) % 2, 1.0, -1.0)[:, None, None] * u))
    for window in (2, 3, 7, 60):
        check = _prefill_ratio(lib, case, [n], 8, 53, "bf16", window, 0.02, e_p=2.0 ** -16)
        assert check <= 1.0, (window, check)


def test_prefill_of_one_value_returns_it(lib):
    """Every V row the same bf16 row: each output is that row, bit for bit.  The weights sum to
    one within 2^-15, less than half a step (at least 2^-9), whatever the running reference."""
    import torch
    n = 500
    case = PC.make(54, "bf16", [n, 77], 2, 128, 16)
    v = PC.bf16_bits(np.random.default_rng(55).standard_normal((2, 128)))
    for s, c in enumerate(case.lens):
        _fill(case, s, V=np.broadcast_to(v, (c, 2, 128)))
    new = [300, 77]
    want = GC.OA.to_f64(v, "bf16").repeat(4, axis=0)
    for scale in (0.01, 0.09, 0.4):
        q = PC.bf16_bits(np.random.default_rng(56).standard_normal((sum(new), 8, 128)))
        for kw in ({}, {"window": 5}, {"window": 130, "sinks": 70}):
            got = prefill(lib, case, new, q, scale, out="bf16", **kw)
            assert np.array_equal(got, np.broadcast_to(want, got.shape)), (scale, kw)


def _prefill_ratio(lib, case, new, hq, seed, out, window, scale, e_p, floor=None, q=None):
    """Largest error of a prefill call over ``attention_bound`` with the given weight term."""
    import torch
    hkv, d = case.k.shape[2:]
    if q is None:
        q = PC.bf16_bits(np.random.default_rng(seed).standard_normal((sum(new), hq, d)))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = prefill(lib, case, new, q, scale, out, status, window=window)
    assert int(status.item()) == 0
    q64, worst, row = GC.OA.to_f64(q, "bf16"), 0.0, 0
    for s, (c, n) in enumerate(zip(case.lens, new)):
        K, V = case.values(s)
        x = q64[row:row + n]
        o, mag, reach = OB.attend(x, np.arange(c - n, c), K, V, scale, window, 0)
        lim = PC.attention_bound(case, x, o, mag, reach, scale, False, out == "bf16", True,
                                 min(c, window) if window else c, e_p=e_p, floor=floor)
        worst = max(worst, float((np.abs(got[row:row + n] - o) / lim).max()))
        row += n
    return worst


def _heavy_key(kv, seed, n, gap):
    """A sequence of n tokens whose first key takes nearly all of every query's weight (the
    others' are about 2^-gap of it) and whose first V row is zero; and q.  All V rows but the
    first are ordinary, so the small weights make the whole result."""
    case = PC.make(seed, kv, [n], 1, 128, 16, scales="head")
    case.ks[:], case.vs[:] = 0.01, 0.02
    rng = np.random.default_rng(seed + 1)
    x = rng.standard_normal((n, 1, 128)).astype(np.float32) * 20
    x[:, 0, :2] = 0.0
    x[0, 0, 0] = 100.0
    y = rng.standard_normal((n, 1, 128)).astype(np.float32) * 30
    y[0] = 0.0
    _fill(case, 0, OB.encode(x, kv), OB.encode(y, kv))
    # q = (a, 0, small ...): the first key's logit is scale * a * 100 * 0.01 = a * scale
    q = rng.standard_normal((n, 4, 128)) * 0.25
    q[..., 0] = gap * np.log(2.0)
    q[..., 1] = 0.0
    return case, PC.bf16_bits(q)


@pytest.mark.parametrize("kv", ["fp8_e4m3", "int8"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("gap", [14, 18, 22])
def test_prefill_small_weights_reach_the_product(lib, kv, out, gap):
    """8-bit caches: the largest weight is at least 2^7 as fp16 holds it, so a small one is off
    by 2^-32 of the largest (2^-25 / 2^7) and by its own relative 2^-11 (2^-22 for float32
    outputs' two parts)."""
    n = 150
    case, q = _heavy_key(kv, 57 + gap, n, gap)
    r = _prefill_ratio(lib, case, [n], 4, 0, out, 1000, 1.0, e_p=2.0 ** -11, floor=2.0 ** -32, q=q)
    assert r <= 1.0, r


@pytest.mark.parametrize("kv", ["fp8_e4m3", "int8"])
def test_prefill_f32_outputs_of_8_bit_caches(lib, kv):
    """Float32 outputs carry the weights as two fp16 parts (2^-22), as decode does."""
    for lens, new, hq, hkv, scale, kw in (([300, 641], [300, 130], 4, 2, 0.05, 0), ([700], [700], 8, 1, 0.2, 90)):
        case = PC.make(58, kv, lens, hkv, 128, 16, scales="block", spread=0.3)
        r = _prefill_ratio(lib, case, new, hq, 59, "f32", kw, scale, e_p=2.0 ** -22, floor=2.0 ** -32)
        assert r <= 1.0, r
    case, q = _heavy_key(kv, 60, 150, 12)
    r = _prefill_ratio(lib, case, [150], 4, 0, "f32", 1000, 1.0, e_p=2.0 ** -22, floor=2.0 ** -32, q=q)
    assert r <= 1.0, r


def test_workspace_of_the_longest_context_is_used_by_shorter_calls(lib):
    """A buffer sized for 16 sequences of up to 6,144 tokens serves smaller calls, whose automatic
    partition may need more scratch than the largest: nothing is allocated beside it."""
    import torch
    cap, hkv, hq, d, bs = 6144, 8, 32, 128, 128
    ws = torch.empty(lib.workspace_bytes(16, hq, hkv, d, cap, window=0), dtype=torch.uint8, device="cuda")
    torch.manual_seed(9)
    k, v = (torch.randn((64, bs, hkv, d), device="cuda").to(torch.bfloat16) for _ in range(2))
    bt = torch.randint(0, 64, (16, cap // bs), dtype=torch.int32, device="cuda")
    q = torch.randn((16, hq, d), device="cuda").to(torch.bfloat16)
    used = 0
    for s, c in ((16, 1024), (16, 1536), (8, 4096), (8, 6144), (4, 6144), (1, 6144), (16, 6144)):
        lens = torch.full((s,), c, dtype=torch.int32, device="cuda")
        out = torch.empty((s, hq, d), dtype=torch.bfloat16, device="cuda")
        args = (q[:s].contiguous(), k, v, bt[:s].contiguous(), lens, 0.09, c)
        own = lib.paged_attention_decode(*args, out_dtype=torch.bfloat16, partition=128)
        torch.cuda.synchronize()
        before = torch.cuda.memory_stats()["allocation.all.allocated"]
        lib.paged_attention_decode(*args, out=out, workspace=ws)
        assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
        used += lib.library().paged_attention_window_call_bytes(s, hq, hkv, d, c, 0, 0, 0, lib.BF16) > 0
        # two bf16 roundings of results that differ by the merges' float32 steps
        assert (out.float() - own.float()).abs().max() <= 2.0 ** -7 * own.float().abs().max()
    assert used


def test_scales_per_head_in_a_column(lib):
    """``[Hkv, 1]`` scales give what ``[Hkv]`` ones do, in the plain and the windowed calls."""
    import torch
    case = PC.make(61, "fp8_e4m3", [300, 77], 2, 128, 16, scales="head")
    d = case.device()
    q = torch.randn((107, 8, 128), device="cuda").to(torch.bfloat16)
    start = torch.tensor([0, 30, 107], dtype=torch.int32, device="cuda")
    for window in (0, 50):
        got = []
        for shape in ((2,), (2, 1), (1, 2)):
            kw = dict(k_scale=d["ks"].view(shape), v_scale=d["vs"].view(shape), window=window)
            got.append((lib.paged_attention_decode(q[:2].contiguous(), d["k"], d["v"], d["tables"], d["lens"],
                                                   0.09, 300, **kw),
                        lib.paged_attention_prefill(q, start, d["k"], d["v"], d["tables"], d["lens"], 0.09,
                                                    77, 300, **kw)))
        assert all(torch.equal(a, b) for g in got for a, b in zip(g, got[0]))


def test_window_over_everything_and_the_plain_decode_agree(lib):
    """A window that covers every context and the plain call: within the sum of both bounds."""
    import torch
    case = PC.make(62, "bf16", [700, 33, 1, 2048], 2, 128, 16)
    scale = 128 ** -0.5
    q = PC.bf16_bits(np.random.default_rng(63).standard_normal((4, 8, 128)))
    d = case.device()
    plain = lib.paged_attention_decode(GC.to_torch(q, "bf16"), d["k"], d["v"], d["tables"], d["lens"],
                                       scale, max(case.lens))
    assert plain.dtype == torch.float32
    plain = plain.cpu().numpy().astype(np.float64)
    got = decode(lib, case, q, "bf16", scale, "f32", window=4096)
    q64 = GC.OA.to_f64(q, "bf16")
    for s, n in enumerate(case.lens):
        K, V = case.values(s)
        o, mag, reach = OB.attend(q64[s:s + 1], [n - 1], K, V, scale, 0, 0)
        lim = [PC.attention_bound(case, q64[s:s + 1], o, mag, reach, scale, False, False, True, n, e_p=e)[0]
               for e in (2.0 ** -24, 2.0 ** -16)]
        assert (np.abs(got[s] - plain[s]) <= lim[0] + lim[1]).all()
        assert (np.abs(got[s] - o[0]) <= lim[0]).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("q_type", ["bf16", "f32"])
def test_decode_weights_in_three_parts(lib, d, q_type):
    """bf16 caches, float32 outputs: weights hold 2^-24, two parts (2^-16) would not pass.

    Each query sees two keys of one chunk, with logits 0 and -1 < z <= 0 from one product each
    (exact) and values +1 and -1.  In units of 2^-23 of sum p |v| = 1: the exponent's argument is
    rounded three times, 2^-24 of at most 1 each (1); ex2.approx 2^-22 (2); the parts 2^-24 (1/2):
    on numerator and denominator, 7.  The products' sums: three MMAs of two terms (6); l, the
    merge of warps and the quotient (2): 15."""
    S, hq = 64, 8
    lens = [18 + (s % 14) for s in range(S)]         # tokens ctx - 2, ctx - 1 in chunk 16 .. 31
    case = PC.make(64, "bf16", lens, 1, d, 16)
    one = PC.bf16_bits(np.ones((1, d)))
    first = np.zeros((1, d))
    first[0, 0] = -1.0
    for s, n in enumerate(lens):
        for t, k, v in ((n - 2, PC.bf16_bits(first), one), (n - 1, PC.bf16_bits(0 * first), one ^ 0x8000)):
            at = case.tables[s][t // 16], t % 16
            case.k[at], case.v[at] = k, v
    q64 = np.random.default_rng(65).standard_normal((S, hq, d))
    q64[..., 0] = np.random.default_rng(66).uniform(0.0, 1.0, (S, hq))
    q64 = GC.OA.to_f64(PC.bf16_bits(q64), "bf16")
    q = q64.astype(np.float32) if q_type == "f32" else PC.bf16_bits(q64)
    got = decode(lib, case, q, q_type, 0.999, "f32", window=2)
    p = np.exp(-q64[..., 0] * float(np.float32(0.999)))
    err = np.abs(got - ((p - 1) / (p + 1))[..., None]).max()
    assert err <= 15 * 2.0 ** -23, err


@pytest.mark.parametrize("q_type", ["bf16", "f32"])
def test_decode_weights_of_fp8_caches_in_two_parts(lib, q_type):
    """FP8 caches, bf16 outputs: a bf16 output is the float32 one rounded.

    Two keys with logits 0 and -0.005 < z <= 0 and values +1 and -1, as above: the outputs are
    below 0.0025, so their rounding (2^-8 of them) is below 2^-16, and one fp16 part (2^-11 of a
    weight) would not pass.  In units of 2^-23: the argument (1), ex2.approx (2) and the parts 2^-22
    (2) on numerator and denominator, 10; the sums (6), l and the quotient (2): 18."""
    S, hq, kv = 64, 8, "fp8_e4m3"
    lens = [34 + (s % 30) for s in range(S)]         # both tokens in chunk 32 .. 63
    case = PC.make(67, kv, lens, 1, 128, 16, scales="head")
    case.ks[:], case.vs[:] = 1.0, 2.0 ** -6
    first = np.zeros((1, 128), dtype=np.float32)
    first[0, 0] = -1.0
    for s, n in enumerate(lens):
        for t, k, v in ((n - 2, first, 64.0), (n - 1, 0 * first, -64.0)):
            at = case.tables[s][t // 16], t % 16
            case.k[at] = OB.encode(k, kv)
            case.v[at] = OB.encode(np.full((1, 128), v, dtype=np.float32), kv)
    q64 = np.zeros((S, hq, 128))
    q64[..., 0] = np.random.default_rng(69).uniform(0.0, 0.005, (S, hq))
    q64 = GC.OA.to_f64(PC.bf16_bits(q64), "bf16")
    q = q64.astype(np.float32) if q_type == "f32" else PC.bf16_bits(q64)
    p = np.exp(-q64[..., 0] * float(np.float32(0.999)))
    want = ((p - 1) / (p + 1))[..., None]
    for out in ("bf16", "f32"):
        got = decode(lib, case, q, q_type, 0.999, out, window=2)
        lim = 18 * 2.0 ** -23 + (2.0 ** -8 * np.abs(want) if out == "bf16" else 0.0)
        assert (np.abs(got - want) <= lim).all(), (out, float((np.abs(got - want) / lim).max()))
