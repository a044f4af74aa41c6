"""Refusals of the block-scaled cache's and the windowed attention's calls (no GPU: every
argument is checked before a launch), and pins of their oracle."""
import ctypes as C

import numpy as np
import pytest
import torch

from oracle import block_scaled as OB
from oracle import attention as OA
from tests import paged_cases as PC

OK, INVALID, UNSUPPORTED = 0, 1, 5
PTR = C.c_void_p(1 << 20)      # aligned, never dereferenced: the calls below are refused first


def quantize(lib, **kw):
    a = dict(k_new=PTR, v_new=PTR, qs=PTR, bt=PTR, ctx=PTR, kc=PTR, vc=PTR, ks=PTR, vs=PTR, S=2, T=8,
             mq=4, hkv=2, d=64, bs=16, nb=10, mb=4, stride=2, src=1, dst=2)
    a.update(kw)
    return lib.library().quantize_and_cache(*a.values(), None, None)


def gather(lib, **kw):
    a = dict(kc=PTR, vc=PTR, bt=PTR, rs=PTR, fp=None, S=2, n=8, mx=4, hkv=2, d=64, bs=16, nb=10, mb=4,
             kv=2, ks=PTR, vs=PTR, stride=2, out=1, ko=PTR, vo=PTR)
    a.update(kw)
    return lib.library().gather_cache(*a.values(), None, None)


def decode(lib, **kw):
    a = dict(q=PTR, kc=PTR, vc=PTR, bt=PTR, ctx=PTR, S=2, hq=8, hkv=2, d=128, bs=16, nb=10, mb=4, mx=64,
             scale=0.1, qt=1, kv=1, ks=None, vs=None, stride=0, window=8, sinks=2, ot=0, out=PTR,
             ws=None, wsb=0, part=0)
    a.update(kw)
    return lib.library().paged_attention_decode_window(*a.values(), None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(S=-1), INVALID), (dict(T=-1), INVALID), (dict(hkv=0), INVALID), (dict(nb=0), INVALID),
    (dict(mb=0), INVALID), (dict(stride=1), INVALID), (dict(mq=9), INVALID),
    (dict(qs=None), INVALID), (dict(qs=None, mq=1, T=1), INVALID),
    (dict(dst=1), UNSUPPORTED), (dict(dst=0), UNSUPPORTED), (dict(src=2), UNSUPPORTED),
    (dict(d=72), UNSUPPORTED), (dict(bs=24), UNSUPPORTED), (dict(bs=8192), UNSUPPORTED),
    (dict(S=65536, T=65536), UNSUPPORTED), (dict(mb=1 << 28), INVALID),
    (dict(k_new=None), INVALID), (dict(v_new=None), INVALID), (dict(bt=None), INVALID),
    (dict(ctx=None), INVALID), (dict(kc=None), INVALID), (dict(ks=None), INVALID),
    (dict(vs=None), INVALID), (dict(k_new=C.c_void_p(8)), INVALID), (dict(kc=C.c_void_p(24)), INVALID),
    (dict(bt=C.c_void_p(2)), INVALID), (dict(S=0), OK), (dict(mq=0), OK)])
def test_quantize_refusals(lib, kw, want):
    assert quantize(lib, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(S=-1), INVALID), (dict(n=-1, mx=-1), INVALID), (dict(mx=9), INVALID), (dict(hkv=0), INVALID),
    (dict(kv=7), UNSUPPORTED), (dict(out=2), UNSUPPORTED), (dict(d=24), UNSUPPORTED),
    (dict(bs=3), UNSUPPORTED), (dict(stride=1), INVALID), (dict(ks=None), INVALID),
    (dict(kc=None), INVALID), (dict(rs=None), INVALID), (dict(ko=None), INVALID),
    (dict(vo=C.c_void_p(4)), INVALID), (dict(rs=C.c_void_p(1)), INVALID),
    (dict(S=0), OK), (dict(mx=0), OK)])
def test_gather_refusals(lib, kw, want):
    assert gather(lib, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(window=0, sinks=1), INVALID),
    (dict(hq=7), INVALID), (dict(part=100), INVALID), (dict(part=-64), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID), (dict(mx=65), INVALID),
    (dict(kv=0), UNSUPPORTED), (dict(d=96), UNSUPPORTED), (dict(kv=2, d=64, ks=PTR, vs=PTR), UNSUPPORTED),
    (dict(qt=2), UNSUPPORTED), (dict(ot=3), UNSUPPORTED), (dict(hq=34), UNSUPPORTED),
    (dict(bs=4, mx=16), UNSUPPORTED), (dict(bs=12, mx=48), UNSUPPORTED), (dict(nb=1 << 31), UNSUPPORTED),
    (dict(kv=2), INVALID), (dict(kv=2, ks=PTR, vs=PTR, stride=1), INVALID),
    (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(out=C.c_void_p(8)), INVALID),
    (dict(bt=C.c_void_p(2)), INVALID), (dict(S=0), OK)])
def test_decode_refusals(lib, kw, want):
    assert decode(lib, **kw) == want


def test_workspace_covers_what_a_query_sees(lib):
    w = lib.library().paged_attention_window_workspace_bytes
    # 4 sinks and a window of 512 touch at most 1 + 17 chunks of 32 tokens
    assert w(2, 8, 2, 128, 100000, 64, 512, 4) == 2 * 8 * 9 * 130 * 4
    assert w(2, 8, 2, 128, 100000, 128, 512, 4) == 0      # few CTAs, up to 8 partitions: none
    assert w(200, 8, 2, 128, 100000, 128, 512, 4) == 200 * 8 * 5 * 130 * 4
    assert w(2, 8, 2, 128, 100000, 320, 256, 4) == 0
    assert w(2, 8, 2, 128, 640, 64, 0, 0) == 2 * 8 * 10 * 130 * 4
    assert w(2, 8, 2, 128, 640, 64, 10 ** 9, 10 ** 9) == 2 * 8 * 10 * 130 * 4
    assert w(2, 7, 2, 128, 640, 64, 0, 0) == 0


def test_python_refusals(lib):
    nb, bs, hkv, d, S = 6, 16, 2, 128, 2
    k8 = torch.zeros((nb, bs, hkv, d), dtype=torch.int8)
    sc, ctx = torch.ones((nb, hkv)), torch.ones(S, dtype=torch.int32)
    bt = torch.zeros((S, 3), dtype=torch.int32)
    new = torch.zeros((S, hkv, d), dtype=torch.bfloat16)
    q = torch.zeros((S, 4, d), dtype=torch.bfloat16)

    def quant(**kw):
        a = dict(k_new=new, v_new=new, k_cache=k8, v_cache=k8, k_scales=sc, v_scales=sc,
                 block_tables=bt, context_lens=ctx)
        a.update(kw)
        lib.quantize_and_cache(**a)

    def dec(**kw):
        a = dict(q=q, k_cache=k8, v_cache=k8, block_tables=bt, context_lens=ctx, scale=0.1,
                 max_context_len=48, k_scale=sc, v_scale=sc)
        a.update(kw)
        lib.paged_attention_decode(**a)

    for kw in (dict(), dict(k_new=new[:, :1]), dict(v_new=new.float()), dict(k_new=new.half()),
               dict(k_scales=sc[0]), dict(k_scales=sc[:3]), dict(v_scales=sc.double()),
               dict(context_lens=ctx.long()), dict(block_tables=bt[:1]), dict(v_cache=k8[:3]),
               dict(query_start=torch.zeros(S, dtype=torch.int32))):
        with pytest.raises(ValueError):      # the first: no CPU path
            quant(**kw)
    for kw in (dict(), dict(k_scale=None), dict(v_scale=sc[0]), dict(k_scale=sc[:, :1], v_scale=sc[:, :1]),
               dict(context_lens=ctx[:1]), dict(q=q.half()), dict(block_tables=bt.long()),
               dict(out=torch.zeros((S, 4, d)), out_dtype=torch.bfloat16)):
        with pytest.raises(ValueError):
            dec(**kw)
    for kw in (dict(k_new=None), dict(k_cache=3), dict(max_query_len="a"), dict(max_query_len=1 << 40)):
        with pytest.raises(ValueError):
            quant(**kw)
    for kw in (dict(scale="x"), dict(window=1.5), dict(window=1 << 33), dict(out_dtype=torch.float16),
               dict(out_dtype="bf16"), dict(workspace=7)):
        with pytest.raises((ValueError, TypeError)):
            dec(**kw)
    with pytest.raises(ValueError):
        lib._binding().decode_window(q)
    rs = torch.zeros(S + 1, dtype=torch.int32)
    for kw in (dict(), dict(row_start=rs[:2]), dict(row_start=rs.long()), dict(k_scale=None),
               dict(first_pos=ctx[:1]), dict(block_tables=bt.long())):
        a = dict(k_cache=k8, v_cache=k8, block_tables=bt, row_start=rs, num_rows=4, max_rows=2,
                 k_scale=sc, v_scale=sc)
        a.update(kw)
        with pytest.raises(ValueError):
            lib.gather_cache(**a)


# ---- the oracle -------------------------------------------------------------------
def test_oracle_visible():
    assert OB.visible(5, 0, 0).tolist() == [0, 1, 2, 3, 4, 5]
    assert OB.visible(9, 3, 2).tolist() == [0, 1, 7, 8, 9]
    assert OB.visible(9, 1, 0).tolist() == [9]
    assert OB.visible(3, 3, 2).tolist() == [0, 1, 2, 3]
    assert OB.visible(0, 1, 4).tolist() == [0]


def test_oracle_window_matches_masked_softmax():
    rng = np.random.default_rng(0)
    n, L, hq, hkv, d = 5, 40, 4, 2, 16
    q, K, V = rng.standard_normal((n, hq, d)), rng.standard_normal((L, hkv, d)), rng.standard_normal((L, hkv, d))
    pos = np.arange(L - n, L)
    o, mag, _ = OB.attend(q, pos, K, V, 0.25, 8, 3)
    k, v = (torch.from_numpy(np.repeat(x, hq // hkv, 1)) for x in (K, V))
    z = torch.einsum("nhd,lhd->nhl", torch.from_numpy(q), k) * 0.25
    i, j = torch.from_numpy(pos)[:, None, None], torch.arange(L)
    z = z.masked_fill(~((j <= i) & ((i - j < 8) | (j < 3))), float("-inf"))
    want = torch.einsum("nhl,lhd->nhd", z.softmax(-1), v)
    assert np.abs(o - want.numpy()).max() < 1e-13
    assert (mag >= np.abs(o) - 1e-15).all()


@pytest.mark.parametrize("kv", ["fp8_e4m3", "int8"])
def test_oracle_append(kv):
    """Scale of a fresh block, growth by the least power of two, codes that move with it."""
    case = PC.make(1, kv, [6], 1, 16, 4)
    b0, b1 = case.tables[0]
    x = np.zeros((6, 1, 16), dtype=np.float32)
    x[:4, 0, 0], x[4:, 0, 0] = [1, 2, 3, 4], [1, 5]
    q = OB.QMAX[kv]
    OB.quantize_and_cache(x[:4], x[:4], [0, 4], case.tables, [4], case.k, case.v, case.ks, case.vs, "f32", kv)
    assert case.ks[b0, 0] == np.float32(4) / q
    OB.quantize_and_cache(x[4:5], x[4:5], [0, 1], case.tables, [5], case.k, case.v, case.ks, case.vs, "f32", kv)
    assert case.ks[b1, 0] == np.float32(1) / q
    c = OB.code_values(case.k[b1, 0, 0, 0], kv)
    assert c == q
    OB.quantize_and_cache(x[5:], x[5:], [0, 1], case.tables, [6], case.k, case.v, case.ks, case.vs, "f32", kv)
    assert case.ks[b1, 0] == np.float32(1) / q * 8       # 5 <= 8
    assert OB.code_values(case.k[b1, 0, 0, 0], kv) == (np.rint(c / 8) if kv == "int8" else c / 8)
    assert OB.grown_scale(np.float32(1), np.float32(448), np.float32(448)) == (1, 0)
    assert OB.grown_scale(np.float32(1), np.float32(449), np.float32(448)) == (2, 1)
    y = OB.gather(case.k, case.ks, case.tables[0], 0, 6, kv)
    assert np.abs(y - x).max() <= (5 / 127 * 2 if kv == "int8" else 5 * 2.0 ** -4)


def test_oracle_gather_of_codes_is_the_static_dequant():
    case = PC.make(2, "fp8_e4m3", [9], 2, 16, 4, scales="head")
    y = OB.gather(case.k, case.ks, case.tables[0], 2, 5, "fp8_e4m3")
    rows = OA.gather_sequence(case.k, case.tables[0], 9)[2:7]
    assert np.array_equal(y.astype(np.float64), OA.fp8_dequant(rows, case.ks))


def prefill(lib, **kw):
    a = dict(q=PTR, qs=PTR, kc=PTR, vc=PTR, bt=PTR, ctx=PTR, S=2, T=8, mq=4, hq=8, hkv=2, d=128, bs=16,
             nb=10, mb=4, mx=64, scale=0.1, causal=1, qt=1, kv=1, ks=None, vs=None, stride=0, window=8,
             sinks=2, ot=0, out=PTR)
    a.update(kw)
    return lib.library().paged_attention_prefill_window(*a.values(), None, None)


@pytest.mark.parametrize("kw,want", [
    (dict(window=-1), INVALID), (dict(sinks=-1), INVALID), (dict(window=0), INVALID),
    (dict(causal=0), INVALID), (dict(causal=2), INVALID), (dict(hq=7), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(mx=65), INVALID), (dict(mq=9), INVALID),
    (dict(mb=1 << 28), INVALID), (dict(kv=0), UNSUPPORTED), (dict(qt=0), UNSUPPORTED),
    (dict(d=64), UNSUPPORTED), (dict(ot=2), UNSUPPORTED), (dict(hq=34), UNSUPPORTED),
    (dict(bs=4, mx=16), UNSUPPORTED), (dict(nb=1 << 31), UNSUPPORTED), (dict(kv=3), INVALID),
    (dict(kv=3, ks=PTR, vs=PTR, stride=1), INVALID), (dict(q=None), INVALID), (dict(qs=None), INVALID),
    (dict(out=C.c_void_p(4)), INVALID), (dict(qs=C.c_void_p(2)), INVALID), (dict(S=0), OK),
    (dict(mq=0), OK)])
def test_prefill_refusals(lib, kw, want):
    assert prefill(lib, **kw) == want


def test_sizes_past_32_bits_are_refused(lib):
    """Places within a block, and sequences times heads, are 32-bit in the kernels."""
    assert quantize(lib, bs=4096, hkv=4096, d=1024, stride=4096, mb=4) == UNSUPPORTED
    assert decode(lib, S=65535, hq=32767 * 2, hkv=32767) == UNSUPPORTED


def test_status_word_is_checked(lib):
    k8 = torch.zeros((4, 16, 2, 128), dtype=torch.int8)
    sc, n = torch.ones((4, 2)), torch.ones(1, dtype=torch.int32)
    bt, rows = torch.zeros((1, 2), dtype=torch.int32), torch.zeros((1, 2, 128))
    start = torch.zeros(2, dtype=torch.int32)
    q = torch.zeros((1, 4, 128), dtype=torch.bfloat16)
    for bad in (torch.zeros(1, dtype=torch.uint8), torch.zeros(0, dtype=torch.int32)):
        kw = dict(device_status=bad)
        for call in (lambda: lib.quantize_and_cache(rows, rows, k8, k8, sc, sc, bt, n, **kw),
                     lambda: lib.gather_cache(k8, k8, bt, start, 1, 1, k_scale=sc, v_scale=sc, **kw),
                     lambda: lib.paged_attention_decode(q, k8, k8, bt, n, 0.1, 32, k_scale=sc, v_scale=sc,
                                                        **kw),
                     lambda: lib.paged_attention_prefill(q, start, k8, k8, bt, n, 0.1, 1, 32, k_scale=sc,
                                                         v_scale=sc, **kw)):
            with pytest.raises(ValueError, match="device_status"):
                call()


def test_calls_with_one_scale_per_head_refuse_block_scales(lib):
    k8 = torch.zeros((4, 16, 2, 128), dtype=torch.int8)
    sc, n = torch.ones((4, 2)), torch.ones(1, dtype=torch.int32)
    bt, rows = torch.zeros((1, 2), dtype=torch.int32), torch.zeros((1, 2, 128))
    slots = torch.zeros(1, dtype=torch.int64)
    q, out = torch.zeros((1, 4, 128), dtype=torch.bfloat16), torch.zeros((1, 4, 128))
    kw = dict(k_scale=sc, v_scale=sc)
    for call in (lambda: lib.reshape_and_cache(rows, rows, slots, k8, k8, **kw),
                 lambda: lib.paged_attention_decode_append(q, rows, rows, slots, k8, k8, bt, n, 0.1, 32, **kw),
                 lambda: lib.paged_attention_decode_noalloc(q, k8, k8, bt, n, 0.1, 32, out, **kw)):
        with pytest.raises(ValueError, match="per head"):
            call()


@pytest.mark.parametrize("per_block", ["k_scale", "v_scale"])
def test_scales_of_two_forms_are_refused(lib, per_block):
    """One scale per head beside scales per block: refused whichever of the two it is."""
    k8 = torch.zeros((4, 16, 2, 128), dtype=torch.int8)
    n, bt = torch.ones(1, dtype=torch.int32), torch.zeros((1, 2), dtype=torch.int32)
    start = torch.tensor([0, 1], dtype=torch.int32)
    q = torch.zeros((1, 4, 128), dtype=torch.bfloat16)
    kw = {"k_scale": torch.ones(2), "v_scale": torch.ones(2), per_block: torch.ones((4, 2))}
    for call in (lambda **m: lib.paged_attention_decode(q, k8, k8, bt, n, 0.1, 32, **kw, **m),
                 lambda **m: lib.paged_attention_prefill(q, start, k8, k8, bt, n, 0.1, 1, 32, **kw, **m)):
        for more in ({}, {"window": 8}):
            with pytest.raises(ValueError, match="k_scale and v_scale must be"):
                call(**more)


@pytest.mark.parametrize("hq,hkv,d", [(32, 8, 128), (8, 8, 64), (16, 1, 256), (20, 2, 128), (96, 8, 128)])
@pytest.mark.parametrize("window,sinks,part", [(0, 0, 0), (1024, 4, 0), (16000, 129, 0), (0, 0, 64),
                                               (700, 64, 320)])
def test_workspace_of_the_largest_call_covers_the_smaller_ones(lib, hq, hkv, d, window, sinks, part):
    """A buffer sized once for the most sequences and the longest context is enough for every
    smaller call of either cache width, and does not shrink as the sizes grow."""
    L = lib.library()
    sizes = [1, 2, 3, 5, 8, 13, 16, 33, 64, 100, 257]
    ctxs = [1, 64, 65, 200, 1024, 1536, 3071, 4096, 6144, 8192, 20000, 65536, 131072, 300000]

    def bound(s, c):
        return L.paged_attention_window_workspace_bytes(s, hq, hkv, d, c, part, window, sinks)

    for s in sizes:
        for c in ctxs:
            need = max(L.paged_attention_window_call_bytes(s, hq, hkv, d, c, part, window, sinks, kv)
                       for kv in (lib.BF16, lib.FP8_E4M3))
            assert need <= bound(s, c)
            for s2, c2 in ((sizes[-1], c), (s, ctxs[-1]), (s + 1, c), (s, c + 64), (sizes[-1], ctxs[-1])):
                assert need <= bound(s2, c2), (s, c, s2, c2)
                assert bound(s, c) <= bound(s2, c2), (s, c, s2, c2)


def test_workspace_query_refuses_nothing_to_size(lib):
    w = lib.library().paged_attention_window_call_bytes
    assert w(2, 7, 2, 128, 640, 64, 0, 0, lib.BF16) == 0
    assert w(0, 8, 2, 128, 640, 64, 0, 0, lib.BF16) == 0
    assert w(2, 8, 2, 128, 640, 64, 0, 0, lib.BF16) == 2 * 8 * 10 * 130 * 4
    assert w(2, 8, 2, 128, 640, 100, 0, 0, lib.BF16) == 0


def test_scales_per_head_in_a_column_are_taken(lib):
    """A contiguous ``[Hkv, 1]`` (or ``[1, Hkv]``) holds one scale per head: every call gets past
    its checks of the scales (and stops at the CPU tensors)."""
    hkv = 2
    k8 = torch.zeros((4, 16, hkv, 128), dtype=torch.int8)
    n, bt = torch.ones(1, dtype=torch.int32), torch.zeros((1, 2), dtype=torch.int32)
    start = torch.tensor([0, 1], dtype=torch.int32)
    rows, slots = torch.zeros((1, hkv, 128)), torch.zeros(1, dtype=torch.int64)
    q, out = torch.zeros((1, 4, 128), dtype=torch.bfloat16), torch.zeros((1, 4, 128))
    for shape in ((hkv, 1), (1, hkv), (hkv,)):
        kw = dict(k_scale=torch.ones(shape), v_scale=torch.ones(shape))
        for call in (lambda: lib.reshape_and_cache(rows, rows, slots, k8, k8, **kw),
                     lambda: lib.paged_attention_decode_append(q, rows, rows, slots, k8, k8, bt, n, 0.1, 32, **kw),
                     lambda: lib.paged_attention_decode_noalloc(q, k8, k8, bt, n, 0.1, 32, out, **kw),
                     lambda: lib.paged_attention_decode(q, k8, k8, bt, n, 0.1, 32, **kw),
                     lambda: lib.paged_attention_decode(q, k8, k8, bt, n, 0.1, 32, window=8, **kw),
                     lambda: lib.paged_attention_prefill(q, start, k8, k8, bt, n, 0.1, 1, 32, **kw),
                     lambda: lib.paged_attention_prefill(q, start, k8, k8, bt, n, 0.1, 1, 32, window=8, **kw),
                     lambda: lib.gather_cache(k8, k8, bt, start, 1, 1, **kw)):
            with pytest.raises(ValueError, match="CUDA tensor"):
                call()
        with pytest.raises(ValueError, match="num_blocks"):
            lib.quantize_and_cache(rows, rows, k8, k8, *kw.values(), bt, n)
    one = torch.zeros((1, 16, hkv, 128), dtype=torch.int8)      # a pool of one block
    with pytest.raises(ValueError, match="CUDA tensor"):
        lib.quantize_and_cache(rows, rows, one, one, torch.ones(1, hkv), torch.ones(1, hkv), bt, n)


def test_causal_must_be_a_truth_value(lib):
    k, n = torch.zeros((4, 16, 2, 128), dtype=torch.bfloat16), torch.ones(1, dtype=torch.int32)
    bt, start = torch.zeros((1, 2), dtype=torch.int32), torch.tensor([0, 1], dtype=torch.int32)
    q = torch.zeros((1, 4, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="causal"):
        lib.paged_attention_prefill(q, start, k, k, bt, n, 0.1, 1, 32, causal=np.array([1, 0]), window=8)
