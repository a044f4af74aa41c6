"""A whole run on a PagedKVCache with block scales: prompts in ragged chunks with chunked
prefill, forked beams with copy-on-write, decode steps with a window and sinks, sequences
swapped to host memory and back, the cache read back - against the oracle pool and the
numpy definitions; codes and scales bit for bit."""
import numpy as np
import pytest

from oracle import attention as OA
from oracle import block_scaled as OB
from oracle import pool as OP
from tests import paged_cases as PC
from tests.gpu_cases import CODE, from_torch, to_torch

pytestmark = pytest.mark.gpu


class Mirror:
    """The engine's steps on the oracle pool and numpy caches."""

    def __init__(self, L, hkv, d, bs, nb, kv, order, H):
        self.op = OP.Pool(L, hkv, d, bs, 1, nb, initial_free_order=order.tolist())
        self.op.host_init(H)
        poison = 0x7F if kv == "fp8_e4m3" else 127
        dt = np.uint8 if kv == "fp8_e4m3" else np.int8
        self.cache = np.full((L, 2, nb, bs, hkv, d), poison, dtype=dt)
        self.scales = np.full((L, 2, nb, -(-hkv // 4) * 4), np.nan, dtype=np.float32)
        self.host = np.zeros((H, L, 2, bs, hkv, d), dtype=dt)
        self.host_scales = np.zeros((H,) + self.scales.shape[:2] + self.scales.shape[3:], dtype=np.float32)
        self.kv = kv

    def copies(self, pairs):
        OA.copy_blocks(self.cache, pairs)
        OA.copy_blocks(self.scales, pairs)

    def swap(self, pairs, out):
        OA.swap_blocks(self.cache, self.host, pairs, out)
        OA.swap_blocks(self.scales, self.host_scales, pairs, out)

    def append(self, l, k, v, starts, tables, lens):
        OB.quantize_and_cache(k, v, starts, tables, lens, self.cache[l, 0], self.cache[l, 1],
                              self.scales[l, 0], self.scales[l, 1], "bf16", self.kv)

    def paged(self, l, tables, lens):
        s = np.nan_to_num(self.scales[l])
        return PC.Paged(self.kv, [int(x) for x in lens], np.asarray(tables), self.cache[l, 0],
                        self.cache[l, 1], s[0], s[1])


def check(got, paged, q, starts, scale, window, sinks, out_bf16, hi_lo):
    q64 = OA.to_f64(q, "bf16")
    for s, c in enumerate(paged.lens):
        a, b = int(starts[s]), int(starts[s + 1])
        K, V = paged.values(s)
        o, mag, reach = OB.attend(q64[a:b], np.arange(c - (b - a), c), K, V, scale, window, sinks)
        lim = PC.attention_bound(paged, q64[a:b], o, mag, reach, scale, False, out_bf16, hi_lo, c)
        assert (np.abs(got[a:b] - o) <= lim).all()


@pytest.mark.parametrize("kv,hkv,window,sinks", [("fp8_e4m3", 2, 0, 0), ("int8", 3, 24, 5)])
def test_run(lib, kv, hkv, window, sinks):
    import torch
    import paged_kv_cache_295_gb300 as pkv
    from paged_kv_cache_295_gb300.engine import PagedKVCache
    L, hq, d, bs, nb, H = 2, hkv * 4, 128, 16, 96, 40
    r = np.random.default_rng(hkv)
    order = r.permutation(nb).astype(np.int32)
    eng = PagedKVCache(L, hkv, d, bs, nb, CODE[kv], initial_free_order=order, block_scales=True)
    eng.host_area(H)
    m = Mirror(L, hkv, d, bs, nb, kv, order, H)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = lambda n, h: PC.bf16_bits(r.standard_normal((n, h, d)) * np.exp(0.7 * r.standard_normal((n, 1, 1))))

    def view(ids):
        mb = max(len(m.op.tables[i]) for i in ids)
        tables, lens = eng.pool.batch_tables(ids, mb)
        t, n = m.op.padded_tables(ids, mb)
        assert np.array_equal(tables, np.asarray(t)) and np.array_equal(lens, n)
        return tables, lens, torch.from_numpy(tables).cuda(), torch.from_numpy(lens).cuda()

    # prompts in two ragged chunks each, attended by prefill
    ids, chunks = [0, 1, 2], [[37, 5, 64], [9, 30, 1]]
    for i in ids:
        eng.pool.seq_create(i)
        m.op.seq_create(i)
    for new in chunks:
        for i, n in zip(ids, new):
            assert eng.pool.append_tokens(i, n).tolist() == m.op.seq_append_tokens(i, n)
        tables, lens, td, ld = view(ids)
        starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        sd = torch.from_numpy(starts).cuda()
        for l in range(L):
            k, v, q = rows(sum(new), hkv), rows(sum(new), hkv), rows(sum(new), hq)
            eng.append_rows(l, to_torch(k, "bf16"), to_torch(v, "bf16"), td, ld, query_start=sd,
                            max_query_len=max(new), device_status=status)
            out = eng.prefill(l, to_torch(q, "bf16"), sd, td, ld, max(new), int(lens.max()),
                              device_status=status, window=window, sinks=sinks)
            m.append(l, k, v, starts, tables, lens)
            check(out.cpu().numpy(), m.paged(l, tables, lens), q, starts, eng.scale, window, sinks,
                  False, False)
    # a beam of each, then decode steps across a block boundary; one sequence swapped in between
    for i in ids:
        n = eng.pool.seq_length(i)
        eng.pool.seq_fork_prefix(10 + i, i, n)
        m.op.seq_fork_prefix(10 + i, i, n)
    beams = ids + [10 + i for i in ids]
    copied = 0
    for step in range(bs + 1):
        if step == 5:     # beam 10 goes to host memory and comes back
            pairs = eng.swap_out(10, device_status=status)
            assert [tuple(x) for x in pairs.tolist()] == m.op.seq_swap_out(10)
            m.swap(pairs.tolist(), True)
            pairs = eng.swap_in(10, device_status=status)
            assert [tuple(x) for x in pairs.tolist()] == m.op.seq_swap_in(10)
            m.swap(pairs.tolist(), False)
        assert eng.pool.append_slots(beams).tolist() == m.op.seq_append_slots(beams)
        pairs = eng.run_copies(device_status=status)
        assert [tuple(x) for x in pairs.tolist()] == m.op.take_copies()
        m.copies(pairs.tolist())
        copied += len(pairs)
        tables, lens, td, ld = view(beams)
        starts = np.arange(len(beams) + 1)
        for l in range(L):
            k, v, q = rows(len(beams), hkv), rows(len(beams), hkv), rows(len(beams), hq)
            out = eng.append_attend(l, to_torch(q, "bf16"), to_torch(k, "bf16"), to_torch(v, "bf16"),
                                    None, td, ld, int(lens.max()), device_status=status,
                                    window=window, sinks=sinks, out_dtype=torch.bfloat16)
            m.append(l, k, v, starts, tables, lens)
            check(out.float().cpu().numpy(), m.paged(l, tables, lens), q, starts, eng.scale, window,
                  sinks, True, False)
    assert copied and int(status.item()) == 0
    assert from_torch(eng.storage, kv).tobytes() == m.cache.tobytes()
    got = eng.scales.cpu().numpy()[..., :hkv]
    assert np.array_equal(got, m.scales[..., :hkv], equal_nan=True)
    # read back everything of two sequences
    tables, lens, td, ld = view([1, 12])
    starts = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    k, v = eng.gather(1, td, torch.from_numpy(starts).cuda(), int(starts[-1]), int(lens.max()),
                      out_dtype=torch.float32, device_status=status)
    p = m.paged(1, tables, lens)
    for s in range(2):
        K, V = p.values(s)
        assert np.array_equal(k[starts[s]:starts[s + 1]].cpu().numpy(), K.astype(np.float32))
        assert np.array_equal(v[starts[s]:starts[s + 1]].cpu().numpy(), V.astype(np.float32))


def test_window_on_a_bf16_cache(lib):
    """append_attend with a window is the append, then the windowed call."""
    import torch
    from paged_kv_cache_295_gb300.engine import PagedKVCache
    eng = [PagedKVCache(1, 2, 128, 16, 40, lib.BF16) for _ in range(2)]
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    k, v = rnd(70, 2, 128), rnd(70, 2, 128)
    kn, vn, q = rnd(1, 2, 128), rnd(1, 2, 128), rnd(1, 8, 128)
    outs = []
    for i, e in enumerate(eng):
        e.pool.seq_create(0)
        e.append(0, k, v, torch.from_numpy(e.pool.append_tokens(0, 70)).cuda())
        slots = torch.from_numpy(e.pool.append_slots([0])).cuda()
        t, n = (torch.from_numpy(x).cuda() for x in e.pool.batch_tables([0], 8))
        if i == 0:
            outs.append(e.append_attend(0, q, kn, vn, slots, t, n, 71, window=20, sinks=4))
        else:
            e.append(0, kn, vn, slots)
            outs.append(lib.paged_attention_decode(q, e.k_cache(0), e.v_cache(0), t, n, e.scale, 71,
                                                   window=20, sinks=4))
    assert torch.equal(*outs)


def test_refusals(lib):
    from paged_kv_cache_295_gb300.engine import PagedKVCache
    with pytest.raises(ValueError):
        PagedKVCache(1, 2, 128, 16, 8, lib.BF16, block_scales=True)
    e = PagedKVCache(1, 2, 128, 16, 8, lib.INT8, block_scales=True)
    with pytest.raises(ValueError):
        e.append(0, None, None, None)
    with pytest.raises(ValueError):
        lib.DecodeGraph(e, 8, 4, [1])
    with pytest.raises(ValueError):
        PagedKVCache(1, 2, 128, 16, 8, lib.INT8).append_rows(0, None, None, None, None)
