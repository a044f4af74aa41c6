"""The step around the cache as a whole: slots from lengths, rotary positions with the append and
attention, prompts and then tokens, against float64."""
import numpy as np
import pytest

from oracle import step as OS
from tests import paged_cases as PC
from tests.test_gpu_packed import BF16

pytestmark = pytest.mark.gpu

HQ, HKV, D, BS = 8, 2, 128, 16
FREQ = 10000.0 ** (-np.arange(64) / 64)


def dev(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


class Model:
    """One layer's rows of a few sequences, their positions on three axes, and what float64 makes of
    them."""

    def __init__(self, lib, kv, seed):
        from paged_kv_cache_295_gb300.engine import PagedKVCache
        self.lib, self.rng = lib, np.random.default_rng(seed)
        self.cache = PagedKVCache(1, HKV, D, BS, 120, kv, initial_free_order=self.rng.permutation(120).tolist())
        if kv == lib.FP8_E4M3:
            self.cache.k_scale.fill_(4.0 / 448)
            self.cache.v_scale.fill_(4.0 / 448)
        self.kv = kv
        self.rotary = lib.Rotary(D, sections=[16, 24, 24])
        self.axes = [0] * 16 + [1] * 24 + [2] * 24
        self.rows = {}      # sequence: float64 K (turned), V so far

    def step(self, rows):
        """Rows [T, HQ + 2 HKV, D] in bf16, as a projection leaves them."""
        import torch
        return torch.from_numpy(self.rng.standard_normal((rows, HQ + 2 * HKV, D)).astype(np.float32)).cuda().bfloat16()

    def grid(self, positions):
        """Time, height and width from a token's place: rows of 7."""
        import torch
        return torch.stack([positions // 49, positions // 7 % 7, positions % 7]).to(torch.int32).contiguous()

    def turned(self, x, pos):
        return OS.rotary(x.double().cpu().numpy(), pos.cpu().numpy(), FREQ, self.axes)

    def remember(self, seqs, starts, k, v):
        for s, a, b in zip(seqs, starts[:-1], starts[1:]):
            old = self.rows.get(s, (np.zeros((0, HKV, D)), np.zeros((0, HKV, D))))
            self.rows[s] = tuple(np.concatenate([o, x[a:b]]) for o, x in zip(old, (k, v)))

    def check(self, got, seqs, starts, q, out_bf16, prompt):
        """Attention over the rows so far.  The operands are the float64 ones rounded: q and k to bf16 (2^-8
        of |q| |k| each in a score, whose effect on the weights is twice that), and in an 8-bit cache
        k and v to E4M3 (2^-4), on top of the kernels' own bound."""
        codes = self.kv == self.lib.FP8_E4M3 and not prompt
        for s, a, b in zip(seqs, starts[:-1], starts[1:]):
            k, v = self.rows[s]
            n = b - a
            o, mag, reach, seen = OS.packed(q[a:b], k, v, [0, n], [0, k.shape[0]], self.cache.scale)
            e_k, e_v = (2.0 ** -4, 2.0 ** -4) if codes else (2.0 ** -8, 0.0)
            if codes:      # the smallest codes: half of their step
                e_v_abs = 2.0 ** -10 * 4.0 / 448
                e_k_abs = 2.0 ** -10 * 4.0 / 448 * np.abs(q[a:b]).sum(-1)
            else:
                e_v_abs, e_k_abs = 0.0, 0.0
            dz = self.cache.scale * (reach * (2.0 ** -8 + e_k) + e_k_abs)
            bound = PC.attention_bound(BF16, q[a:b], o, mag, reach, self.cache.scale, False, out_bf16, not out_bf16,
                                       int(seen.max()))
            bound = bound + 2 * np.expm1(2 * dz)[..., None] * mag + e_v * mag + e_v_abs
            assert (np.abs(got[a:b].double().cpu().numpy() - o) <= bound).all()


@pytest.mark.parametrize("kv", ["BF16", "FP8_E4M3"])
def test_prompts_then_tokens(lib, kv):
    """Three prompts of very different lengths, a token each, one more prompt beside two of
    them, and a captured loop of tokens; the host pool, told of the same appends, has the same tables."""
    import torch
    m = Model(lib, getattr(lib, kv), 3)
    cache, pool = m.cache, m.cache.pool
    free, start = dev(pool.free_list()), dev([0])
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    tables, lens = torch.full((4, 40), -1, dtype=torch.int32, device="cuda"), dev([0, 0, 0, 0])

    def prompts(new):
        T = sum(new)
        x = m.step(T)
        q, k, v = x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]
        sl = cache.slots(tables, lens, dev(new), free, T, free_start=start, context_out=lens, free_next=start,
                         device_status=status)
        pos = m.grid(sl.positions)
        out = cache.prompt(0, q, k, v, pos, m.rotary, sl, out_dtype=torch.bfloat16, device_status=status)
        starts = [0, *np.cumsum(new)]
        m.remember(range(4), starts, m.turned(k, pos), v.double().cpu().numpy())
        seqs = [s for s in range(4) if new[s]]
        at = [starts[s] for s in seqs] + [T]
        m.check(out, seqs, at, m.turned(q, pos), True, True)

    def tell_the_pool(new):
        for s, n in enumerate(new):
            if n:
                if not any(s == x for x in told):
                    pool.seq_create(s)
                    told.append(s)
                pool.append_tokens(s, n)
        assert np.array_equal(tables[told].cpu().numpy(), pool.batch_tables(told, 40)[0])
        assert np.array_equal(lens[told].cpu().numpy(), pool.batch_tables(told, 40)[1])
        assert free[int(start.item()):].tolist() == pool.free_list()

    told = []
    prompts([37, 200, 1, 0])
    tell_the_pool([37, 200, 1, 0])

    x = torch.empty((4, HQ + 2 * HKV, D), dtype=torch.bfloat16, device="cuda")
    alive = dev([1, 1, 1, 0])
    slots = torch.empty(4, dtype=torch.int64, device="cuda")
    pos, q_out = torch.empty(4, dtype=torch.int32, device="cuda"), torch.empty((4, HQ, D), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((4, HQ, D), device="cuda")
    ws = cache.workspace_for(4, HQ, 640)

    def token():
        sl = cache.slots(tables, lens, alive, free, row_per_sequence=True, free_start=start, context_out=lens,
                         free_next=start, slot_mapping=slots, positions=pos, device_status=status)
        cache.append_rotary(0, x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], m.grid(sl.positions), m.rotary,
                            sl.slot_mapping, q_out=q_out, device_status=status)
        cache.attend(0, q_out, tables, lens, 640, out=out, workspace=ws, device_status=status)

    def check_token(new):
        torch.cuda.synchronize()
        g = m.grid(pos)
        k, v = m.turned(x[:, HQ:HQ + HKV], g), x[:, HQ + HKV:].double().cpu().numpy()
        q = m.turned(x[:, :HQ], g)
        for s in range(4):
            if new[s]:
                m.remember([s], [0, 1], k[s:s + 1], v[s:s + 1])
                m.check(out[s:s + 1], [s], [0, 1], q[s:s + 1], False, False)
            else:
                assert int(slots[s].item()) == -1
        tell_the_pool(new)

    for _ in range(3):
        x.copy_(m.step(4))
        token()
        check_token([1, 1, 1, 0])
    prompts([0, 0, 0, 50])
    tell_the_pool([0, 0, 0, 50])
    # a captured step: the lengths, the free list and the tables go on by themselves
    alive.copy_(dev([1, 0, 1, 1]))
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        token()
    for _ in range(20):
        x.copy_(m.step(4))
        g.replay()
        check_token([1, 0, 1, 1])
    assert int(status.item()) == 0


def test_chunk_behind_a_cached_prefix(lib):
    """A prompt's second chunk: its rows are rotated and appended, the attention reads the cache."""
    import torch
    m = Model(lib, lib.BF16, 5)
    cache = m.cache
    free, start, lens = dev(cache.pool.free_list()), dev([0]), dev([0, 0])
    tables = torch.full((2, 20), -1, dtype=torch.int32, device="cuda")
    for new in ([100, 3], [30, 77]):
        T = sum(new)
        x = m.step(T)
        q, k, v = x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]
        sl = cache.slots(tables, lens, dev(new), free, T, free_start=start, context_out=lens, free_next=start)
        pos = m.grid(sl.positions)
        qr, _ = cache.append_rotary(0, q, k, v, pos, m.rotary, sl.slot_mapping)
        out = cache.prefill(0, qr, sl.query_start, tables, lens, max(new), 320)
        starts = [0, *np.cumsum(new)]
        m.remember(range(2), starts, m.turned(k, pos), v.double().cpu().numpy())
        m.check(out, range(2), starts, m.turned(q, pos), False, False)


def test_prompt_equals_prefill_through_the_cache(lib):
    """The packed call and the paged one over the same rows, within both bounds."""
    import torch
    rng = np.random.default_rng(6)
    lens = [130, 1, 300]
    T, qs = sum(lens), dev([0, 130, 131, 431])
    q, k, v = (torch.from_numpy(rng.standard_normal((T, h, D)).astype(np.float32)).cuda().bfloat16()
               for h in (HQ, HKV, HKV))
    from paged_kv_cache_295_gb300.engine import PagedKVCache
    cache = PagedKVCache(1, HKV, D, BS, 40, lib.BF16)
    tables = torch.full((3, 20), -1, dtype=torch.int32, device="cuda")
    sl = cache.slots(tables, dev([0, 0, 0]), dev(lens), dev(cache.pool.free_list()), T)
    cache.append(0, k, v, sl.slot_mapping)
    for kw in ({}, {"window": 100, "sinks": 3}):
        a = cache.prefill(0, q, qs, tables, sl.context_lens, 300, 320, **kw)
        b = lib.packed_attention_prefill(q, k, v, qs, cache.scale, **kw)
        x = [t.double().cpu().numpy() for t in (q, k, v)]
        o, mag, reach, seen = OS.packed(*x, [0, 130, 131, 431], [0, 130, 131, 431], cache.scale, True,
                                        kw.get("window", 0), kw.get("sinks", 0))
        e = PC.attention_bound(BF16, x[0], o, mag, reach, cache.scale, False, False, True, 300)
        assert (np.abs((a - b).double().cpu().numpy()) <= 2 * e).all()


def test_engine_refusals(lib):
    import torch
    from paged_kv_cache_295_gb300.engine import PagedKVCache
    cache = PagedKVCache(1, 2, 128, 16, 4, lib.INT8, block_scales=True)
    q = torch.zeros((1, 2, 128), device="cuda", dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        cache.append_rotary(0, q, q, q, dev([0]), lib.Rotary(128), torch.zeros(1, dtype=torch.int64, device="cuda"))


def test_a_prompt_that_is_refused_appends_nothing(lib):
    import torch
    from paged_kv_cache_295_gb300.engine import PagedKVCache
    cache = PagedKVCache(num_layers=1, num_kv_heads=2, head_dim=64, block_size=16, num_blocks=4, kv_dtype=lib.F32)
    cache.k_cache(0).zero_()
    lens = torch.zeros(1, dtype=torch.int32, device="cuda")
    sl = cache.slots(torch.zeros((1, 4), dtype=torch.int32, device="cuda"), lens, lens + 5,
                     torch.arange(4, dtype=torch.int32, device="cuda"), 5)
    q, k = torch.ones((5, 4, 64), device="cuda"), torch.ones((5, 2, 64), device="cuda")
    with pytest.raises(ValueError):
        cache.prompt(0, q, k, k, sl.positions, lib.Rotary(64), sl)
    assert not cache.k_cache(0).any()


def test_every_refusal_of_a_prompt_comes_before_its_append(lib):
    """What the rotary call would take and the attention refuses: neither cache is written."""
    import torch
    from paged_kv_cache_295_gb300.engine import PagedKVCache
    T, i32 = 5, dict(dtype=torch.int32, device="cuda")
    cache = PagedKVCache(num_layers=1, num_kv_heads=2, head_dim=64, block_size=16, num_blocks=4, kv_dtype=lib.BF16)
    cache.storage.zero_()
    sl = cache.slots(torch.zeros((1, 4), **i32), torch.zeros(1, **i32), torch.full((1,), T, **i32),
                     torch.arange(4, **i32), T)
    rows = dict(dtype=torch.bfloat16, device="cuda")
    q, k, v = (torch.ones((T, h, 64), **rows) for h in (4, 2, 2))
    off = torch.ones(T * 2 * 64 + 1, **rows)[1:].view(T, 2, 64)          # on no 16-byte boundary
    odd = torch.ones((T, 2, 68), **rows)[..., :64]                       # strides of 68
    over = torch.ones((T, 4, 64), **rows)
    plan, done = lib.Rotary(64), dict(out_dtype=torch.bfloat16)

    def call(q=q, v=v, sl=sl, **kw):
        return cache.prompt(0, q, k, v, sl.positions, plan, sl, **kw)

    for kw in (dict(window=-1), dict(sinks=4), dict(window=8, sinks=-1), dict(window="x"), dict(window=2 ** 31),
               dict(out=over[:4]), dict(out=over.double()), dict(out=over.half()), dict(out=over.cpu()),
               dict(out=over.transpose(0, 1)), dict(out=over, out_dtype=torch.float32), dict(out_dtype=torch.float16),
               dict(v=over[:, 2:], out=over), dict(v=off), dict(v=odd), dict(sl=sl._replace(query_start=None)),
               dict(sl=sl._replace(query_start=sl.query_start.long())), dict(q=torch.ones((T, 3, 64), **rows)),
               dict(q=torch.ones((T, 2 * 129, 64), **rows)), dict(q=q[:4]), dict(v=v[:, :1]),
               dict(device_status=torch.zeros(1, device="cuda"))):
        for stream in (None, torch.cuda.Stream()):
            with pytest.raises((ValueError, lib.PagedKVError)):
                call(stream=stream, **kw)
            torch.cuda.synchronize()
            assert not cache.storage.any(), kw
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = call(stream=side, **done)
    side.synchronize()
    assert torch.equal(out, torch.ones_like(out))     # every v is 1
    assert torch.equal(cache.v_cache(0).flatten(0, 1)[:T], v) and cache.k_cache(0).flatten(0, 1)[:T].any()
    assert call(out=over, **done) is over or torch.equal(over, out)


@pytest.mark.parametrize("out_type", ["bfloat16", "float32"])
def test_a_prompt_behind_a_cached_prefix_is_flagged(lib, out_type):
    """A second chunk in prompt: its sequence has no attention rows and the status says so; a new sequence beside it
    and one without tokens are as they should be."""
    import torch
    m = Model(lib, lib.BF16, 7)
    cache, dt = m.cache, getattr(torch, out_type)
    free, start, lens = dev(cache.pool.free_list()), dev([0]), dev([0, 0, 0, 0])
    tables = torch.full((4, 20), -1, dtype=torch.int32, device="cuda")
    for new, flagged in (([40, 0, 0, 9], []), ([0, 130, 0, 0], []), ([0, 5, 33, 1], [1, 3]), ([0, 0, 0, 0], [])):
        T = sum(new)
        x = m.step(T)
        q, k, v = x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]
        sl = cache.slots(tables, lens, dev(new), free, T, free_start=start, context_out=lens, free_next=start)
        status, out = dev([0]), torch.full((T, HQ, D), 5.0, dtype=dt, device="cuda")
        cache.prompt(0, q, k, v, m.grid(sl.positions), m.rotary, sl, out=out, device_status=status)
        assert int(status.item()) == (lib.DEV_BAD_CONTEXT if flagged else 0)
        qr, kr = lib.rotary_and_cache(q, k, None, m.grid(sl.positions), m.rotary)
        want = lib.packed_attention_prefill(qr, kr, v, sl.query_start, cache.scale, out_dtype=dt)
        at = [0, *np.cumsum(new)]
        for s in range(4):
            rows = slice(at[s], at[s + 1])
            assert torch.equal(out[rows], torch.full_like(out[rows], 5.0) if s in flagged else want[rows])
    q, k, v = (torch.zeros((4, h, D), dtype=torch.bfloat16, device="cuda") for h in (HQ, HKV, HKV))
    for bad in (dev([4]).long(), dev([4, 4]), torch.tensor([4], dtype=torch.int32)):
        with pytest.raises(ValueError):
            lib.packed_attention_prefill(q, k, v, dev([0, 4]), 0.1, context_lens=bad)


def test_a_captured_prompt(lib):
    """Slots, rotary positions, append and attention of a step in one graph, replayed on other rows and lengths; the
    replay writes what the same calls one by one do."""
    import torch
    m = Model(lib, lib.BF16, 9)
    cache, T = m.cache, 300
    x, new = m.step(T), dev([100, 3, 150])
    free = dev(cache.pool.free_list())
    tables, lens, start = torch.full((3, 20), -1, dtype=torch.int32, device="cuda"), dev([0, 0, 0]), dev([0])
    out, status = torch.zeros((T, HQ, D), dtype=torch.bfloat16, device="cuda"), dev([0])

    def step(stream=None):
        sl = cache.slots(tables, lens, new, free, T, free_start=start, device_status=status)
        cache.prompt(0, x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:], m.grid(sl.positions), m.rotary, sl, window=90,
                     sinks=2, out=out, device_status=status, stream=stream)

    step()
    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        step()
    for lengths in ([100, 3, 150], [0, 299, 1], [1, 1, 1], [0, 0, 0], [60, 60, 60]):
        x.copy_(m.step(T))
        new.copy_(dev(lengths))
        got = []
        for run in (g.replay, step):
            out.fill_(9.0)
            cache.storage.zero_()
            tables.fill_(-1)
            run()
            torch.cuda.synchronize()
            got.append((out.clone(), cache.storage.clone(), tables.clone()))
        assert int(status.item()) == 0 and all(torch.equal(a, b) for a, b in zip(*got))
        assert (got[0][0][sum(lengths):] == 9.0).all() and not (got[0][0][:sum(lengths)] == 9.0).all(-1).any()
