"""Slots from request lengths on the GPU, against the token-by-token oracle and the host pool."""
import numpy as np
import pytest

from oracle import step as OS

pytestmark = pytest.mark.gpu

FLAGS = {"block": "DEV_BAD_BLOCK", "context": "DEV_BAD_CONTEXT", "free": "DEV_NO_FREE_BLOCK"}


def dev(x):
    import torch
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def check(lib, tables, ctx, new, free, start, bs, T, nb, per_row=False, held=False):
    """One call against the oracle: every output, the flags, and the tables in place."""
    import torch
    want = OS.slots(tables, ctx, new, free, start, bs, T, nb, per_row, held)
    t, status = dev(tables), torch.zeros(1, dtype=torch.int32, device="cuda")
    got = lib.slots_from_lengths(t, dev(ctx), None if new is None else dev(new), dev(free), nb, bs, T,
                                 free_start=dev([start]), row_per_sequence=per_row, first_block_held=held,
                                 device_status=status)
    assert int(status.item()) == sum(getattr(lib, FLAGS[f]) for f in want[6])
    assert np.array_equal(t.cpu().numpy(), want[0])
    assert np.array_equal(got.slot_mapping.cpu().numpy(), want[1])
    assert np.array_equal(got.positions.cpu().numpy(), want[2])
    if per_row:
        assert got.query_start is None
    else:
        assert np.array_equal(got.query_start.cpu().numpy(), want[3])
    assert np.array_equal(got.context_lens.cpu().numpy(), want[4])
    assert got.free_start.tolist() == [want[5]]
    return want


def batch(rng, seqs, bs, ctx, new, held=False):
    """Tables of sequences of 0..ctx tokens, new lengths 0..new, the free blocks behind them."""
    c, n = rng.integers(0, ctx + 1, seqs), rng.integers(0, new + 1, seqs)
    mb = max(1, -(-(ctx + new) // bs))
    need = np.maximum(-(-c // bs), 1 if held else 0)
    perm = rng.permutation(int(need.sum()) + int((-(-(c + n) // bs)).sum()) + 5).astype(np.int32)
    tables, at = np.full((seqs, mb), -1, dtype=np.int32), 0
    for s in range(seqs):
        tables[s, :need[s]] = perm[at:at + need[s]]
        at += need[s]
    return tables, c, n, perm[at:], perm.size


@pytest.mark.parametrize("seqs,bs,ctx,new", [
    (1, 16, 0, 0), (1, 1, 5, 3), (7, 16, 40, 50), (33, 24, 100, 1), (64, 8, 300, 2000), (5, 4096, 9000, 9000),
    (1023, 16, 60, 9), (1024, 16, 60, 9), (1025, 3, 20, 7), (2500, 16, 90, 30)])
@pytest.mark.parametrize("held", [False, True])
def test_batches(lib, seqs, bs, ctx, new, held):
    """One tile of sequences and several, one CTA and several, sequences without new tokens, more
    rows than tokens."""
    rng = np.random.default_rng(seqs + bs)
    tables, c, n, free, nb = batch(rng, seqs, bs, ctx, new, held)
    for pad, start in ((0, 0), (13, 3)):
        check(lib, tables, c, n, free, start, bs, int(n.sum()) + pad, nb, held=held)


@pytest.mark.parametrize("seqs", [1, 9, 1100])
def test_decode_rows(lib, seqs):
    """A row per sequence: one token each, or none for some of them."""
    rng = np.random.default_rng(seqs)
    tables, c, n, free, nb = batch(rng, seqs, 16, 70, 1)
    check(lib, tables, c, None, np.concatenate([free, np.arange(seqs)]), 0, 16, seqs, nb + seqs, per_row=True)
    check(lib, tables, c, n, free, 1, 16, seqs + 3, nb, per_row=True)
    check(lib, tables, c, None, np.concatenate([free, np.arange(seqs)]), 0, 16, seqs, nb + seqs)


def test_all_or_nothing(lib):
    rng = np.random.default_rng(1)
    tables, c, n, free, nb = batch(rng, 40, 16, 90, 60)
    need = int(np.maximum(-(-(c + n) // 16) - -(-c // 16), 0).sum())
    T = int(n.sum())
    for f, start in ((free[:need], 0), (free, len(free) - need)):
        assert not check(lib, tables, c, n, f, start, 16, T, nb)[6]
    for f, start, rows, flag in ((free[:need - 1], 0, T, "free"), (free, len(free) - need + 1, T, "free"),
                                 (free, -1, T, "free"), (free, 10 ** 6, T, "free"), (free[:0], 0, T, "free"),
                                 (free, 0, T - 1, "context"), (free, 0, 0, "context")):
        assert check(lib, tables, c, n, f, start, 16, rows, nb)[6] == {flag}
    # nothing is needed from an empty or used-up list
    assert not check(lib, tables, c, 0 * n, free[:0], 0, 16, 4, nb)[6]
    check(lib, tables, c, 0 * n, free, 10 ** 6, 16, 0, nb)


def test_bad_lengths_and_blocks(lib):
    rng = np.random.default_rng(2)
    tables, c, n, free, nb = batch(rng, 30, 16, 90, 60)
    T = int(n.sum()) + 200
    for at, cc, nn in ((3, -1, 5), (4, 10 ** 9, 1), (5, 2 ** 31 - 1, 2 ** 31 - 1), (6, 5, -3), (29, 16 * tables.shape[1], 1)):
        c2, n2 = c.copy(), n.copy()
        c2[at], n2[at] = cc, nn
        assert "context" in check(lib, tables, c2, n2, free, 0, 16, T, nb)[6]
        if nn > 1:
            assert "context" in check(lib, tables, c2, np.minimum(n2, 2), free, 0, 16, 90, nb, per_row=True)[6]
    c2 = c.copy()
    c2[7], n[7] = 20, 60
    t2 = tables.copy()
    t2[7, :2] = [0, 10 ** 6]              # the open block: tokens up to its end have no slot
    assert check(lib, t2, c2, n, free, 0, 16, T, nb)[6] == {"block"}
    f2 = free.copy()
    f2[2] = -7
    assert check(lib, tables, c, n, f2, 0, 16, T, nb)[6] == {"block"}


def test_no_sequences(lib):
    check(lib, np.zeros((0, 4), dtype=np.int32), [], [], np.arange(3), 1, 16, 5, 8)


def test_the_pool_takes_the_same_blocks(lib):
    """The device's appends, then the same ones on the host pool: blocks, slots and free list."""
    rng = np.random.default_rng(3)
    pool = lib.Pool(1, 1, 64, 16, lib.BF16, num_blocks=400, initial_free_order=rng.permutation(400).astype(np.int32))
    lens = [0, 5, 16, 31, 200]
    for s, n in enumerate(lens):
        pool.seq_create(s)
        if n:
            pool.append_tokens(s, n)
    tables, ctx = pool.batch_tables(range(5), 40)
    t, c, free = dev(tables), dev(ctx), dev(pool.free_list())
    start = dev([0])
    for new in ([100, 1, 0, 17, 3], None, [0, 0, 0, 0, 0], [1, 16, 32, 0, 250], None):
        import torch
        n = None if new is None else dev(new)
        got = lib.slots_from_lengths(t, c, n, free, 400, 16, 400, free_start=start, first_block_held=True,
                                     context_out=c, free_next=start)
        slots = got.slot_mapping.cpu().numpy()
        want = [pool.append_tokens(s, 1 if new is None else new[s]) for s in range(5)]
        want = np.concatenate(want)
        assert np.array_equal(slots[:want.size], want) and (slots[want.size:] == -1).all()
        tables, ctx = pool.batch_tables(range(5), 40)
        assert np.array_equal(t.cpu().numpy(), tables) and np.array_equal(c.cpu().numpy(), ctx)
        assert free[int(start.item()):].tolist() == pool.free_list()
        torch.cuda.synchronize()


def test_a_captured_step_goes_on_by_itself(lib):
    """Lengths and the free list's start in place: every replay is one more step."""
    import torch
    rng = np.random.default_rng(4)
    tables, c, _, free, nb = batch(rng, 1500, 16, 40, 30)
    free = np.concatenate([free, nb + np.arange(3000)]).astype(np.int32)
    nb += 3000
    mb = tables.shape[1]
    t, cd, fd, start = dev(tables), dev(c), dev(free), dev([2])
    out = {"slot_mapping": torch.empty(1500, dtype=torch.int64, device="cuda"),
           "positions": torch.empty(1500, dtype=torch.int32, device="cuda")}

    def step():
        lib.slots_from_lengths(t, cd, None, fd, nb, 16, free_start=start, row_per_sequence=True, context_out=cd,
                               free_next=start, **out)

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):        # loads the kernel; then everything as it was
        step()
    torch.cuda.synchronize()
    t.copy_(dev(tables))
    cd.copy_(dev(c))
    start.fill_(2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step()
    at = 2
    for _ in range(20):
        g.replay()
        torch.cuda.synchronize()
        tables, slot, pos, _, c, at, flags = OS.slots(tables, c, None, free, at, 16, 1500, nb, True)
        assert not flags and c.max() <= mb * 16
        assert np.array_equal(out["slot_mapping"].cpu().numpy(), slot)
        assert np.array_equal(out["positions"].cpu().numpy(), pos)
        assert np.array_equal(t.cpu().numpy(), tables) and start.tolist() == [at]


def test_streams_and_arguments(lib):
    import torch
    rng = np.random.default_rng(6)
    tables, c, n, free, nb = batch(rng, 9, 16, 90, 60)
    T = int(n.sum())
    want = OS.slots(tables, c, n, free, 0, 16, T, nb)
    t, s = dev(tables), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = lib.slots_from_lengths(t, dev(c), dev(n), dev(free), nb, 16, T, stream=s)
    s.synchronize()
    assert np.array_equal(got.slot_mapping.cpu().numpy(), want[1])
    args = (dev(tables), dev(c), dev(n), dev(free), nb, 16, T)
    for kw in (dict(slot_mapping=torch.empty(T, dtype=torch.int32, device="cuda")),
               dict(positions=torch.empty(T + 1, dtype=torch.int32, device="cuda")),
               dict(query_start=torch.empty(9, dtype=torch.int32, device="cuda")),
               dict(context_out=torch.empty((9, 2), dtype=torch.int32, device="cuda")[:, 0]),
               dict(free_next=torch.empty(1, dtype=torch.int32)), dict(row_per_sequence="x", query_start=dev([0] * 10))):
        with pytest.raises(ValueError):
            lib.slots_from_lengths(*args, **kw)


def call_in_place(lib, tables, c, n, free, start, bs, T, nb, which, per_row=False):
    """One call whose lengths, list start or both take the old ones' place, against the oracle."""
    import torch
    want = OS.slots(tables, c, n, free, start, bs, T, nb, per_row)
    t, cd, fs, status = dev(tables), dev(c), dev([start]), torch.zeros(1, dtype=torch.int32, device="cuda")
    kw = {}
    if "lengths" in which:
        kw["context_out"] = cd
    if "start" in which:
        kw["free_next"] = fs
    got = lib.slots_from_lengths(t, cd, None if n is None else dev(n), dev(free), nb, bs, T, free_start=fs,
                                 row_per_sequence=per_row, device_status=status, **kw)
    assert int(status.item()) == sum(getattr(lib, FLAGS[f]) for f in want[6])
    assert np.array_equal(t.cpu().numpy(), want[0])
    assert np.array_equal(got.slot_mapping.cpu().numpy(), want[1])
    assert np.array_equal(got.positions.cpu().numpy(), want[2])
    if not per_row:
        assert np.array_equal(got.query_start.cpu().numpy(), want[3])
    assert np.array_equal(got.context_lens.cpu().numpy(), want[4])
    assert got.free_start.tolist() == [want[5]]
    assert cd.tolist() == (want[4] if "lengths" in which else np.asarray(c)).tolist()
    assert fs.tolist() == [want[5] if "start" in which else start]
    return want


@pytest.mark.parametrize("which", [("lengths",), ("start",), ("lengths", "start")])
@pytest.mark.parametrize("seqs,bs,ctx,new", [
    (7, 16, 900, 1000), (40, 24, 300, 350), (64, 16, 2000, 2047), (1500, 16, 60, 4), (2500, 16, 90, 6),
    (3100, 3, 40, 45)])
def test_in_place_over_several_ctas(lib, which, seqs, bs, ctx, new):
    """Prompts and chunks of 3,000 to 70,000 rows, which two, four or eight CTAs fill while the lengths and
    the list's start that all of them read are written; up to four tiles of sequences; rows without a token."""
    rng = np.random.default_rng(seqs)
    tables, c, n, free, nb = batch(rng, seqs, bs, ctx, new)
    T = int(n.sum())
    assert T > 2048
    for pad, start in ((0, 0), (5000, 3)):
        want = call_in_place(lib, tables, c, n, free, start, bs, T + pad, nb, which)
        assert not want[6] and (want[4] != c).any()


@pytest.mark.parametrize("seqs", [2500, 9000, 20000])
def test_decode_rows_in_place_over_several_ctas(lib, seqs):
    rng = np.random.default_rng(seqs)
    tables, c, n, free, nb = batch(rng, seqs, 16, 30, 1)
    for T in (seqs, seqs + 99):
        call_in_place(lib, tables, c, n, free, 0, 16, T, nb, ("lengths", "start"), per_row=True)
    free = np.concatenate([free, nb + np.arange(seqs)])
    call_in_place(lib, tables, c, None, free, 0, 16, seqs, nb + seqs, ("lengths", "start"), per_row=True)


@pytest.mark.parametrize("seqs,new", [(60, 200), (1700, 8)])
def test_all_or_nothing_in_place_over_several_ctas(lib, seqs, new):
    """Too few blocks or rows: no CTA writes a table, the lengths and the list's start stay; bad sequences among good
    ones; nothing to do."""
    rng = np.random.default_rng(seqs)
    tables, c, n, free, nb = batch(rng, seqs, 16, 90, new)
    need, T = int(np.maximum(-(-(c + n) // 16) - -(-c // 16), 0).sum()), int(n.sum())
    assert T > 4096
    both = ("lengths", "start")
    for f, start, rows, flag in ((free[:need - 1], 0, T, "free"), (free, len(free) - need + 1, T, "free"),
                                 (free, -1, T, "free"), (free, 0, T - 1, "context")):
        want = call_in_place(lib, tables, c, n, f, start, 16, rows, nb, both)
        assert want[6] == {flag} and np.array_equal(want[4], c)
    assert not call_in_place(lib, tables, c, n, free[:need], 0, 16, T, nb, both)[6]
    assert not call_in_place(lib, tables, c, 0 * n, free[:0], 0, 16, 5000, nb, both)[6]
    c2, n2 = c.copy(), n.copy()
    c2[[3, seqs - 1]], n2[5] = (-1, 10 ** 9), -4
    assert "context" in call_in_place(lib, tables, c2, n2, free, 0, 16, T, nb, both)[6]


def test_captured_prompts_in_place(lib):
    """A captured step of 9,000 rows, replayed with new lengths: every replay goes on from the last one."""
    import torch
    rng = np.random.default_rng(8)
    seqs, T, bs = 90, 9000, 16
    tables = np.full((seqs, 160), -1, dtype=np.int32)
    free = rng.permutation(6000).astype(np.int32)
    c, at = np.zeros(seqs, dtype=np.int32), 0
    t, cd, fd, start, nd = dev(tables), dev(c), dev(free), dev([0]), dev(c)
    kw = {"slot_mapping": torch.empty(T, dtype=torch.int64, device="cuda"),
          "positions": torch.empty(T, dtype=torch.int32, device="cuda"),
          "query_start": torch.empty(seqs + 1, dtype=torch.int32, device="cuda")}

    def step():
        lib.slots_from_lengths(t, cd, nd, fd, 6000, bs, T, free_start=start, context_out=cd, free_next=start, **kw)

    side, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        step()                             # no new tokens: loads the kernel
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        step()
    for _ in range(12):
        n = rng.integers(0, 100, seqs).astype(np.int32)
        nd.copy_(dev(n))
        g.replay()
        torch.cuda.synchronize()
        tables, slot, pos, qs, c, at, flags = OS.slots(tables, c, n, free, at, bs, T, 6000)
        assert not flags
        for name, x in (("slot_mapping", slot), ("positions", pos), ("query_start", qs)):
            assert np.array_equal(kw[name].cpu().numpy(), x)
        assert np.array_equal(t.cpu().numpy(), tables) and np.array_equal(cd.cpu().numpy(), c)
        assert start.tolist() == [at]
