"""The 8-bit cache with a scale per block and head on the GPU: appended, read back and
attended, against the numpy definitions.  Codes and scales are compared bit for bit."""
import numpy as np
import pytest

from oracle import block_scaled as OB
from tests import gpu_cases as GC
from tests import paged_cases as PC

pytestmark = pytest.mark.gpu


def rows(seed, t, hkv, d, src, spread=1.0):
    """Token rows whose sizes differ from token to token (scales then grow)."""
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((t, hkv, d)) * np.exp(spread * rng.standard_normal((t, 1, 1)))
    return x.astype(np.float32) if src == "f32" else PC.bf16_bits(x)


def append(lib, case, k_new, v_new, new, src, status=None, dev=None, **kw):
    """The call on the device caches of ``case``; returns them as numpy."""
    import torch
    d = case.device() if dev is None else dev
    qs = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    lib.quantize_and_cache(GC.to_torch(k_new, src), GC.to_torch(v_new, src), d["k"], d["v"],
                           d["ks"], d["vs"], d["tables"], d["lens"], query_start=qs,
                           max_query_len=max(max(new), 0), device_status=status, **kw)
    torch.cuda.synchronize()
    return [GC.from_torch(d[n], case.kv if n in "kv" else "f32") for n in ("k", "v", "ks", "vs")]


def check_append(lib, case, k_new, v_new, new, src):
    qs = np.concatenate([[0], np.cumsum(new)])
    want = [x.copy() for x in (case.k, case.v, case.ks, case.vs)]
    OB.quantize_and_cache(k_new, v_new, qs, case.tables, case.lens, *want, src, case.kv)
    got = append(lib, case, k_new, v_new, new, src)
    for name, a, b in zip(("k", "v", "k_scale", "v_scale"), got, want):
        assert a.tobytes() == b.tobytes(), name
    return got


@pytest.mark.parametrize("kv", ["fp8_e4m3", "int8"])
@pytest.mark.parametrize("src", ["bf16", "f32"])
@pytest.mark.parametrize("bs,d,hkv", [(16, 128, 8), (1, 64, 3), (8, 80, 1), (32, 256, 5),
                                      (64, 128, 2), (256, 128, 3), (4096, 16, 1), (128, 144, 2)])
def test_append(lib, kv, src, bs, d, hkv):
    """Chunks that begin blocks, continue them (with growth and without), cross several,
    an empty one and single tokens."""
    lens = [1, 2 * bs, bs + 1, 3 * bs + bs // 2 + 1, 7, 5 * bs]
    new = [1, 2 * bs, 1, 2 * bs + 1, 0, bs // 2 + 1]
    new = [min(n, c) for n, c in zip(new, lens)]
    case = PC.make(bs + d, kv, lens, hkv, d, bs, stride=hkv + 2, spread=0.2)
    # half of the older scales are small, so that the new rows make them grow
    case.ks[::2] *= 0.01
    case.vs[1::2] *= 0.003
    check_append(lib, case, rows(1, sum(new), hkv, d, src), rows(2, sum(new), hkv, d, src), new, src)


@pytest.mark.parametrize("kv", ["fp8_e4m3", "int8"])
def test_append_step_by_step_stays_within_one_step(lib, kv):
    """A block filled token by token, its scale growing often: codes are the definition's,
    and every value is within one step of its final scale (E4M3: 2^-3 of the value, or half
    of the smallest step 2^-9 twice)."""
    import torch
    bs, d, hkv, n = 16, 128, 4, 35
    case = PC.make(3, kv, [n, n], hkv, d, bs, spread=0.0)
    case.k[:], case.v[:] = GC.POISON[kv][1], GC.POISON[kv][1]
    case.ks[:], case.vs[:] = np.nan, 0.0
    want = [x.copy() for x in (case.k, case.v, case.ks, case.vs)]
    dev = case.device()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ramp = 1.35 ** np.arange(n)     # ascending sizes: growth on most steps
    kk = PC.bf16_bits(np.random.default_rng(5).standard_normal((n, 2, hkv, d)) * ramp[:, None, None, None])
    vv = rows(6, 2 * n, hkv, d, "bf16").reshape(n, 2, hkv, d)
    for i in range(n):
        lens = torch.full((2,), i + 1, dtype=torch.int32, device="cuda")
        lib.quantize_and_cache(GC.to_torch(kk[i], "bf16"), GC.to_torch(vv[i], "bf16"), dev["k"],
                               dev["v"], dev["ks"], dev["vs"], dev["tables"], lens,
                               device_status=status)
        OB.quantize_and_cache(kk[i], vv[i], [0, 1, 2], case.tables, [i + 1, i + 1], *want, "bf16", kv)
    got = [GC.from_torch(dev[m], kv if m in "kv" else "f32") for m in ("k", "v", "ks", "vs")]
    for a, b in zip(got, want):
        assert a.tobytes() == b.tobytes()
    assert int(status.item()) == 0
    for s in range(2):
        for new, c, sc in ((kk, got[0], got[2]), (vv, got[1], got[3])):
            x = np.stack([GC.OA.to_f64(new[i, s], "bf16") for i in range(n)])
            y = OB.gather(c, sc, case.tables[s], 0, n, kv).astype(np.float64)
            step = sc[case.tables[s][np.arange(n) // bs]][:, :, None].astype(np.float64)
            # the last term: the float32 rounding of the quotient and of code * scale
            lim = step * 1.0 if kv == "int8" else np.abs(x) * 2.0 ** -4 + step * 2.0 ** -9
            assert (np.abs(x - y) <= lim * 1.001 + np.abs(x) * 2.0 ** -22).all()


@pytest.mark.parametrize("kv", ["fp8_e4m3", "int8"])
@pytest.mark.parametrize("src", ["bf16", "f32"])
def test_append_special_values(lib, kv, src):
    """Zeros, NaN, infinities, the largest and smallest finite values, exact ties."""
    bs, d, hkv = 16, 64, 6
    lens, new = [16, 20, 9], [16, 4, 9]
    case = PC.make(9, kv, lens, hkv, d, bs, spread=0.1)
    x = rows(10, sum(new), hkv, d, "f32")
    x[:, 0] = 0.0
    x[::2, 0, ::3] = -0.0
    x[3, 1, 5], x[4, 1, 6], x[5, 1, 7] = np.nan, np.inf, -np.inf
    x[17, 1] = np.nan                       # a continued block, one row with no finite value
    x[0, 2, 0], x[18, 2, 1] = 3.3e38, -3.3e38
    x[:, 3] = 1e-38
    x[20:, 4] = 2.0 ** -60
    x[:, 5] = np.arange(d) / 64.0           # x / scale falls on ties
    x[:, 5, 0] = 7.0
    y = x[::-1].copy()
    if src == "bf16":
        x, y = PC.bf16_bits(x), PC.bf16_bits(y)
    check_append(lib, case, x, y, new, src)


def test_quotient_is_ieee(lib):
    """The codes of many quotients next to ties equal those of IEEE division (oracle)."""
    bs, d, hkv = 64, 256, 8
    rng = np.random.default_rng(12)
    for kv in ("fp8_e4m3", "int8"):
        n = 4 * bs
        case = PC.make(13, kv, [n], hkv, d, bs)
        a = rng.uniform(0.5, 2.0, (1, hkv, 1)).astype(np.float32)
        grid = (rng.integers(-127, 128, (n, hkv, d)) + 0.5 if kv == "int8" else
                rng.integers(-15, 16, (n, hkv, d)) * 2.0 ** rng.integers(-10, 6, (n, hkv, d)))
        x = (grid * a / OB.QMAX[kv]).astype(np.float32)
        x = np.clip(x, -a, a)
        x[:, :, 0] = a[0, :, 0]
        x = np.nextafter(x, np.where(rng.random(x.shape) < 0.5, np.float32(9), np.float32(-9))) \
            if kv == "int8" else x
        check_append(lib, case, x.astype(np.float32), x[::-1].astype(np.float32).copy(), [n], "f32")


def test_append_one_row_per_sequence_and_padding(lib):
    """Without query_start: row s; a sequence of context 0 is a padded one."""
    import torch
    kv, bs, d, hkv = "fp8_e4m3", 16, 128, 4
    lens = [17, 0, 33, 16]
    case = PC.make(20, kv, lens, hkv, d, bs)
    x, y = rows(21, 4, hkv, d, "bf16"), rows(22, 4, hkv, d, "bf16")
    keep = [0, 2, 3]
    want = [a.copy() for a in (case.k, case.v, case.ks, case.vs)]
    OB.quantize_and_cache(x[keep], y[keep], [0, 1, 2, 3], case.tables[keep], [lens[i] for i in keep],
                          *want, "bf16", kv)
    d_ = case.device()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.quantize_and_cache(GC.to_torch(x, "bf16"), GC.to_torch(y, "bf16"), d_["k"], d_["v"], d_["ks"],
                           d_["vs"], d_["tables"], d_["lens"], device_status=status)
    for n, b in zip(("k", "v", "ks", "vs"), want):
        assert GC.from_torch(d_[n], kv if n in "kv" else "f32").tobytes() == b.tobytes()
    assert int(status.item()) == 0


def test_append_flags_bad_input_and_touches_nothing_else(lib):
    """Bad blocks, contexts and query_start values are skipped and flagged."""
    import torch
    kv, bs, d, hkv = "int8", 16, 64, 2
    lens = [40, 20, 30, 10]
    case = PC.make(30, kv, lens, hkv, d, bs)
    good = case.tables.copy()
    case.tables[0, 1] = 10 ** 6           # middle block of sequence 0
    new = [40, 5, 8, 10]
    x, y = rows(31, sum(new), hkv, d, "bf16"), rows(32, sum(new), hkv, d, "bf16")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = append(lib, case, x, y, new, "bf16", status=status)
    assert int(status.item()) == lib.DEV_BAD_BLOCK
    want = [a.copy() for a in (case.k, case.v, case.ks, case.vs)]
    OB.quantize_and_cache(x, y, np.concatenate([[0], np.cumsum(new)]), good, lens, *want, "bf16", kv)
    b = good[0, 1]
    for a, w, o in zip(got, want, (case.k, case.v, case.ks, case.vs)):
        w[b] = o[b]                       # the block in question keeps what it held
        assert a.tobytes() == w.tobytes()
    # contexts beyond the table and shorter than the chunk: the sequences are left alone
    case.tables[:] = good
    case.lens = [40, 10 ** 6, 30, 3]
    status.zero_()
    got = append(lib, case, x, y, new, "bf16", status=status)
    assert int(status.item()) == lib.DEV_BAD_CONTEXT
    want = [a.copy() for a in (case.k, case.v, case.ks, case.vs)]
    sel = np.r_[0:40, 45:53]
    OB.quantize_and_cache(x[sel], y[sel], [0, 40, 48], good[[0, 2]], [40, 30], *want, "bf16", kv)
    for a, w in zip(got, want):
        assert a.tobytes() == w.tobytes()


@pytest.mark.parametrize("kv,scales", [("fp8_e4m3", "block"), ("int8", "block"), ("fp8_e4m3", "head"),
                                       ("int8", "head"), ("bf16", None), ("f32", None)])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("bs,d,hkv", [(16, 128, 8), (1, 64, 3), (256, 80, 5)])
def test_read_back(lib, kv, scales, out, bs, d, hkv):
    """Rows from any position on, empty sequences; rows between sequences keep their bytes."""
    import torch
    lens = [5, 3 * bs + 7, bs, 1, 2 * bs + 40]
    first = [0, bs + 2, 0, 0, 31]
    n = [5, 2 * bs + 5, 0, 1, 2 * bs + 9]
    case = PC.make(40 + bs, kv, lens, hkv, d, bs, scales=scales, stride=hkv + 1)
    d_ = case.device()
    start = np.concatenate([[0], np.cumsum(n)])
    total = int(start[-1]) + 3            # three rows behind the last sequence
    dt = torch.bfloat16 if out == "bf16" else torch.float32
    ko = torch.full((total, hkv, d), 7.0, dtype=dt, device="cuda")
    vo = torch.full_like(ko, 7.0)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    lib.gather_cache(d_["k"], d_["v"], d_["tables"], torch.from_numpy(start).int().cuda(), total,
                     max(n), first_pos=torch.tensor(first, dtype=torch.int32, device="cuda"),
                     k_scale=d_.get("ks"), v_scale=d_.get("vs"), k_out=ko, v_out=vo,
                     device_status=status)
    assert int(status.item()) == 0
    for got, c, sc in ((ko, case.k, case.ks), (vo, case.v, case.vs)):
        want = torch.full((total, hkv, d), 7.0)
        for s in range(len(lens)):
            want[start[s]:start[s + 1]] = torch.from_numpy(
                OB.gather(c, sc, case.tables[s], first[s], n[s], kv))
        assert torch.equal(got.cpu(), want.to(dt))


def test_read_back_flags(lib):
    import torch
    kv, bs, d, hkv = "fp8_e4m3", 16, 64, 2
    case = PC.make(50, kv, [40, 20, 30], hkv, d, bs)
    case.tables[0, 1] = -1
    d_ = case.device()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    start = torch.tensor([0, 40, 60, 90], dtype=torch.int32, device="cuda")
    k, v = lib.gather_cache(d_["k"], d_["v"], d_["tables"], start, 90, 40, k_scale=d_["ks"],
                            v_scale=d_["vs"], out_dtype=torch.float32, device_status=status)
    assert int(status.item()) == lib.DEV_BAD_BLOCK
    assert (k[16:32] == 0).all() and (v[16:32] == 0).all()
    assert torch.equal(k[60:90].cpu(), torch.from_numpy(OB.gather(case.k, case.ks, case.tables[2], 0, 30, kv)))
    # a start beyond the output, positions beyond the table: skipped
    status.zero_()
    ko = torch.full((90, hkv, d), 3.0, device="cuda")
    lib.gather_cache(d_["k"], d_["v"], d_["tables"],
                     torch.tensor([0, 10, 200, 90], dtype=torch.int32, device="cuda"), 90, 40,
                     first_pos=torch.tensor([10 ** 6, 0, 0], dtype=torch.int32, device="cuda"),
                     k_scale=d_["ks"], v_scale=d_["vs"], k_out=ko, v_out=torch.empty_like(ko),
                     device_status=status)
    assert int(status.item()) == lib.DEV_BAD_CONTEXT
    assert (ko == 3.0).all()


# ---- attention over the cache ---------------------------------------------------
def decode(lib, case, q, q_type, scale, out, status=None, partition=0, window=0, sinks=0, **kw):
    import torch
    d = case.device()
    mx = max(case.lens + [1])
    r = lib.paged_attention_decode(
        GC.to_torch(q, q_type), d["k"], d["v"], d["tables"], d["lens"], scale, mx,
        k_scale=d.get("ks"), v_scale=d.get("vs"), partition=partition, window=window, sinks=sinks,
        out_dtype=torch.bfloat16 if out == "bf16" else torch.float32, device_status=status, **kw)
    return r.float().cpu().numpy().astype(np.float64)


def check_decode(lib, case, hq, seed, q_type="bf16", out="bf16", partition=0, window=0, sinks=0,
                 scale=None, qmul=1.0):
    import torch
    S, (hkv, d) = len(case.lens), case.k.shape[2:]
    scale = d ** -0.5 if scale is None else scale
    x = np.random.default_rng(seed).standard_normal((S, hq, d)) * qmul
    q = x.astype(np.float32) if q_type == "f32" else PC.bf16_bits(x)
    q64 = GC.OA.to_f64(q, q_type)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = decode(lib, case, q, q_type, scale, out, status, partition, window, sinks)
    assert int(status.item()) == 0
    worst = 0.0
    for s, n in enumerate(case.lens):
        if n == 0:
            assert (got[s] == 0).all()
            continue
        K, V = case.values(s)
        o, mag, reach = OB.attend(q64[s:s + 1], [n - 1], K, V, scale, window, sinks)
        hi_lo = case.kv == "bf16" or out == "f32"
        lim = PC.attention_bound(case, q64[s:s + 1], o, mag, reach, scale, q_type == "f32",
                                 out == "bf16", hi_lo, min(n, window + sinks) if window else n)
        worst = max(worst, float((np.abs(got[s] - o[0]) / lim[0]).max()))
    assert worst <= 1.0, worst
    return worst


@pytest.mark.parametrize("kv", ["fp8_e4m3", "int8"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("bs,hq,hkv", [(16, 8, 8), (8, 8, 2), (32, 6, 2), (64, 5, 1), (256, 16, 2),
                                       (16, 9, 1), (16, 15, 1), (128, 32, 2)])
def test_decode(lib, kv, out, bs, hq, hkv):
    case = PC.make(60 + bs + hq, kv, [1, 17, 64, 300, 0, 129], hkv, 128, bs, stride=hkv + 1)
    check_decode(lib, case, hq, 61, out=out)


@pytest.mark.parametrize("kv", ["fp8_e4m3", "int8"])
@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("q_type", ["bf16", "f32"])
def test_decode_split_and_static_scales(lib, kv, out, q_type):
    for scales in ("block", "head"):
        case = PC.make(70, kv, [1, 700, 2049, 64, 65], 2, 128, 16, scales=scales)
        w = 4096 if scales == "head" else 0   # without a window, one scale per head is plain decode
        check_decode(lib, case, 8, 71, q_type=q_type, out=out, partition=64, window=w)
        check_decode(lib, case, 8, 72, q_type=q_type, out=out, scale=-0.05, window=w)
        check_decode(lib, case, 8, 73, q_type=q_type, out=out, scale=0.0, window=w)


@pytest.mark.parametrize("kv", ["fp8_e4m3", "int8"])
def test_decode_scales_far_apart(lib, kv):
    """Scales of neighbouring blocks that differ by e^6 and more: the weights stay in range."""
    case = PC.make(80, kv, [500, 33, 257], 2, 128, 16, spread=3.0)
    case.ks = np.minimum(case.ks, np.float32(8.0 / OB.QMAX[kv]))
    for out in ("bf16", "f32"):
        check_decode(lib, case, 8, 81, out=out)
    case.vs[:] *= np.float32(2.0 ** -40)
    check_decode(lib, case, 8, 82, out="f32")
    case.vs[:] *= np.float32(2.0 ** 90)
    check_decode(lib, case, 8, 83, out="f32")
    check_decode(lib, case, 8, 84, out="f32", qmul=1e-5)


def test_write_then_attend_then_read(lib):
    """The calls as a decode loop uses them: append a prompt, then tokens one by one, attend
    after each, read the cache back; the same step captured into a graph and replayed."""
    import torch
    kv, bs, d, hkv, hq = "fp8_e4m3", 16, 128, 2, 8
    lens = [37, 5, 64]
    steps = 6
    case = PC.make(90, kv, [n + steps for n in lens], hkv, d, bs)
    case.lens = list(lens)
    case.ks[:], case.vs[:] = np.nan, np.nan
    dev = case.device()
    x, y = rows(91, sum(lens), hkv, d, "bf16"), rows(92, sum(lens), hkv, d, "bf16")
    append(lib, case, x, y, lens, "bf16", dev=dev)
    want = [a.copy() for a in (case.k, case.v, case.ks, case.vs)]
    OB.quantize_and_cache(x, y, np.concatenate([[0], np.cumsum(lens)]), case.tables, lens, *want,
                          "bf16", kv)
    kn = torch.empty((3, hkv, d), dtype=torch.bfloat16, device="cuda")
    vn, q = torch.empty_like(kn), torch.empty((3, hq, d), dtype=torch.bfloat16, device="cuda")
    out = torch.empty((3, hq, d), dtype=torch.float32, device="cuda")
    cap = case.tables.shape[1] * bs
    ws = torch.empty(max(16, lib.workspace_bytes(3, hq, hkv, d, cap, 64, window=0)),
                     dtype=torch.uint8, device="cuda")

    def step():
        lib.quantize_and_cache(kn, vn, dev["k"], dev["v"], dev["ks"], dev["vs"], dev["tables"],
                               dev["lens"])
        lib.paged_attention_decode(q, dev["k"], dev["v"], dev["tables"], dev["lens"], d ** -0.5, cap,
                                   out=out, k_scale=dev["ks"], v_scale=dev["vs"], workspace=ws,
                                   partition=64)

    graph = None
    for i in range(steps):
        a, b = rows(100 + i, 3, hkv, d, "bf16"), rows(200 + i, 3, hkv, d, "bf16")
        qn = rows(300 + i, 3, hq, d, "bf16", 0.0)
        kn.copy_(GC.to_torch(a, "bf16"))
        vn.copy_(GC.to_torch(b, "bf16"))
        q.copy_(GC.to_torch(qn, "bf16"))
        dev["lens"] += 1
        now = [n + i + 1 for n in lens]
        OB.quantize_and_cache(a, b, [0, 1, 2, 3], case.tables, now, *want, "bf16", kv)
        if i < 2:
            step()
        else:
            if graph is None:
                torch.cuda.synchronize()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    step()
            graph.replay()
        torch.cuda.synchronize()
        now_case = PC.Paged(kv, now, case.tables, *want)
        q64 = GC.OA.to_f64(qn, "bf16")
        for s, n in enumerate(now):
            K, V = now_case.values(s)
            o, mag, reach = OB.attend(q64[s:s + 1], [n - 1], K, V, d ** -0.5, 0, 0)
            # scales of untouched blocks are NaN: bound from those in use
            used = PC.Paged(kv, now, case.tables, *want[:2], np.nan_to_num(want[2]), np.nan_to_num(want[3]))
            lim = PC.attention_bound(used, q64[s:s + 1], o, mag, reach, d ** -0.5, False, False, True, n)
            assert (np.abs(out[s].cpu().numpy() - o[0]) <= lim[0]).all()
    for n, w in zip(("k", "v", "ks", "vs"), want):
        assert GC.from_torch(dev[n], kv if n in "kv" else "f32").tobytes() == w.tobytes()


def test_other_stream(lib):
    """Allocation, append, read and attention on a given stream."""
    import torch
    kv, bs, d, hkv = "int8", 16, 128, 2
    case = PC.make(95, kv, [100, 50], hkv, d, bs)
    dev = case.device()
    q = torch.randn((2, 8, d), device="cuda").to(torch.bfloat16)
    start = torch.tensor([0, 100, 150], dtype=torch.int32, device="cuda")
    args = (q, dev["k"], dev["v"], dev["tables"], dev["lens"], d ** -0.5, 100)
    kw = {"k_scale": dev["ks"], "v_scale": dev["vs"]}
    a = lib.paged_attention_decode(*args, partition=64, **kw)
    ka, va = lib.gather_cache(dev["k"], dev["v"], dev["tables"], start, 150, 100, **kw)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    b = lib.paged_attention_decode(*args, partition=64, stream=st, **kw)
    kb, vb = lib.gather_cache(dev["k"], dev["v"], dev["tables"], start, 150, 100, stream=st, **kw)
    st.synchronize()
    assert torch.equal(a, b) and torch.equal(ka, kb) and torch.equal(va, vb)


def test_empty_batches(lib):
    """No sequence, and sequences without rows: nothing is written, outputs are empty or 0."""
    import torch
    nb, bs, hkv, d = 4, 16, 2, 128
    cache = torch.full((nb, bs, hkv, d), 5, dtype=torch.int8, device="cuda")
    sc = torch.ones((nb, hkv), device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    rows = torch.zeros((0, hkv, d), device="cuda")
    kw = {"k_scale": sc, "v_scale": sc}
    q = torch.zeros((0, 4, d), dtype=torch.bfloat16, device="cuda")
    for S, start in ((0, i32(0)), (2, i32(0, 0, 0))):
        bt = torch.zeros((S, 2), dtype=torch.int32, device="cuda")
        lens = torch.zeros(S, dtype=torch.int32, device="cuda")
        lib.quantize_and_cache(rows, rows, cache, cache, sc, sc, bt, lens, query_start=start,
                               max_query_len=0)
        k, v = lib.gather_cache(cache, cache, bt, start, 0, 0, **kw)
        assert k.shape == v.shape == (0, hkv, d)
        assert lib.paged_attention_prefill(q, start, cache, cache, bt, lens, 0.1, 0, 0, **kw).shape == (0, 4, d)
        qs = torch.ones((S, 4, d), dtype=torch.bfloat16, device="cuda")
        out = lib.paged_attention_decode(qs, cache, cache, bt, lens, 0.1, 0, **kw)
        assert out.shape == (S, 4, d) and (out == 0).all()
    assert (cache == 5).all() and (sc == 1).all()


def test_requantise_chain(lib):
    """Rows read back and appended to another cache at once, call after call with new rows in
    the same buffers: each call sees what the one before it wrote."""
    import torch
    nb, bs, hkv, d, n = 40, 16, 8, 128, 600
    torch.manual_seed(3)
    xs = [torch.randn((n, hkv, d), device="cuda") * (i + 1) for i in range(20)]
    bt = torch.randperm(nb, device="cuda").to(torch.int32)[None, :38].contiguous()
    lens, start = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in ([n], [0, n]))
    new = lambda dt: (torch.zeros((nb, bs, hkv, d), dtype=dt, device="cuda"),
                      torch.zeros((nb, hkv), device="cuda"))

    def step(x, c, e, buf, wait):
        sync = torch.cuda.synchronize if wait else (lambda: None)
        lib.quantize_and_cache(x, x, c[0], c[2], c[1], c[3], bt, lens, start, n)
        sync()
        lib.gather_cache(c[0], c[2], bt, start, n, n, k_scale=c[1], v_scale=c[3], k_out=buf[0], v_out=buf[1])
        sync()
        lib.quantize_and_cache(buf[0], buf[1], e[0], e[2], e[1], e[3], bt, lens, start, n)
        sync()
        return lib.gather_cache(e[0], e[2], bt, start, n, n, k_scale=e[1], v_scale=e[3],
                                out_dtype=torch.float32)[0]
    runs = []
    for wait in (True, False):
        c, e = new(torch.int8) + new(torch.int8), new(torch.uint8) + new(torch.uint8)
        buf = [torch.zeros((n, hkv, d), device="cuda") for _ in range(2)]
        runs.append([step(x, c, e, buf, wait) for x in xs])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(*runs))


@pytest.mark.parametrize("kv", ["int8", "bf16"])
def test_blocks_past_32_bit_offsets(lib, kv):
    """Blocks beyond 4 GiB of a cache give what the same blocks of a small cache give."""
    import torch
    bs, hkv, d, S, n = 64, 8, 128, 3, 200
    size = 1 if kv == "int8" else 2
    nb = (1 << 32) // (bs * hkv * d * size) + 64
    dt = torch.int8 if kv == "int8" else torch.bfloat16
    big = [torch.empty((nb, bs, hkv, d), dtype=dt, device="cuda") for _ in range(2)]
    far = torch.arange(nb - 16, nb - 16 + 4 * S, device="cuda").to(torch.int32).view(S, 4)
    near = (far - (nb - 16)).contiguous()
    torch.manual_seed(5)
    small = [torch.randint(-127, 128, (16, bs, hkv, d), device="cuda").to(dt) for _ in range(2)]
    for b, s in zip(big, small):
        b[nb - 16:] = s
    lens = torch.full((S,), n, dtype=torch.int32, device="cuda")
    start = torch.arange(0, S * 30 + 1, 30, device="cuda").to(torch.int32)
    q = torch.randn((S * 30, 16, d), device="cuda").to(torch.bfloat16)
    res = []
    for (k, v), bt, blocks in ((big, far, nb), (small, near, 16)):
        kw = {}
        if kv == "int8":
            kw = {w: torch.zeros((blocks, hkv), device="cuda") for w in ("k_scale", "v_scale")}
            torch.manual_seed(6)
            for x in kw.values():
                x[-16:] = torch.rand((16, hkv), device="cuda") + 0.5
            torch.manual_seed(7)
            x = torch.randn((S * 30, hkv, d), device="cuda") * 90
            lib.quantize_and_cache(x, x, k, v, kw["k_scale"], kw["v_scale"], bt, lens, start, 30)
        first = lens - 100
        rows = torch.arange(0, S * 100 + 1, 100, device="cuda").to(torch.int32)
        r = list(lib.gather_cache(k, v, bt, rows, S * 100, 100, first_pos=first, **kw))
        r.append(lib.paged_attention_decode(q[:S].contiguous(), k, v, bt, lens, 0.01, n, window=90, **kw))
        r.append(lib.paged_attention_prefill(q, start, k, v, bt, lens, 0.01, 30, n, window=90, **kw))
        res.append(r)
    assert all(torch.equal(a, b) for a, b in zip(*res))


def test_two_streams_at_once(lib):
    """Calls on two streams, each with its own buffers, as one after the other."""
    import torch
    kv, bs, d, hkv = "fp8_e4m3", 16, 128, 4
    case = PC.make(96, kv, [700, 333, 12], hkv, d, bs)
    q = torch.randn((3, 16, d), device="cuda").to(torch.bfloat16)
    streams = [torch.cuda.Stream() for _ in range(2)]
    devs = [case.device() for _ in range(2)]
    x = torch.randn((3, hkv, d), device="cuda") * 3
    torch.cuda.synchronize()

    def step(dev, st):
        lib.quantize_and_cache(x, x, dev["k"], dev["v"], dev["ks"], dev["vs"], dev["tables"], dev["lens"],
                               stream=st)
        return lib.paged_attention_decode(q, dev["k"], dev["v"], dev["tables"], dev["lens"], 0.08, 700,
                                          k_scale=dev["ks"], v_scale=dev["vs"], partition=64, stream=st)
    ref = case.device()
    torch.cuda.synchronize()
    want = [step(ref, torch.cuda.current_stream()) for _ in range(8)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(8):
        for i in range(2):
            got[i].append(step(devs[i], streams[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
