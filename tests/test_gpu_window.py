"""Attention with a sliding window and sinks on the GPU, against the numpy definition."""
import numpy as np
import pytest

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
    ws = torch.empty(lib.workspace_bytes(2, 8, 2, 128, 900, 64, window=0), dtype=torch.uint8, device="cuda")
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
