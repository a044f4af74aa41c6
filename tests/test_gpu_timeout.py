"""The bounded device waits, made to run out without faulting anything.

Every mbarrier wait in the TMA decode kernels gives up after 2 s: the warp
flags PKV_DEV_TIMEOUT in the caller's status word, waits (again bounded) for
its other copies in flight, leaves its share out and returns, so the context
stays usable.  pkv_test_decode_stall arms one barrier phase of the transposed
kernel for 16 bytes more than its copies bring; the copies land, that phase
never completes and the wait runs out.  A normal call right after must match
the oracle again.
"""
import time

import numpy as np
import pytest

import workloads as W
from tests import gpu_cases as GC

pytestmark = pytest.mark.gpu


def test_decode_wait_runs_out_flags_timeout_and_the_next_call_is_clean(lib):
    import torch
    assert torch.cuda.is_available()
    w = W.DecodeWorkload("stall", 3, 8, 2, 128, 16, "bf16", "bf16", seed=71, ctx_law="fixed")
    case, _ = GC.make_small(w, lens=[700, 40, 300])
    eng, outs, st = GC.run_gpu(case, partition=64)
    assert st == 0
    kc, vc = GC.oracle_caches(case, 0)
    ref = GC.oracle_out(case, 0, kc, vc)
    assert np.abs(outs[0].astype(np.float64) - ref).max() <= 2e-3
    q = GC.to_torch(case.q[0], "bf16")
    tables = torch.from_numpy(case.tables).cuda()
    ctx = torch.from_numpy(case.lens.astype(np.int32)).cuda()
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    lib.stall_decode_for_test(16)
    try:
        t0 = time.monotonic()
        eng.attend(0, q, tables, ctx, int(case.lens.max()), partition=64, device_status=status)
        torch.cuda.synchronize()
        waited = time.monotonic() - t0
    finally:
        lib.stall_decode_for_test(0)
    assert int(status.item()) & lib.DEV_TIMEOUT, int(status.item())
    assert 1.5 <= waited < 30.0, waited    # the 2 s bound ran out, once
    # the context is still usable and the next call is exact again
    status.zero_()
    out = eng.attend(0, q, tables, ctx, int(case.lens.max()), partition=64,
                     device_status=status)
    torch.cuda.synchronize()
    assert int(status.item()) == 0
    got = out.cpu().numpy()
    assert got.tobytes() == outs[0].tobytes()
    assert np.abs(got.astype(np.float64) - ref).max() <= 2e-3


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3", "int8"])
def test_windowed_waits_run_out_and_the_next_calls_are_clean(lib, kv):
    """Windowed decode and prefill: the prefill's first V tile is a cut one, so the softmax
    warps that would clear its hidden rows give up beside the product's issuer."""
    import torch
    from tests import paged_cases as PC
    lens, new = [50, 40, 300], [50, 1, 130]
    case = PC.make(72, kv, lens, 2, 128, 16)
    d = case.device()
    q = torch.randn((sum(new), 8, 128), device="cuda").to(torch.bfloat16)
    start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device="cuda")
    kw = {"k_scale": d.get("ks"), "v_scale": d.get("vs"), "window": 30, "sinks": 2}
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def both():
        for call in (lambda: lib.paged_attention_decode(q[:3].contiguous(), d["k"], d["v"], d["tables"],
                                                        d["lens"], 0.09, 300, device_status=status, **kw),
                     lambda: lib.paged_attention_prefill(q, start, d["k"], d["v"], d["tables"], d["lens"],
                                                         0.09, 130, 300, device_status=status, **kw)):
            status.zero_()
            torch.cuda.synchronize()
            t0 = time.monotonic()
            out = call()
            torch.cuda.synchronize()
            yield out, int(status.item()), time.monotonic() - t0

    clean = [(out, st) for out, st, _ in both()]
    assert [st for _, st in clean] == [0, 0]
    lib.stall_decode_for_test(16)
    try:
        for _, st, waited in both():
            assert st & lib.DEV_TIMEOUT, st
            assert 1.5 <= waited < 30.0, waited
    finally:
        lib.stall_decode_for_test(0)
    for (out, st, _), (want, _) in zip(both(), clean):
        assert st == 0 and torch.equal(out, want)


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3", "int8"])
def test_prefill_waits_run_out_and_the_next_call_is_clean(lib, kv):
    """The plain prefill, whose only V tile is a cut one: as above."""
    import torch
    from tests import paged_cases as PC
    lens = [50, 40, 30]
    case = PC.make(73, kv, lens, 2, 128, 16, scales="head")
    d = case.device()
    q = torch.randn((sum(lens), 8, 128), device="cuda").to(torch.bfloat16)
    start = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def call():
        status.zero_()
        torch.cuda.synchronize()
        t0 = time.monotonic()
        out = lib.paged_attention_prefill(q, start, d["k"], d["v"], d["tables"], d["lens"], 0.09, 50, 50,
                                          k_scale=d.get("ks"), v_scale=d.get("vs"), device_status=status)
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
