"""Operators measured as a user's program calls them: the cache written in 8 bits with a scale
per block and head, read back, attention over it, and attention with a sliding window and sinks.

``own`` False: plain torch (products, sums, exp, comparisons, indexing) in 32 bits.
``own`` True: the calls of this package on the same inputs.
"""
import math

import torch

own = False

CODES = {"fp8": torch.float8_e4m3fn, "int8": torch.int8}
QMAX = {"fp8": 448.0, "int8": 127.0}
FLOATS = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4, "fp8": 1, "int8": 1}
MIN_SCALE = 2.0 ** -64


# ------------------------------------------------------------------ cases
def _write(name, kv, src, seqs, heads, dim, block, new_min, new, ctx_min, ctx):
    """Append new_min..new tokens a sequence, whose context is then ctx_min..ctx tokens."""
    return {"name": name, "op": "write", "kv": kv, "src": src, "seqs": seqs, "heads": heads,
            "dim": dim, "block": block, "new_min": new_min, "new": new, "ctx_min": ctx_min,
            "ctx": ctx}


def _read(name, kv, out, seqs, heads, dim, block, ctx_min, ctx):
    return {"name": name, "op": "read", "kv": kv, "out": out, "seqs": seqs, "heads": heads,
            "dim": dim, "block": block, "ctx_min": ctx_min, "ctx": ctx}


def _attend(name, op, kv, out, seqs, group, heads, dim, block, new_min, new, ctx_min, ctx, window,
            sinks):
    return {"name": name, "op": op, "kv": kv, "out": out, "seqs": seqs, "group": group,
            "heads": heads, "dim": dim, "block": block, "new_min": new_min, "new": new,
            "ctx_min": ctx_min, "ctx": ctx, "window": window, "sinks": sinks}


def listed():
    return [
        # one decode step's append for a small batch: the smallest call
        _write("write_step_fp8", "fp8", "bf16", 8, 8, 128, 16, 1, 1, 40, 900),
        # the append of a full chunked-prefill step: 16 chunks of 512 tokens, 32 heads
        _write("write_chunk_fp8", "fp8", "bf16", 16, 32, 128, 16, 512, 512, 512, 4096),
        # ragged chunks that start inside blocks, fp32 rows, odd head count
        _write("write_ragged_int8", "int8", "f32", 37, 5, 64, 32, 1, 131, 131, 700),
        # cached contexts read back for reuse elsewhere (prefix export)
        _read("read_fp8_bf16", "fp8", "bf16", 16, 8, 128, 16, 512, 4096),
        # a few short, odd lengths and an odd row
        _read("read_ragged_int8", "int8", "f32", 5, 3, 80, 8, 1, 301),
        # one decode layer with 32 heads and contexts of 512..4096 tokens
        _attend("decode_block_fp8", "decode", "fp8", "bf16", 32, 1, 32, 128, 16, 1, 1, 512, 4096,
                0, 0),
        # few long contexts: the work is split along the context
        _attend("decode_block_int8_long", "decode", "int8", "f32", 8, 4, 8, 128, 256, 1, 1, 32768,
                131072, 0, 0),
        # a grouped-query layer that attends 1024 recent tokens and 4 first ones
        _attend("decode_window_bf16", "decode", "bf16", "f32", 64, 8, 8, 128, 128, 1, 1, 1024, 8192,
                1024, 4),
        # a small batch of short contexts, some inside the window: latency
        _attend("decode_window_small", "decode", "bf16", "bf16", 4, 4, 8, 128, 16, 1, 1, 1, 600,
                256, 4),
        # a chunked-prefill step, 32 heads, behind cached prefixes
        _attend("prefill_window_bf16", "prefill", "bf16", "f32", 16, 1, 32, 128, 16, 512, 512, 512,
                4096, 1024, 4),
        # ragged chunks of a grouped-query layer, a wide window and many sinks
        _attend("prefill_window_ragged", "prefill", "bf16", "bf16", 3, 8, 8, 128, 128, 1, 700, 700,
                9000, 4096, 128),
        # a chunked-prefill step over a cache held in 8 bits
        _attend("prefill_block_fp8", "prefill", "fp8", "bf16", 16, 4, 8, 128, 16, 512, 512, 512,
                4096, 0, 0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: batch, lengths and heads over their ranges, odd sizes among them."""
    op = rng.choice(["write", "read", "decode", "decode", "prefill"])
    kv = rng.choice(["fp8", "int8"])
    block = rng.choice([8, 16, 32, 64, 128, 256])
    heads = rng.choice([1, 2, 3, 4, 5, 8, 16, 32])
    seqs = _log(rng, 1, 128)
    ctx = _log(rng, 1, 32768)
    ctx_min = max(1, int(ctx * rng.uniform(0.02, 1.0)))
    new = min(ctx, _log(rng, 1, 2048))
    new_min = max(1, int(new * rng.uniform(0.02, 1.0)))
    if op in ("write", "read"):
        dim, kind = rng.choice([64, 80, 128, 256]), rng.choice(["bf16", "f32"])
        if op == "read":
            heads = min(heads, 10 ** 8 // (ctx * dim))
            seqs = max(1, min(seqs, 10 ** 8 // (ctx * heads * dim)))
            case = _read("", kv, kind, seqs, heads, dim, block, ctx_min, ctx)
        else:
            seqs = max(1, min(seqs, 2 ** 25 // (new * heads * dim), 2 ** 28 // (ctx * heads * dim)))
            case = _write("", kv, kind, seqs, heads, dim, block, new_min, new, max(ctx_min, new), ctx)
    else:
        # a 16-bit cache is read through a window, an 8-bit one with or without
        kv = rng.choice(["bf16", kv])
        group = rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16])
        window = _log(rng, 16, 8192) if kv == "bf16" or rng.random() < 0.5 else 0
        sinks = rng.choice([0, 1, 4, 64, 129]) if window else 0
        out = rng.choice(["bf16", "f32"])
        if op == "decode":
            dim = rng.choice([64, 128, 128, 256]) if kv == "bf16" else 128
            seqs = max(1, min(seqs, 2 ** 28 // (ctx * heads * dim)))
            new = new_min = 1
        else:
            dim, out = 128, out if kv == "bf16" else "bf16"
            seen = min(ctx, window + sinks + new) if window else ctx
            heads = max(1, min(heads, 7 * 10 ** 8 // (group * new * seen)))
            seqs = max(1, min(seqs, 7 * 10 ** 8 // (group * heads * new * seen), 2 ** 21 // (ctx * heads)))
        case = _attend("", op, kv, out, seqs, group, heads, dim, block, new_min, new,
                       max(ctx_min, new), ctx, window, sinks)
    del case["name"]
    return case


def _spread(n, lo, hi, step):
    """n lengths between lo and hi, both ends among them where n allows; the same for every seed."""
    if n == 1:
        return [hi]
    return [hi if i == 0 else lo if i == 1 else lo + int((hi - lo + 1) * ((i * step) % 1.0))
            for i in range(n)]


def _lengths(case):
    """Contexts (new tokens included) and new tokens of each sequence."""
    n = case["seqs"]
    ctx = _spread(n, case["ctx_min"], case["ctx"], 0.6180339887)
    if case["op"] in ("decode", "read"):
        return ctx, [1] * n
    return ctx, _spread(n, case["new_min"], case["new"], 0.7548776662)


def _visible(case, pos):
    """Keys that the query at position pos sees."""
    if not case["window"]:
        return pos + 1
    return pos + 1 - max(0, pos + 1 - case["window"] - case["sinks"])


def work(case):
    ctx, new = _lengths(case)
    heads, dim, block = case["heads"], case["dim"], case["block"]
    if case["op"] == "write":
        rows = sum(new) * heads * 2
        blocks = sum((c - 1) // block - (c - n) // block + 1 for c, n in zip(ctx, new))
        return {"bytes": rows * dim * (BYTES[case["src"]] + 1) + blocks * heads * 2 * 4,
                "flops": 3 * rows * dim}
    if case["op"] == "read":
        rows = sum(ctx) * heads * 2
        blocks = sum(-(-c // block) for c in ctx)
        return {"bytes": rows * dim * (BYTES[case["out"]] + 1) + blocks * heads * 2 * 4,
                "flops": rows * dim}
    # attention: every row of the cache that some query sees, q and the output once
    q_heads = heads * case["group"]
    keys = pairs = 0
    for c, n in zip(ctx, new):
        if case["window"]:
            first = c - n          # the chunk's first position
            start = max(0, first + 1 - case["window"])
            keys += c - start + min(case["sinks"], start)
        else:
            keys += c
        pairs += sum(_visible(case, p) for p in range(c - n, c))
    scale_bytes = 0 if case["kv"] == "bf16" else keys * heads * 2 * 4 // block
    return {"bytes": keys * heads * dim * 2 * BYTES[case["kv"]] + scale_bytes
            + sum(new) * q_heads * dim * (2 + BYTES[case["out"]]),
            "flops": 4 * pairs * q_heads * dim}


# ----------------------------------------------------------------- inputs
def _normal(gen, shape, spread):
    """Rows of a projection: normal values, channels of unequal size."""
    size = torch.exp(spread * torch.randn(shape[-2:], generator=gen, device="cuda"))
    return torch.randn(shape, generator=gen, device="cuda") * size


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    ctx, new = _lengths(case)
    heads, dim, block, kv = case["heads"], case["dim"], case["block"], case["kv"]
    n, per = case["seqs"], -(-max(ctx) // block)
    need = [-(-c // block) for c in ctx]
    total = sum(need) + sum(need) // 8 + 1
    # the pool's blocks are handed out in no order; table entries past a context are -1
    perm = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    start = torch.tensor([0] + need, device="cuda").cumsum(0)[:-1]
    col = torch.arange(per, device="cuda")
    used = col[None, :] < torch.tensor(need, device="cuda")[:, None]
    at = (start[:, None] + col[None, :]).clamp(max=total - 1)
    tables = torch.where(used, perm[at], -1).to(torch.int32).contiguous()
    state = {"case": case, "tables": tables, "ctx": torch.tensor(ctx, dtype=torch.int32, device="cuda"),
             "max_ctx": max(ctx), "max_new": max(new), "tokens": sum(new),
             "starts": torch.tensor([0] + new, device="cuda").cumsum(0).to(torch.int32),
             "rows": torch.tensor([0] + ctx, device="cuda").cumsum(0).to(torch.int32),
             "num_rows": sum(ctx), "scale": float(torch.tensor(dim ** -0.5, dtype=torch.float32))}
    shape = (total, block, heads, dim)
    for name in ("k", "v"):
        if kv == "bf16":
            state[name + "_cache"] = _normal(gen, shape, 0.3).to(torch.bfloat16)
            continue
        # codes that fill their type's range, scales that differ from block to block
        x = torch.randn(shape, generator=gen, device="cuda") * (QMAX[kv] / 4.0)
        state[name + "_cache"] = (x.clamp(-448, 448).to(CODES[kv]) if kv == "fp8"
                                  else x.round().clamp(-127, 127).to(torch.int8))
        s = torch.exp(0.3 * torch.randn((total, heads), generator=gen, device="cuda"))
        state[name + "_scale"] = s * (4.0 / QMAX[kv])
    if case["op"] == "write":
        for name in ("k", "v"):
            x = _normal(gen, (sum(new), heads, dim), 0.3)
            state[name + "_new"] = x.to(FLOATS[case["src"]])
    elif case["op"] in ("decode", "prefill"):
        rows = (sum(new), heads * case["group"], dim)
        state["q"] = torch.randn(rows, generator=gen, device="cuda").to(torch.bfloat16)
    return state


# ------------------------------------------------------------ plain forms
def _bits(cache):
    """The cache as something that indexing takes."""
    return cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache


def _values(rows, like):
    return (rows.view(like.dtype) if like.dtype == torch.float8_e4m3fn else rows).float()


def _encode(x, kv):
    if kv == "fp8":
        return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.nan_to_num(x, nan=0.0).round().clamp(-128, 127).to(torch.int8)


def _token_places(starts, first, rows):
    """For every row of a ragged batch: its sequence and its position."""
    row = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(starts[1:].long(), row, right=True)
    return seq, first.long()[seq] + row - starts.long()[seq]


def _plain_write(state):
    case = state["case"]
    kv, block, heads = case["kv"], case["block"], case["heads"]
    qmax = torch.full((), QMAX[kv], device="cuda")   # a tensor: divided by, not multiplied
    first = state["ctx"] - (state["starts"][1:] - state["starts"][:-1])
    seq, pos = _token_places(state["starts"], first, state["tokens"])
    blk = state["tables"][seq, pos // block].long()
    off = pos % block
    total = state["k_scale"].shape[0]
    # the first new offset of every touched block; `block` where none is touched
    begin = torch.full((total,), block, device="cuda").scatter_reduce(0, blk, off, "amin")
    touched = begin < block
    # only the block in which a sequence's new tokens begin can hold older ones
    joined = state["tables"].gather(1, first[:, None].long() // block)[:, 0].long()
    older = torch.arange(block, device="cuda")[None, :] < (first % block)[:, None]
    for name in ("k", "v"):
        x = state[name + "_new"].float()
        finite = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
        amax = torch.zeros((total, heads), device="cuda").scatter_reduce(
            0, blk[:, None].expand(-1, heads), finite, "amax")
        cache, scales = _bits(state[name + "_cache"]), state[name + "_scale"]
        fresh = (amax / qmax).clamp(min=MIN_SCALE)
        # a block with older tokens: its scale grows by the least power of two that fits
        _, e = torch.frexp(amax / (scales * qmax))
        steps = torch.ldexp(torch.ones_like(amax), (e - 1).clamp(min=0))
        steps = torch.where(amax > steps * scales * qmax, 2 * steps, steps)
        grown = scales * torch.where(amax > scales * qmax, steps, 1.0)
        s = torch.where(begin[:, None] == 0, fresh, grown)
        s = torch.where(touched[:, None], s, scales)
        kept = cache[joined]
        again = _values(kept, state[name + "_cache"]) * (scales / s)[joined][:, None, :, None]
        cache[joined] = torch.where(older[:, :, None, None], _encode(again, kv), kept)
        cache[blk, off] = _encode(x / s[blk][..., None], kv)
        scales.copy_(s)
    return {k: state[k] for k in ("k_cache", "v_cache", "k_scale", "v_scale")}


def _rows(state, name, blk, off):
    """Rows [.., heads, dim] of the cache at (block, offset), as the values they stand for."""
    cache = state[name + "_cache"]
    x = _values(_bits(cache)[blk, off], cache)
    return x * state[name + "_scale"][blk][..., None] if name + "_scale" in state else x


def _plain_read(state):
    case = state["case"]
    seq, pos = _token_places(state["rows"], torch.zeros_like(state["ctx"]), state["num_rows"])
    blk = state["tables"][seq, pos // case["block"]].long()
    return {name: _rows(state, name, blk, pos % case["block"]).to(FLOATS[case["out"]])
            for name in ("k", "v")}


def _plain_attend(state):
    """Sequences side by side, padded; scores, mask, softmax and products in 32 bits."""
    case = state["case"]
    heads, group, dim, block = case["heads"], case["group"], case["dim"], case["block"]
    window, sinks, n = case["window"], case["sinks"], state["max_new"]
    ctx = state["ctx"].long()
    count = (state["starts"][1:] - state["starts"][:-1]).long()
    first = ctx - count
    # the keys of a sequence: all of its context, or the sinks and what its queries' windows reach
    if window:
        low = (first + 1 - window).clamp(min=0)
        span = min(state["max_ctx"], n + window - 1)
        key = torch.cat([torch.arange(sinks, device="cuda").expand(ctx.shape[0], sinks),
                         low[:, None] + torch.arange(span, device="cuda")], 1)
        is_sink = torch.arange(sinks + span, device="cuda") < sinks
        real = torch.where(is_sink, key < low[:, None], key < ctx[:, None])
    else:
        key = torch.arange(state["max_ctx"], device="cuda").expand(ctx.shape[0], -1)
        real = key < ctx[:, None]
    at = torch.where(real, key, 0)
    blk = state["tables"].gather(1, at // block).long()
    k, v = (_rows(state, name, blk, at % block) for name in ("k", "v"))  # [S, L, heads, dim]
    query = first[:, None] + torch.arange(n, device="cuda")              # positions [S, n]
    there = torch.arange(n, device="cuda") < count[:, None]
    row = torch.where(there, state["starts"][:-1, None].long() + torch.arange(n, device="cuda"), 0)
    q = state["q"].float()[row].view(-1, n, heads, group, dim).permute(0, 2, 3, 1, 4)
    s = q.reshape(-1, heads, group * n, dim) @ k.permute(0, 2, 3, 1)
    s = s.view(-1, heads, group, n, key.shape[1]) * state["scale"]
    sees = real[:, None, :] & (key[:, None, :] <= query[..., None])
    if window:
        sees = sees & ((key[:, None, :] > query[..., None] - window) | (key[:, None, :] < sinks))
    s = s.masked_fill(~sees[:, None, None], float("-inf"))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = p.view(-1, heads, group * n, key.shape[1]) @ v.permute(0, 2, 1, 3)
    o = o.view(-1, heads, group, n, dim).permute(0, 3, 1, 2, 4).reshape(-1, n, heads * group, dim)
    return o[there].to(FLOATS[case["out"]])


# ------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if not own:
        return {"write": _plain_write, "read": _plain_read, "decode": _plain_attend,
                "prefill": _plain_attend}[case["op"]](state)
    import paged_kv_cache_295_gb300 as pkv
    if case["op"] == "write":
        pkv.quantize_and_cache(state["k_new"], state["v_new"], state["k_cache"], state["v_cache"],
                               state["k_scale"], state["v_scale"], state["tables"], state["ctx"],
                               query_start=state["starts"], max_query_len=state["max_new"])
        return {k: state[k] for k in ("k_cache", "v_cache", "k_scale", "v_scale")}
    if case["op"] == "read":
        k, v = pkv.gather_cache(state["k_cache"], state["v_cache"], state["tables"], state["rows"],
                                state["num_rows"], state["max_ctx"], k_scale=state["k_scale"],
                                v_scale=state["v_scale"], out_dtype=FLOATS[case["out"]])
        return {"k": k, "v": v}
    more = {"k_scale": state.get("k_scale"), "v_scale": state.get("v_scale"),
            "window": case["window"], "sinks": case["sinks"], "out_dtype": FLOATS[case["out"]]}
    if case["op"] == "prefill":
        return pkv.paged_attention_prefill(state["q"], state["starts"], state["k_cache"],
                                           state["v_cache"], state["tables"], state["ctx"],
                                           state["scale"], state["max_new"], state["max_ctx"], **more)
    if "workspace" not in state:   # kept by the program from step to step
        size = pkv.workspace_bytes(case["seqs"], case["heads"] * case["group"], case["heads"],
                                   case["dim"], state["max_ctx"], window=case["window"],
                                   sinks=case["sinks"])
        state["workspace"] = torch.empty(max(size, 16), dtype=torch.uint8, device="cuda")
    return pkv.paged_attention_decode(state["q"], state["k_cache"], state["v_cache"], state["tables"],
                                      state["ctx"], state["scale"], state["max_ctx"],
                                      workspace=state["workspace"], **more)


# ---------------------------------------------------------- 64-bit results
def _round_code(x, kv):
    """The nearest code's value, ties to even, of float64 x."""
    if kv == "int8":
        return torch.round(x).clamp(-128, 127)
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -30))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_write(state, case):
    kv, block = case["kv"], case["block"]
    qmax = QMAX[kv]
    tables, ctx, starts = (state[k].tolist() for k in ("tables", "ctx", "starts"))
    out = {}
    for name in ("k", "v"):
        x = state[name + "_new"].double()
        values = state[name + "_cache"].float().double()
        scales = state[name + "_scale"].double().clone()
        for s, c in enumerate(ctx):
            row, pos = starts[s], c - (starts[s + 1] - starts[s])
            # whole blocks at once, then the partly filled ends one by one
            while pos < c:
                b, off = tables[s][pos // block], pos % block
                blocks = (c - pos) // block if off == 0 else 0
                if blocks > 1:
                    ids = torch.tensor(tables[s][pos // block: pos // block + blocks], device="cuda")
                    part = x[row: row + blocks * block].view(blocks, block, *x.shape[1:])
                    sc = (part.abs().amax((1, 3)) / qmax).clamp(min=MIN_SCALE).float().double()
                    values[ids] = _round_code((part / sc[:, None, :, None]).float().double(), kv)
                    scales[ids] = sc
                    row, pos = row + blocks * block, pos + blocks * block
                    continue
                m = min(block - off, c - pos)
                part = x[row: row + m]
                top = part.abs().amax((0, 2))
                if off == 0:
                    sc = (top / qmax).clamp(min=MIN_SCALE).float().double()
                else:
                    old = scales[b].clone()
                    k = torch.ceil(torch.log2((top / (old * qmax).float().double()))).clamp(min=0)
                    sc = old * torch.exp2(k)
                    kept = values[b, :off]
                    moved = _round_code(kept * torch.exp2(-k)[None, :, None], kv)
                    values[b, :off] = torch.where((k > 0)[None, :, None], moved, kept)
                values[b, off: off + m] = _round_code((part / sc[None, :, None]).float().double(), kv)
                scales[b] = sc
                row, pos = row + m, pos + m
        out[name + "_cache"] = values if kv == "fp8" else None
        out[name + "_scale"] = scales
    return out


def _exact_values(state, name, ids):
    """float64 [tokens, heads, dim] of the blocks `ids`, in their order."""
    x = state[name + "_cache"][ids] if state[name + "_cache"].dtype != torch.float8_e4m3fn else \
        state[name + "_cache"].view(torch.uint8)[ids].view(torch.float8_e4m3fn)
    x = x.double() if x.dtype != torch.float8_e4m3fn else x.float().double()
    if name + "_scale" in state:
        x = x * state[name + "_scale"][ids].double()[:, None, :, None]
    return x.flatten(0, 1)


def exact(case, seed):
    state = prepare(case, seed)
    if case["op"] == "write":
        return _exact_write(state, case)
    ctx, new = _lengths(case)
    block = case["block"]
    parts = {"k": [], "v": [], "o": []}
    row = 0
    for s, (c, n) in enumerate(zip(ctx, new)):
        ids = state["tables"][s, : -(-c // block)].long()
        k, v = (_exact_values(state, name, ids)[:c] for name in ("k", "v"))
        if case["op"] == "read":
            parts["k"].append(k)
            parts["v"].append(v)
            continue
        q = state["q"][row: row + n].double()
        row += n
        j = torch.arange(c, device="cuda")
        o = torch.empty_like(q)
        for h in range(case["heads"]):
            mine = slice(h * case["group"], (h + 1) * case["group"])
            for a in range(0, n, 256):
                p = torch.arange(c - n + a, min(c - n + a + 256, c), device="cuda")
                sees = j[None, :] <= p[:, None]
                if case["window"]:
                    sees &= (p[:, None] - j[None, :] < case["window"]) | (j[None, :] < case["sinks"])
                z = torch.einsum("tgd,jd->tgj", q[a: a + 256, mine], k[:, h]) * state["scale"]
                z = torch.where(sees[:, None, :], z, float("-inf"))
                o[a: a + 256, mine] = torch.einsum("tgj,jd->tgd", torch.softmax(z, -1), v[:, h])
        parts["o"].append(o)
    if case["op"] == "read":
        return {name: torch.cat(parts[name]) for name in ("k", "v")}
    return torch.cat(parts["o"])
