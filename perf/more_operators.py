"""Operators of the step around the cache, measured as a user's program calls them: block tables
and slots built on the GPU from request lengths, rotary positions (one axis or several) with the
append of the rotated rows, and attention over whole packed prompts.

``own`` False: plain torch (products, sums, exp, comparisons, indexing) in 32 bits.
``own`` True: the calls of this package on the same inputs.
"""
import math

import torch

own = False

FLOATS = {"bf16": torch.bfloat16, "f32": torch.float32}
CACHES = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f32": 4, "fp8": 1}


# ------------------------------------------------------------------ cases
def _slots(name, seqs, block, new_min, new, ctx_min, ctx):
    """Sequences of ctx_min..ctx cached tokens that get new_min..new more."""
    return {"name": name, "op": "slots", "seqs": seqs, "block": block, "new_min": new_min,
            "new": new, "ctx_min": ctx_min, "ctx": ctx}


def _rotary(name, src, kv, tokens, heads, kv_heads, dim, rot, axes, adjacent, far, keep_k):
    """``kv``: the cache's type, "" for none; ``far``: positions go up to this."""
    return {"name": name, "op": "rotary", "src": src, "kv": kv, "tokens": tokens, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "rot": rot, "axes": axes, "adjacent": adjacent,
            "far": far, "keep_k": keep_k, "block": 16}


def _prompt(name, out, seqs, heads, kv_heads, dim, new_min, new, extra, causal, window, sinks):
    """``extra``: keys that a sequence has before its queries (0: as many keys as queries)."""
    return {"name": name, "op": "prompt", "out": out, "seqs": seqs, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "new_min": new_min, "new": new, "extra": extra,
            "causal": causal, "window": window, "sinks": sinks}


def listed():
    return [
        # one decode step of a small batch: the smallest call
        _slots("slots_step_small", 8, 16, 1, 1, 40, 900),
        # one decode step of a large batch
        _slots("slots_step", 512, 16, 1, 1, 1, 8192),
        # prompts and chunks of very different lengths scheduled together
        _slots("slots_prompts", 64, 16, 1, 2047, 0, 4096),
        # one decode step's rotation and append for a small batch
        _rotary("rotary_step", "bf16", "bf16", 8, 32, 8, 128, 128, 1, False, 4096, False),
        # a prompt with images: time, height and width; the rotated keys also go to the attention
        _rotary("rotary_prompt_axes", "bf16", "bf16", 8192, 32, 8, 128, 128, 3, False, 32768, True),
        # a chunked-prefill step into an 8-bit cache, at far positions
        _rotary("rotary_far_fp8", "bf16", "fp8", 8191, 32, 32, 128, 128, 1, False, 1000000, False),
        # part of each head rotated, neighbouring dims as pairs, float32 rows, no cache
        _rotary("rotary_part_f32", "f32", "", 777, 6, 2, 80, 32, 2, True, 5000, True),
        # a few very short prompts: latency
        _prompt("prompt_small", "bf16", 4, 32, 8, 128, 1, 60, 0, True, 0, 0),
        # prompts of a layer with 32 heads
        _prompt("prompt_mha", "bf16", 16, 32, 32, 128, 512, 512, 0, True, 0, 0),
        # a few long prompts of very different lengths, grouped heads
        _prompt("prompt_long", "bf16", 3, 32, 8, 128, 700, 8192, 0, True, 0, 0),
        # ragged chunks behind keys of their own, a window and sinks, float32 output
        _prompt("prompt_window_f32", "f32", 9, 16, 2, 64, 1, 1500, 333, True, 1024, 4),
        # patches of images: every patch sees its whole image, heads of 80
        _prompt("prompt_images", "bf16", 11, 16, 16, 80, 64, 1156, 0, False, 0, 0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case: batch, lengths and heads over their ranges, odd sizes among them."""
    op = rng.choice(["slots", "rotary", "rotary", "prompt", "prompt", "prompt"])
    if op == "slots":
        seqs, ctx = _log(rng, 1, 1024), _log(rng, 1, 16384)
        new = rng.choice([1, _log(rng, 1, 4096)])
        new = max(1, min(new, 65536 // seqs))
        case = _slots("", seqs, rng.choice([8, 16, 24, 32, 64, 128, 256]),
                      1 if new == 1 else int(new * rng.uniform(0.0, 1.0)), new,
                      int(ctx * rng.uniform(0.0, 1.0)), ctx)
    elif op == "rotary":
        src = rng.choice(["bf16", "bf16", "f32"])
        kv = rng.choice(["", src, "fp8"])
        dim = rng.choice([64, 80, 96, 128, 256])
        rot = rng.choice([dim, dim, dim // 2, 16, 32])
        kv_heads, group = rng.choice([1, 2, 3, 4, 5, 8, 16, 32]), rng.choice([1, 2, 3, 4, 6, 7, 8])
        tokens = _log(rng, 1, 16384)
        tokens = max(1, min(tokens, 70 * 10 ** 6 // (kv_heads * (group + 2) * dim * BYTES[src] // 2)))
        case = _rotary("", src, kv, tokens, kv_heads * group, kv_heads, dim, rot,
                       rng.choice([1, 1, 2, 3]), rng.random() < 0.3, _log(rng, 64, 10 ** 6),
                       kv == "" or rng.random() < 0.5)
    else:
        dim = rng.choice([64, 128, 128, 80, 96])
        kv_heads, group = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8, 16])
        seqs, new = _log(rng, 1, 64), _log(rng, 1, 8192)
        extra = rng.choice([0, 0, _log(rng, 1, 2000)])
        causal = rng.random() < 0.75
        window = _log(rng, 16, 4096) if causal and rng.random() < 0.4 else 0
        sinks = rng.choice([0, 1, 4, 64, 129]) if window else 0
        # no more scores and rows than the largest listed case has
        kv_heads = max(1, min(kv_heads, 14 * 10 ** 8 // (group * new * (new + extra))))
        seqs = max(1, min(seqs, 14 * 10 ** 8 // (kv_heads * group * new * (new + extra)),
                          6 * 10 ** 7 // ((kv_heads * group * new + kv_heads * extra) * dim)))
        case = _prompt("", rng.choice(["bf16", "bf16", "f32"]), seqs, kv_heads * group, kv_heads,
                       dim, max(1, int(new * rng.uniform(0.02, 1.0))), new, extra, causal, window,
                       sinks)
    del case["name"]
    return case


def _spread(n, lo, hi, step):
    """n lengths between lo and hi, both ends among them where n allows; the same for every seed."""
    if n == 1:
        return [hi]
    return [hi if i == 0 else lo if i == 1 else lo + int((hi - lo + 1) * ((i * step) % 1.0))
            for i in range(n)]


def _lengths(case):
    """Cached tokens and new ones of each sequence; keys and queries of a prompt."""
    new = _spread(case["seqs"], case["new_min"], case["new"], 0.7548776662)
    if case["op"] == "slots":
        return _spread(case["seqs"], case["ctx_min"], case["ctx"], 0.6180339887), new
    return [n + case["extra"] for n in new], new


def _sections(case):
    """How many frequencies each axis has: about a quarter for the first of several."""
    half, axes = case["rot"] // 2, case["axes"]
    if axes == 1:
        return [half]
    first = half // 4 if axes == 3 else half // 3
    rest = (half - first) // (axes - 1)
    return [first] + [rest] * (axes - 2) + [half - first - rest * (axes - 2)]


def work(case):
    if case["op"] == "slots":
        ctx, new = _lengths(case)
        block = case["block"]
        need = sum(-(-(c + n) // block) - -(-c // block) for c, n in zip(ctx, new))
        opened = sum(1 for c in ctx if c % block)
        return {"bytes": 16 * len(ctx) + 4 * opened + 8 * need + 12 * sum(new), "flops": 0}
    if case["op"] == "rotary":
        src, dim, t = BYTES[case["src"]], case["dim"], case["tokens"]
        rows = case["heads"] * 2 + case["kv_heads"] * (1 + (1 if case["keep_k"] else 0))
        bytes_ = rows * dim * src * t + 4 * case["axes"] * t
        if case["kv"]:
            bytes_ += case["kv_heads"] * dim * (src + 2 * BYTES[case["kv"]]) * t + 8 * t
        return {"bytes": bytes_,
                "flops": 3 * t * (case["heads"] + case["kv_heads"]) * case["rot"]}
    keys, new = _lengths(case)
    pairs = 0
    for c, n in zip(keys, new):
        if not case["causal"]:
            pairs += c * n
            continue
        for p in range(c - n, c):
            pairs += p + 1
            if case["window"]:
                pairs -= max(0, p + 1 - case["window"] - case["sinks"])
    return {"bytes": sum(new) * case["heads"] * case["dim"] * (2 + BYTES[case["out"]])
            + sum(keys) * case["kv_heads"] * case["dim"] * 4,
            "flops": 4 * pairs * case["heads"] * case["dim"]}


# ----------------------------------------------------------------- inputs
def _normal(gen, shape, spread):
    """Rows of a projection: normal values, channels of unequal size."""
    size = torch.exp(spread * torch.randn(shape[-2:], generator=gen, device="cuda"))
    return torch.randn(shape, generator=gen, device="cuda") * size


def _starts(lengths):
    return torch.tensor([0] + lengths, device="cuda").cumsum(0).to(torch.int32)


def _prepare_slots(case, gen):
    ctx, new = _lengths(case)
    block, n = case["block"], case["seqs"]
    # no two seeds have the same lengths at the same places
    order = torch.randperm(n, generator=gen, device="cuda")
    ctx = torch.tensor(ctx, dtype=torch.int32, device="cuda")[order].contiguous()
    new_lens = torch.tensor(new, dtype=torch.int32, device="cuda")[order].contiguous()
    width = -(-(case["ctx"] + case["new"]) // block)
    held = (ctx + block - 1) // block
    most = n * (-(-case["new"] // block) + 1)
    used = n * -(-case["ctx"] // block)
    total = used + most + 7
    # the pool's blocks in no order: some are the sequences', the others free; 5 have been taken
    perm = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")
    first = held.cumsum(0) - held
    at = (first[:, None] + col[None, :]).clamp(max=total - 1)
    tables = torch.where(col[None, :] < held[:, None], perm[at], -1).to(torch.int32).contiguous()
    return {"case": case, "ctx": ctx, "new": new_lens, "tables": tables, "num_blocks": total,
            "free": perm[used:].contiguous(),
            "free_start": torch.full((1,), 5, dtype=torch.int32, device="cuda"),
            "tokens": sum(new),
            # the program's buffers, kept from step to step
            "slot_mapping": torch.empty(sum(new), dtype=torch.int64, device="cuda"),
            "positions": torch.empty(sum(new), dtype=torch.int32, device="cuda"),
            "query_start": torch.empty(n + 1, dtype=torch.int32, device="cuda"),
            "context_out": torch.empty(n, dtype=torch.int32, device="cuda"),
            "free_next": torch.empty(1, dtype=torch.int32, device="cuda")}


def _prepare_rotary(case, gen):
    t, heads, kv_heads, dim = (case[k] for k in ("tokens", "heads", "kv_heads", "dim"))
    # q, k and v are parts of one projection's rows
    qkv = _normal(gen, (t, heads + 2 * kv_heads, dim), 0.3).to(FLOATS[case["src"]])
    state = {"case": case, "q": qkv[:, :heads], "k": qkv[:, heads: heads + kv_heads],
             "v": qkv[:, heads + kv_heads:]}
    begin = torch.randint(0, case["far"], (case["axes"], 1), generator=gen, device="cuda")
    step = torch.arange(t, device="cuda")
    grid = torch.stack([step, step // 16, step % 16][: case["axes"]])
    state["positions"] = (begin + grid).to(torch.int32).contiguous()
    half = case["rot"] // 2
    freq = 10000.0 ** (-torch.arange(half, dtype=torch.float64) / half)
    state["freq"] = freq.cuda()
    state["axis"] = torch.repeat_interleave(torch.arange(case["axes"]),
                                            torch.tensor(_sections(case))).cuda()
    if case["kv"]:
        blocks = -(-t // case["block"]) + 3
        state["slots"] = torch.randperm(blocks * case["block"], generator=gen, device="cuda")[:t].contiguous()
        for name in ("k", "v"):
            shape = (blocks, case["block"], kv_heads, dim)
            x = torch.randn(shape, generator=gen, device="cuda")
            state[name + "_cache"] = x.to(CACHES[case["kv"]])
            if case["kv"] == "fp8":
                # four standard deviations of a channel reach the largest code
                s = torch.exp(0.3 * torch.randn(kv_heads, generator=gen, device="cuda"))
                state[name + "_scale"] = s * (4.0 / 448.0)
    return state


def _prepare_prompt(case, gen):
    keys, new = _lengths(case)
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    state = {"case": case, "q_start": _starts(new), "k_start": _starts(keys), "most_new": max(new),
             "most_keys": max(keys), "scale": float(torch.tensor(dim ** -0.5, dtype=torch.float32))}
    if case["extra"]:
        state["q"] = torch.randn((sum(new), heads, dim), generator=gen, device="cuda").to(torch.bfloat16)
        for name in ("k", "v"):
            state[name] = _normal(gen, (sum(keys), kv_heads, dim), 0.3).to(torch.bfloat16)
    else:
        # as many keys as queries: q, k and v are parts of one projection's rows
        qkv = torch.randn((sum(new), heads + 2 * kv_heads, dim), generator=gen, device="cuda")
        qkv[:, heads:] *= torch.exp(0.3 * torch.randn((2 * kv_heads, dim), generator=gen, device="cuda"))
        qkv = qkv.to(torch.bfloat16)
        state["q"], state["k"] = qkv[:, :heads], qkv[:, heads: heads + kv_heads]
        state["v"] = qkv[:, heads + kv_heads:]
    return state


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    return {"slots": _prepare_slots, "rotary": _prepare_rotary,
            "prompt": _prepare_prompt}[case["op"]](case, gen)


# ------------------------------------------------------------ plain forms
def _plain_slots(state):
    block, tables, rows = state["case"]["block"], state["tables"], state["tokens"]
    ctx, new = state["ctx"].long(), state["new"].long()
    held = (ctx + block - 1) // block
    end = (ctx + new + block - 1) // block
    need = end - held
    base = state["free_start"].long() + need.cumsum(0) - need
    starts = torch.cat([torch.zeros(1, dtype=torch.int64, device="cuda"), new.cumsum(0)])
    col = torch.arange(tables.shape[1], device="cuda")
    taken = (col[None, :] >= held[:, None]) & (col[None, :] < end[:, None])
    at = torch.where(taken, base[:, None] + col[None, :] - held[:, None], 0)
    tables.copy_(torch.where(taken, state["free"][at], tables))
    row = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(starts[1:], row, right=True)
    pos = ctx[seq] + row - starts[seq]
    slots = tables[seq, pos // block].long() * block + pos % block
    return {"tables": tables, "slot_mapping": slots, "positions": pos.to(torch.int32),
            "query_start": starts.to(torch.int32), "context_lens": (ctx + new).to(torch.int32),
            "free_start": (state["free_start"] + need.sum()).to(torch.int32)}


def _turn(x, cos, sin, case):
    """Rows [T, heads, dim] turned by the angles [T, rot / 2]."""
    rot = case["rot"]
    if case["adjacent"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
    y1, y2 = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([y1, y2], -1).flatten(-2) if case["adjacent"] else torch.cat([y1, y2], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_rotary(state):
    case = state["case"]
    # positions up to a million: the angles in 64 bits
    angle = state["positions"].double()[state["axis"]].t() * state["freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q = _turn(state["q"].float(), cos, sin, case)
    k = _turn(state["k"].float(), cos, sin, case)
    out = {"q": q.to(state["q"].dtype)}
    if case["keep_k"]:
        out["k"] = k.to(state["k"].dtype)
    if case["kv"]:
        for name, x in (("k", k), ("v", state["v"].float())):
            cache = state[name + "_cache"]
            flat = cache.view(-1, *cache.shape[2:])
            if case["kv"] == "fp8":
                codes = (x / state[name + "_scale"][:, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
                flat.view(torch.uint8)[state["slots"]] = codes.view(torch.uint8)
            else:
                flat[state["slots"]] = x.to(cache.dtype)
            out[name + "_cache"] = cache
    return out


def _plain_prompt(state):
    """Sequences side by side, padded; scores, mask, softmax and products in 32 bits."""
    case = state["case"]
    heads, kv_heads, dim = case["heads"], case["kv_heads"], case["dim"]
    group, n, c = heads // kv_heads, state["most_new"], state["most_keys"]
    q_start, k_start = state["q_start"].long(), state["k_start"].long()
    new, keys = q_start[1:] - q_start[:-1], k_start[1:] - k_start[:-1]
    i, j = torch.arange(n, device="cuda"), torch.arange(c, device="cuda")
    there, real = i < new[:, None], j < keys[:, None]
    q_row = torch.where(there, q_start[:-1, None] + i, 0)
    k_row = torch.where(real, k_start[:-1, None] + j, 0)
    q = state["q"].float()[q_row].view(-1, n, kv_heads, group, dim).permute(0, 2, 3, 1, 4)
    k = state["k"].float()[k_row].permute(0, 2, 3, 1)
    v = state["v"].float()[k_row].permute(0, 2, 1, 3)
    s = (q.reshape(-1, kv_heads, group * n, dim) @ k).view(-1, kv_heads, group, n, c) * state["scale"]
    sees = real[:, None, :].expand(-1, n, -1)
    if case["causal"]:
        place = (keys - new)[:, None, None] + i[:, None]
        sees = sees & (j <= place)
        if case["window"]:
            sees = sees & ((j > place - case["window"]) | (j < case["sinks"]))
    s = s.masked_fill(~sees[:, None, None], float("-inf"))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    p = p / p.sum(-1, keepdim=True)
    o = p.view(-1, kv_heads, group * n, c) @ v
    o = o.view(-1, kv_heads, group, n, dim).permute(0, 3, 1, 2, 4).reshape(-1, n, heads, dim)
    return o[there].to(FLOATS[case["out"]])


# ------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    if not own:
        return {"slots": _plain_slots, "rotary": _plain_rotary,
                "prompt": _plain_prompt}[case["op"]](state)
    import paged_kv_cache_295_gb300 as pkv
    if case["op"] == "slots":
        got = pkv.slots_from_lengths(
            state["tables"], state["ctx"], state["new"], state["free"], state["num_blocks"],
            case["block"], state["tokens"], free_start=state["free_start"],
            slot_mapping=state["slot_mapping"], positions=state["positions"],
            query_start=state["query_start"], context_out=state["context_out"],
            free_next=state["free_next"])
        return {"tables": state["tables"], "slot_mapping": got.slot_mapping,
                "positions": got.positions, "query_start": got.query_start,
                "context_lens": got.context_lens, "free_start": got.free_start}
    if case["op"] == "rotary":
        if "plan" not in state:   # kept by the model
            state["plan"] = pkv.Rotary(case["rot"], base=10000.0, sections=_sections(case),
                                       adjacent=case["adjacent"])
        caches = {}
        if case["kv"]:
            caches = {"slot_mapping": state["slots"], "k_cache": state["k_cache"],
                      "v_cache": state["v_cache"], "k_scale": state.get("k_scale"),
                      "v_scale": state.get("v_scale")}
        q, k = pkv.rotary_and_cache(state["q"], state["k"], state["v"], state["positions"],
                                    state["plan"], keep_k=case["keep_k"], **caches)
        out = {"q": q}
        if case["keep_k"]:
            out["k"] = k
        if case["kv"]:
            out["k_cache"], out["v_cache"] = state["k_cache"], state["v_cache"]
        return out
    return pkv.packed_attention_prefill(
        state["q"], state["k"], state["v"], state["q_start"], state["scale"],
        key_start=state["k_start"] if case["extra"] else None, causal=case["causal"],
        window=case["window"], sinks=case["sinks"], out_dtype=FLOATS[case["out"]])


# ---------------------------------------------------------- 64-bit results
def _nearest_e4m3(x):
    """The nearest E4M3 value, ties to even, of float64 x."""
    e = torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -30))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_rotary(state, case):
    half, rot = case["rot"] // 2, case["rot"]
    sections = _sections(case)
    out = {}
    rows = {"q": state["q"].double(), "k": state["k"].double()}
    for x in rows.values():
        low = 0
        for axis, count in enumerate(sections):
            for f in range(low, low + count):
                turn = state["positions"][axis].double() * (10000.0 ** (-f / half))
                a, b = (2 * f, 2 * f + 1) if case["adjacent"] else (f, f + half)
                c, s = torch.cos(turn)[:, None], torch.sin(turn)[:, None]
                u, w = x[:, :, a].clone(), x[:, :, b].clone()
                x[:, :, a], x[:, :, b] = u * c - w * s, u * s + w * c
            low += count
        assert low * 2 == rot
    out["q"] = rows["q"]
    if case["keep_k"]:
        out["k"] = rows["k"]
    if case["kv"]:
        for name, x in (("k", rows["k"]), ("v", state["v"].double())):
            cache = state[name + "_cache"]
            full = cache.float().double().flatten(0, 1)
            if case["kv"] == "fp8":
                x = _nearest_e4m3(x / state[name + "_scale"].double()[:, None])
            full[state["slots"]] = x
            out[name + "_cache"] = full.view(cache.shape)
    return out


def exact(case, seed):
    if case["op"] == "slots":       # whole numbers only
        return None
    state = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(state, case)
    if work(case)["flops"] > 1.5e12:
        return None
    q_at, k_at = state["q_start"].tolist(), state["k_start"].tolist()
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(state["q"].shape, dtype=torch.float64, device="cuda")
    for s in range(case["seqs"]):
        q = state["q"][q_at[s]: q_at[s + 1]]
        k, v = (state[x][k_at[s]: k_at[s + 1]] for x in ("k", "v"))
        n, c = q.shape[0], k.shape[0]
        for a in range(0, n, 1024):
            b = min(a + 1024, n)
            last = c - n + b if case["causal"] else c     # keys that some of these queries see
            place = torch.arange(c - n + a, c - n + b, device="cuda")[:, None]
            j = torch.arange(last, device="cuda")[None, :]
            hidden = torch.zeros((b - a, last), dtype=torch.bool, device="cuda")
            if case["causal"]:
                hidden |= j > place
            if case["window"]:
                hidden |= (place - j >= case["window"]) & (j >= case["sinks"])
            for h in range(case["heads"]):
                z = q[a:b, h].double() @ k[:last, h // group].double().t() * state["scale"]
                z[hidden] = float("-inf")
                out[q_at[s] + a: q_at[s] + b, h] = torch.softmax(z, -1) @ v[:last, h // group].double()
    return out
