"""Cases of one serving step of a sliding-window model: plain torch forms, the library's calls, and 64-bit results.

Four operators, in the order a step calls them:

- tables: block tables, lengths, slots and positions of the step's new tokens, from how many tokens each request brings;
- norm_rope: each head's query and key rows normalised and rotated by their positions on the way into the paged cache;
- window_decode: attention of one query token a sequence over its last `window` cached tokens and its first `sinks` ones;
- window_prefill: the same for a chunk of new tokens of each sequence.

Blocks that no query of the step can see are not held: their table entries are -1, as an engine leaves them that gives
such blocks to other requests.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}
E4M3 = torch.float8_e4m3fn
# Cached codes are N(0, 56^2) (K) and N(0, 44^2) (V) draws, as in the library's E4M3 workloads.
K_SCALE, V_SCALE = 1.0 / 56.0, 1.0 / 44.0
# What the normalised rows of a head are stored by in an E4M3 cache: rows of about unit size, times weights around 1.
NORM_K_SCALE = 1.0 / 64.0
EPS = 1e-6


def _tables(name, batch, tokens, cached, block, free=1.25, spare=0):
    return {"name": name, "op": "tables", "batch": batch, "tokens": tokens, "cached": cached, "block": block, "free": free, "spare": spare}


def _norm_rope(name, tokens, heads, kv_heads, dim, rot, dtype, cache="same", interleaved=False, axes=1, packed=True, block=16,
               far=4096, weights="same", per_head=False):
    return {"name": name, "op": "norm_rope", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim, "rot": rot,
            "dtype": dtype, "cache": cache, "interleaved": interleaved, "axes": axes, "packed": packed, "block": block, "far": far,
            "weights": weights, "per_head": per_head}


def _decode(name, batch, heads, kv_heads, dim, dtype, window, sinks, context, cache="same", block=16, short=0):
    return {"name": name, "op": "window_decode", "batch": batch, "heads": heads, "kv_heads": kv_heads, "dim": dim, "dtype": dtype,
            "window": window, "sinks": sinks, "context": context, "cache": cache, "block": block, "short": short}


def _prefill(name, batch, tokens, heads, kv_heads, dim, dtype, window, sinks, cached, cache="same", block=16, even=False, spare=0):
    return {"name": name, "op": "window_prefill", "batch": batch, "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "dtype": dtype, "window": window, "sinks": sinks, "cached": cached, "cache": cache, "block": block, "even": even,
            "spare": spare}


def listed():
    return [
        # A decode step of a full batch: every request brings one token, a few need a new block. Latency is all there is.
        _tables("tables_decode_256", 256, 256, 32768, 16, spare=0),
        # Prompts of very different lengths at once, more than the free blocks hold: the last ones are refused.
        _tables("tables_prompts", 1000, 262144, 0, 32, free=0.9, spare=77),
        # One request decoding alone.
        _norm_rope("norm_rope_one_token", 1, 32, 8, 128, 128, "bf16"),
        # One token budget of chunked prefill, rows taken out of the packed projection.
        _norm_rope("norm_rope_chunk_16384", 16384, 32, 8, 128, 128, "bf16", far=32768),
        # Part of each head rotated, neighbouring elements paired, on the way into an E4M3 cache.
        _norm_rope("norm_rope_e4m3", 1023, 20, 4, 128, 64, "f16", cache="e4m3", interleaved=True, weights="f32"),
        # One request decoding alone behind a long context.
        _decode("window_decode_one", 1, 32, 8, 128, "bf16", 1024, 4, 5000),
        # The batch-32 decode layer with contexts up to 32k under a 4,096-token window.
        _decode("window_decode_b32", 32, 32, 8, 128, "bf16", 4096, 4, 32768),
        # An E4M3 cache; the window and the first tokens end inside blocks, some sequences are shorter than the window.
        _decode("window_decode_e4m3", 48, 32, 8, 128, "bf16", 2047, 5, 9001, cache="e4m3", block=32, short=1),
        # A full serving batch, most of it past the window.
        _decode("window_decode_b256", 256, 32, 8, 128, "f16", 2048, 16, 16384, block=32),
        # A small mixed step: short chunks and decoding requests together, 64 dims, no first tokens.
        _prefill("window_prefill_mixed", 13, 300, 16, 2, 64, "bf16", 128, 0, 700, block=32, spare=3),
        # One token budget: eight prompts' chunks of 2,048 tokens.
        _prefill("window_prefill_chunks", 8, 16384, 32, 8, 128, "bf16", 1024, 4, 6000, even=True),
        # A long prompt's chunk far into its context: the largest call, bound by the matrix products.
        _prefill("window_prefill_long", 1, 16384, 32, 8, 128, "f16", 4096, 4, 16384, block=64),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, even over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["tables", "norm_rope", "window_decode", "window_prefill"])
    if op == "tables":
        batch = _spread(rng, 1, 1024)
        case = _tables("", batch, batch + _spread(rng, 1, 65536) - 1, rng.choice([0, _spread(rng, 1, 32768)]), rng.choice([8, 16, 32, 48, 128]),
                       rng.choice([0.7, 1.0, 1.25, 2.0]), rng.choice([0, 0, 1, 100]))
    elif op == "norm_rope":
        dim, rot = rng.choice([(64, 64), (64, 32), (80, 20), (96, 96), (128, 128), (128, 64), (128, 96), (256, 64), (256, 256)])
        kv = rng.choice([1, 2, 3, 4, 8])
        cache = rng.choice(["same", "same", "same", "e4m3"])
        case = _norm_rope("", _spread(rng, 1, 16384), kv * rng.choice([1, 2, 3, 4]), kv, dim, rot, rng.choice(["bf16", "bf16", "f16", "f32"]),
                          cache, rng.random() < 0.4, rng.choice([1, 1, 2, 3]), rng.random() < 0.6, rng.choice([8, 16, 32, 48]),
                          _spread(rng, 64, 1000000), rng.choice(["same", "f32"]), rng.random() < 0.25)
        if cache == "e4m3":
            case["tokens"] = min(case["tokens"], 2_500_000 // (kv * dim))
    else:
        cache = rng.choice(["same", "same", "same", "e4m3"])
        dtype = rng.choice(["f16", "bf16"]) if cache == "e4m3" else rng.choice(["f16", "bf16", "bf16", "f32"])
        dim = 128 if cache == "e4m3" else rng.choice([64, 128, 128])
        block = rng.choice([8, 16, 24, 64]) if dtype == "f32" else rng.choice([16, 16, 32, 48, 64, 128])
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 4, 8])
        window, sinks = _spread(rng, 1, 8192), rng.choice([0, 1, 4, 4, 16, 100])
        if op == "window_decode":
            batch = _spread(rng, 1, 256)
            while batch * window * kv * dim > 256 * 2048 * 8 * 128 or (dtype == "f32" and batch * window * heads * dim > 1 << 30):
                window = max(1, window // 2)
            case = _decode("", batch, heads, kv, dim, dtype, window, sinks, _spread(rng, 1, 32768), cache, block, rng.choice([0, 0, 1, 3]))
            case["short"] = min(case["short"], batch - 1)
        else:
            tokens = _spread(rng, 1, 16384)
            limit = 1 << (30 if dtype == "f32" else 35 if cache == "e4m3" else 38)
            while tokens * window * heads * dim > limit:
                tokens, window = max(1, tokens * 2 // 3), max(1, window * 2 // 3)
            batch = rng.randint(1, min(tokens, 40))
            case = _prefill("", batch, tokens, heads, kv, dim, dtype, window, sinks, rng.choice([0, _spread(rng, 1, 32768)]), cache, block,
                            rng.random() < 0.3, rng.choice([0, 0, 1, 5]))
    del case["name"]
    return case


# ------------------------------------------------------------------ inputs


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _codes(g, shape, sigma):
    return (torch.randn(shape, generator=g, device="cuda") * sigma).clamp_(-448.0, 448.0).to(E4M3)


def _permutation(g, n):
    return torch.randperm(n, generator=g, device="cuda").cpu().numpy().astype(np.int32)


def _device(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).cuda()


def _asked(case):
    """New tokens of each request: one each, and the rest in shares that grow linearly over the batch."""
    b, rest = case["batch"], case["tokens"] - case["batch"]
    edge = [rest * i * (i + 1) // (b * (b + 1)) for i in range(b + 1)]
    return [1 + edge[i + 1] - edge[i] for i in range(b)]


def _held(case):
    """Cached tokens of each request before the step, evenly spread (before they are shuffled)."""
    return [case["cached"] * (i + 1) // case["batch"] for i in range(case["batch"])]


def _prepare_tables(case, seed):
    g = _generator(seed)
    bs = case["block"]
    order = _permutation(g, case["batch"])
    held, asked = np.array(_held(case), np.int64)[order], np.array(_asked(case), np.int64)[_permutation(g, case["batch"])]
    old, new = -(-held // bs), -(-(held + asked) // bs)
    used = int(old.sum())
    free = max(1, int((new - old).sum() * case["free"]))
    nb = used + free
    ids = _permutation(g, nb)
    mb = int(new.max())
    tables = np.full((case["batch"], mb), -1, np.int32)
    at = 0
    for s, n in enumerate(old):
        tables[s, :n] = ids[at:at + n]
        at += n
    # The free blocks stand in a ring of all blocks' size, from a place that many steps have moved it to.
    head = int(ids[0]) * 7919 % nb
    queue = np.full(nb, -1, np.int32)
    queue[(head + np.arange(free)) % nb] = ids[used:]
    T = case["tokens"] + case["spare"]
    s = {"op": "tables", "tables": _device(tables), "held": _device(held), "asked": _device(asked), "queue": _device(queue),
         "state": _device([head, free]), "bs": bs, "T": T, "new_blocks": int((new - old).sum())}
    if own:
        import paged_kv_cache_slots_gb300 as pkv

        s["out"] = pkv.make_step_tables(case["batch"], T, device="cuda")
    return s


def _axis_of(case):
    """Axis of each frequency: sections as even as they come, the first ones longer."""
    n, a = case["rot"] // 2, case["axes"]
    return [min(i * a // n, a - 1) for i in range(n)]


def _prepare_norm_rope(case, seed):
    g = _generator(seed)
    T, H, KV, D, bs = case["tokens"], case["heads"], case["kv_heads"], case["dim"], case["block"]
    dt = DTYPES[case["dtype"]]
    fp8 = case["cache"] == "e4m3"
    if case["packed"]:  # slices of the fused projection's output
        qkv = _normal(g, (T, H + 2 * KV, D), dt)
        q, k, v = qkv[:, :H], qkv[:, H:H + KV], qkv[:, H + KV:]
    else:
        q, k, v = (_normal(g, (T, n, D), dt) for n in (H, KV, KV))
    wt = DTYPES["f32" if case["weights"] == "f32" else case["dtype"]]
    qw, kw = ((1.0 + 0.2 * torch.randn((n, D) if case["per_head"] else (D,), generator=g, device="cuda")).to(wt) for n in (H, KV))
    # The tokens go to slots of a pool that has a quarter more blocks than they fill, in any order of blocks; of a longer
    # batch two tokens bring no row of their own (their slot is -1) and one is padding (its sequence id is negative).
    NB = -(-T // bs) * 5 // 4 + 1
    blocks = torch.randperm(NB, generator=g, device="cuda")[:-(-T // bs)]
    t = torch.arange(T, device="cuda")
    slots = (blocks[t // bs] * bs + t % bs).to(torch.int32)
    ids = torch.zeros(T, dtype=torch.int32, device="cuda")
    if T >= 8:
        slots[T // 3] = slots[T // 2] = -1
        ids[T - 1] = -1
    positions = torch.randint(0, case["far"], (case["axes"], T), generator=g, device="cuda", dtype=torch.int32)
    inv_freq = 10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64) / case["rot"])
    cache_dt = E4M3 if fp8 else dt
    one = NB * KV * bs * D
    buffer = torch.zeros(2 * one * SIZES["e4m3" if fp8 else case["dtype"]], dtype=torch.uint8, device="cuda")
    kc, vc = (x.view(cache_dt).view(NB, KV, bs, D) for x in buffer.chunk(2))
    s = {"op": "norm_rope", "q": q, "k": k, "v": v, "qw": qw, "kw": kw, "slots": slots, "ids": ids, "positions": positions,
         "inv_freq": inv_freq.cuda(), "axis": torch.tensor(_axis_of(case), device="cuda"), "interleaved": case["interleaved"],
         "kc": kc, "vc": vc, "bs": bs, "fp8": fp8, "q_out": torch.zeros((T, H, D), dtype=dt, device="cuda"),
         "written": ((slots >= 0) & (ids >= 0)).nonzero()[:, 0], "rotated": (ids >= 0).nonzero()[:, 0]}
    if own:
        import paged_kv_cache_slots_gb300 as pkv

        s["pool"] = pkv.KVPool(1, NB, bs, KV, D, cache_dt, device="cuda", buffer=buffer)
        s["rope"] = pkv.Rope(inv_freq, interleaved=case["interleaved"], axes=_axis_of(case))
    return s


def _cache(case, g, firsts, ctx):
    """Tables and a cache for sequences of ctx tokens of which the first `sinks` and those from firsts on can be seen."""
    bs, sinks, KV, D = case["block"], case["sinks"], case["kv_heads"], case["dim"]
    rows = [sorted({*range(-(-min(sinks, c) // bs)), *range(f // bs, -(-c // bs))}) for f, c in zip(firsts, ctx)]
    total = sum(len(r) for r in rows)
    NB = total * 9 // 8 + 1
    ids = _permutation(g, NB)
    tables = np.full((len(ctx), max(1, max(-(-c // bs) for c in ctx))), -1, np.int32)
    at = 0
    for s, r in enumerate(rows):
        tables[s, r] = ids[at:at + len(r)]
        at += len(r)
    fp8 = case["cache"] == "e4m3"
    shape, dt = (NB, KV, bs, D), DTYPES[case["dtype"]]
    kc = _codes(g, shape, 56.0) if fp8 else _normal(g, shape, dt)
    vc = _codes(g, shape, 44.0) if fp8 else _normal(g, shape, dt)
    return {"kc": kc, "vc": vc, "tables": _device(tables), "ctx": _device(ctx), "scale": 1.0 / math.sqrt(D), "fp8": fp8,
            "window": case["window"], "sinks": sinks}


def _contexts(case):
    """Contexts of 1 to `context` tokens, evenly spread (before they are shuffled), the first `short` ones empty."""
    n, b = case["context"], case["batch"]
    return [0 if i < case["short"] else n - (b - 1 - i) * (n - 1) // max(1, b - 1) for i in range(b)]


def _prepare_decode(case, seed):
    g = _generator(seed)
    ctx = np.array(_contexts(case), np.int64)[_permutation(g, case["batch"])]
    s = {"op": "window_decode", **_cache(case, g, np.maximum(ctx - case["window"], 0).tolist(), ctx.tolist())}
    shape, dt = (case["batch"], case["heads"], case["dim"]), DTYPES[case["dtype"]]
    s["q"], s["out"] = _normal(g, shape, dt), torch.empty(shape, dtype=dt, device="cuda")
    s["seen"] = max(1, min(case["window"], int(ctx.max())))
    if own:
        import paged_kv_cache_slots_gb300 as pkv

        s["workspace"] = pkv.make_workspace(case["batch"], case["heads"], case["kv_heads"], case["dim"], device="cuda")
    return s


def _chunks(case):
    """New tokens of each sequence: even shares, or all of one size class from single tokens to long chunks."""
    if not case["even"]:
        return _asked(case)
    b, T = case["batch"], case["tokens"]
    return [T * (i + 1) // b - T * i // b for i in range(b)]


def _prepare_prefill(case, seed):
    g = _generator(seed)
    new, held = _chunks(case), _held(case)
    ctx = [n + h for n, h in zip(new, held)]
    s = {"op": "window_prefill", **_cache(case, g, [max(0, h + 1 - case["window"]) for h in held], ctx)}
    # `spare` rows of the batch's buffers stand behind its last sequence.
    shape, dt = (case["tokens"] + case["spare"], case["heads"], case["dim"]), DTYPES[case["dtype"]]
    s["q"], s["out"] = _normal(g, shape, dt), torch.zeros(shape, dtype=dt, device="cuda")
    s["start"] = _device(np.concatenate([[0], np.cumsum(new)]))
    s["new"], s["held"] = new, held
    if own:
        import paged_kv_cache_slots_gb300 as pkv

        s["workspace"] = pkv.make_window_prefill_workspace(case["batch"], shape[0], case["heads"], case["kv_heads"], case["dim"],
                                                           device="cuda")
    return s


def prepare(case, seed):
    return {"tables": _prepare_tables, "norm_rope": _prepare_norm_rope, "window_decode": _prepare_decode,
            "window_prefill": _prepare_prefill}[case["op"]](case, seed)


# ------------------------------------------------------------- plain forms


def _plain_tables(s):
    bs, T, tables = s["bs"], s["T"], s["tables"]
    held, asked, state = s["held"].long(), s["asked"].long(), s["state"].long()
    B, MB = tables.shape
    cap = s["queue"].shape[0]
    old, new = (held + bs - 1) // bs, (held + asked + bs - 1) // bs
    need = new - old
    upto = need.cumsum(0)
    granted = ((need == 0) | (upto <= state[1])) & (asked.cumsum(0) <= T) & (new <= MB)
    n = asked * granted
    first = upto - need
    # The new entries of each row.
    e = torch.arange(MB, device=held.device)
    fresh = granted[:, None] & (e >= old[:, None]) & (e < new[:, None])
    taken = s["queue"][(state[0] + first[:, None] + e - old[:, None]) % cap]
    tables.copy_(torch.where(fresh, taken, tables))
    # The tokens, in the sequences' order.
    end = n.cumsum(0)
    t = torch.arange(T, device=held.device)
    seq = torch.searchsorted(end, t, right=True)
    live = seq < B
    seq = seq.clamp(max=B - 1)
    pos = held[seq] + t - (end - n)[seq]
    block = tables[seq, (pos // bs).clamp(max=MB - 1)].long()
    minus = torch.full_like(t, -1)
    used = (need * granted).sum()
    return (tables, (held + n).int(), torch.cat((torch.zeros_like(end[:1]), end)).int(), torch.where(live, block * bs + pos % bs, minus).int(),
            torch.where(live, pos, torch.zeros_like(t)).int(), torch.where(live, seq, minus).int(),
            torch.stack(((state[0] + used) % cap, state[1] - used)).int())


def _rotate(x, cos, sin, interleaved):
    """x [T, heads, D] in fp32, its first 2n elements rotated pair by pair by the angles whose cos, sin are [T, n]."""
    n = cos.shape[1]
    cos, sin = cos[:, None], sin[:, None]
    if interleaved:
        a, b = x[..., 0:2 * n:2], x[..., 1:2 * n:2]
        turned = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :n], x[..., n:2 * n]
        turned = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((turned, x[..., 2 * n:]), -1)


def _normed(x, w):
    x = x.float()
    return x * torch.rsqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + EPS) * w.float()


def _plain_norm_rope(s):
    angle = s["positions"][s["axis"]].t().double() * s["inv_freq"]  # far positions need more than 32 bits
    cos, sin = angle.cos().float(), angle.sin().float()
    q = _rotate(_normed(s["q"], s["qw"]), cos, sin, s["interleaved"]).to(s["q_out"].dtype)
    s["q_out"][s["rotated"]] = q[s["rotated"]]
    w = s["written"]
    k = _rotate(_normed(s["k"], s["kw"]), cos, sin, s["interleaved"])[w]
    v = s["v"].float()[w]
    at = s["slots"][w].long()
    kc, vc = s["kc"], s["vc"]
    if s["fp8"]:
        k = (k / NORM_K_SCALE).clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)
        v = (v / V_SCALE).clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)
        kc, vc = kc.view(torch.uint8), vc.view(torch.uint8)
    kc[at // s["bs"], :, at % s["bs"]] = k.to(kc.dtype)
    vc[at // s["bs"], :, at % s["bs"]] = v.to(vc.dtype)
    return s["q_out"], s["kc"], s["vc"]


def _rows(s, name, tables, pos):
    """Rows at positions pos (per table row) of a paged cache in fp32, [n, KV, count, D]; what lies past a table is any row."""
    cache = s[name]
    bs = cache.shape[2]
    blk = tables.gather(1, (pos // bs).clamp(0, tables.shape[1] - 1)).clamp(min=0).long()
    if not s["fp8"]:
        return cache[blk, :, pos % bs].float().transpose(1, 2)
    codes = cache.view(torch.uint8)[blk, :, pos % bs].contiguous().view(E4M3)
    return (codes.float() * (K_SCALE if name == "kc" else V_SCALE)).transpose(1, 2)


def _softmax(scores, seen):
    """exp(scores - their maximum) where seen, and their sum (1 where nothing is seen)."""
    scores = scores.masked_fill(~seen, -torch.inf)
    top = scores.amax(-1, keepdim=True)
    e = (scores - torch.where(top == -torch.inf, torch.zeros_like(top), top)).exp_()
    total = e.sum(-1, keepdim=True)
    return e, torch.where(total == 0, torch.ones_like(total), total)


def _plain_decode(s):
    B, H, D = s["q"].shape
    KV = s["kc"].shape[1]
    ctx = s["ctx"].long()[:, None]
    lo = (ctx - s["window"]).clamp(min=0)
    near = lo + torch.arange(s["seen"], device=ctx.device)
    far = torch.arange(s["sinks"], device=ctx.device).expand(B, -1)
    pos = torch.cat((far, near), 1)
    seen = torch.cat((far < lo, near < ctx), 1)
    scores = s["q"].float().view(B, KV, H // KV, D) * s["scale"] @ _rows(s, "kc", s["tables"], pos).transpose(-1, -2)
    e, total = _softmax(scores, seen[:, None, None])
    # (What stands behind a hidden weight is any row: weights of 0 meet finite values only.)
    return (e @ _rows(s, "vc", s["tables"], pos) / total).view(B, H, D).to(s["q"].dtype)


def _plain_prefill(s, step=1024):
    H, D = s["q"].shape[1:]
    KV = s["kc"].shape[1]
    at = 0
    for i, (n, held) in enumerate(zip(s["new"], s["held"])):
        for t0 in range(0, n, step):
            m = min(step, n - t0)
            p = held + t0 + torch.arange(m, device="cuda")[:, None]
            lo = max(0, held + t0 + 1 - s["window"])
            pos = torch.cat((torch.arange(min(s["sinks"], lo), device="cuda"), torch.arange(lo, held + t0 + m, device="cuda")))
            seen = (pos <= p) & ((pos > p - s["window"]) | (pos < s["sinks"]))
            row = slice(at + t0, at + t0 + m)
            q = s["q"][row].float().view(m, KV, H // KV, D).permute(1, 2, 0, 3) * s["scale"]  # [KV, G, m, D]
            k, v = (_rows(s, name, s["tables"][i:i + 1], pos[None])[0] for name in ("kc", "vc"))
            e, total = _softmax(q @ k.transpose(-1, -2)[:, None], seen)
            s["out"][row] = (e @ v[:, None] / total).permute(2, 0, 1, 3).reshape(m, H, D).to(s["out"].dtype)
        at += n
    return s["out"]


def run(state):
    s = state
    if not own:
        return {"tables": _plain_tables, "norm_rope": _plain_norm_rope, "window_decode": _plain_decode,
                "window_prefill": _plain_prefill}[s["op"]](s)
    import paged_kv_cache_slots_gb300 as pkv

    if s["op"] == "tables":
        o = pkv.extend_tables(s["tables"], s["held"], s["asked"], s["queue"], s["state"], s["bs"], s["T"], out=s["out"])
        return s["tables"], o.context_lens, o.query_start, o.slot_mapping, o.positions, o.seq_ids, o.queue_state
    if s["op"] == "norm_rope":
        scales = {"k_scale": NORM_K_SCALE, "v_scale": V_SCALE} if s["fp8"] else {}
        s["pool"].append_norm_rope(0, s["k"], s["v"], s["slots"], s["positions"], s["rope"], s["kw"], q=s["q"], q_weight=s["qw"], eps=EPS,
                                   q_out=s["q_out"], seq_ids=s["ids"], **scales)
        return s["q_out"], s["kc"], s["vc"]
    scales = {"k_scale": K_SCALE, "v_scale": V_SCALE} if s["fp8"] else {}
    if s["op"] == "window_decode":
        return pkv.paged_window_decode_attention(s["q"], s["kc"], s["vc"], s["tables"], s["ctx"], s["scale"], s["window"], s["sinks"],
                                                 out=s["out"], workspace=s["workspace"], **scales)
    return pkv.paged_window_prefill_attention(s["q"], s["kc"], s["vc"], s["tables"], s["start"], s["ctx"], s["scale"], s["window"],
                                              s["sinks"], out=s["out"], workspace=s["workspace"], **scales)


# ----------------------------------------------------------- work and exact


def _grants(case):
    """(granted requests' tokens, their new blocks) with the requests in listed order: what a step of this size hands out."""
    bs, want, tokens, blocks = case["block"], 0, 0, 0
    held, asked = _held(case), _asked(case)
    need = [-(-(h + n) // bs) - -(-h // bs) for h, n in zip(held, asked)]
    free = max(1, int(sum(need) * case["free"]))
    for n, b in zip(asked, need):
        want += b
        if b == 0 or want <= free:
            tokens, blocks = tokens + n, blocks + b
    return tokens, blocks


def work(case):
    if case["op"] == "tables":
        tokens, blocks = _grants(case)
        B, T = case["batch"], case["tokens"] + case["spare"]
        return {"bytes": 4 * (2 * B + 4 + 2 * B + 1 + 3 * T + 2 * blocks + min(B, tokens)), "flops": 8 * T}
    e = SIZES[case["dtype"]]
    c = SIZES["e4m3"] if case["cache"] == "e4m3" else e
    H, KV, D = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "norm_rope":
        T = case["tokens"]
        kept = T - 3 if T >= 8 else T
        weights = (H + KV if case["per_head"] else 2) * D * (4 if case["weights"] == "f32" else e)
        moved = T * (2 * H * D * e) + kept * 2 * KV * D * (e + c) + T * 4 * (2 + case["axes"]) + weights
        return {"bytes": moved, "flops": T * (H + KV) * (4 * D + case["rot"] * 3)}
    window, sinks, bs = case["window"], case["sinks"], case["block"]
    if case["op"] == "window_decode":
        ctx = _contexts(case)
        pairs = keys = sum(min(x, window) + min(sinks, max(0, x - window)) for x in ctx)
        rows, lists = case["batch"], len(ctx)
    else:
        new, held = _chunks(case), _held(case)
        pairs = keys = 0
        for n, h in zip(new, held):
            p = np.arange(h, h + n)
            pairs += int((np.minimum(p + 1, window) + np.minimum(sinks, np.maximum(0, p + 1 - window))).sum())
            lo = max(0, h + 1 - window)
            keys += h + n - lo + min(sinks, lo)
        rows, lists = case["tokens"], 2 * len(new) + 1
    return {"bytes": 2 * keys * KV * D * c + 2 * rows * H * D * e + 4 * (keys // bs + lists), "flops": 4 * pairs * H * D}


def _exact_tables(case, s):
    """Request by request, as a queue and lists would have it."""
    bs, T = s["bs"], s["T"]
    tables, held, asked = s["tables"].cpu().numpy().copy(), s["held"].tolist(), s["asked"].tolist()
    head, free = s["state"].tolist()
    ring = s["queue"].tolist()
    start, slots, positions, seqs = [0], [], [], []
    ctx = list(held)
    want = taken = brought = 0
    for r, (h, n) in enumerate(zip(held, asked)):
        have, upto = -(-h // bs), -(-(h + n) // bs)
        want += upto - have
        brought += n
        if n > 0 and upto <= tables.shape[1] and brought <= T and (upto == have or want <= free):
            for b in range(have, upto):
                tables[r, b] = ring[(head + taken) % len(ring)]
                taken += 1
            p = np.arange(h, h + n)
            slots.append(tables[r, p // bs].astype(np.int64) * bs + p % bs)
            positions.append(p)
            seqs.append(np.full(n, r))
            ctx[r] += n
        start.append(start[-1] + (ctx[r] - h))
    fill = T - start[-1]

    def column(parts, rest):
        return _device(np.concatenate([*parts, np.full(fill, rest)]))

    return (_device(tables), _device(ctx), _device(start), column(slots, -1), column(positions, 0), column(seqs, -1),
            _device([(head + taken) % len(ring), free - taken]))


def _exact_norm_rope(case, s):
    T = case["tokens"]
    n = case["rot"] // 2
    pos = s["positions"].double()
    cos, sin = (torch.empty((T, 1, n), dtype=torch.float64, device="cuda") for _ in range(2))
    for i, axis in enumerate(_axis_of(case)):
        angle = pos[axis] * float(s["inv_freq"][i])
        cos[:, 0, i], sin[:, 0, i] = torch.cos(angle), torch.sin(angle)

    def turn(x, w):
        x = x.double()
        x = x / torch.sqrt(torch.mean(x ** 2, -1, keepdim=True) + EPS) * w.double()
        y = x.clone()
        lo = slice(0, 2 * n, 2) if case["interleaved"] else slice(0, n)
        hi = slice(1, 2 * n, 2) if case["interleaved"] else slice(n, 2 * n)
        a, b = x[..., lo], x[..., hi]
        y[..., lo] = cos * a - sin * b
        y[..., hi] = sin * a + cos * b
        return y

    live = s["ids"] >= 0
    q = turn(s["q"], s["qw"]) * live[:, None, None]
    ks, vs = (NORM_K_SCALE, V_SCALE) if s["fp8"] else (1.0, 1.0)
    kc, vc = (torch.zeros(s["kc"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
    put = live & (s["slots"] >= 0)
    blk, off = s["slots"][put].long() // s["bs"], s["slots"][put].long() % s["bs"]
    top = 448.0 if s["fp8"] else math.inf
    kc[blk, :, off] = (turn(s["k"], s["kw"])[put] / ks).clamp(-top, top)
    vc[blk, :, off] = (s["v"][put].double() / vs).clamp(-top, top)
    return q, kc, vc


def _sequence(case, s, row, c):
    """K and V of a sequence's c tokens in 64 bits, [KV, c, D]; zeros where a block is not held."""
    blocks = s["tables"][row, :-(-c // case["block"])].long()

    def rows(cache, scale):
        x = cache.view(torch.uint8)[blocks].view(E4M3).float().double() * scale if s["fp8"] else cache[blocks].double()
        return (x * (blocks >= 0)[:, None, None, None]).transpose(0, 1).flatten(1, 2)[:, :c]

    return rows(s["kc"], K_SCALE), rows(s["vc"], V_SCALE)


def _exact_decode(case, s):
    """Sequence by sequence over its whole table, what is out of sight masked."""
    B, H, D = s["q"].shape
    KV = case["kv_heads"]
    out = torch.zeros((B, H, D), dtype=torch.float64, device="cuda")
    for b, c in enumerate(s["ctx"].tolist()):
        if c == 0:
            continue
        k, v = _sequence(case, s, b, c)
        j = torch.arange(c, device="cuda")
        hidden = (j < c - case["window"]) & (j >= case["sinks"])
        x = (s["q"][b].double().view(KV, H // KV, D) @ k.mT * s["scale"]).masked_fill(hidden, -torch.inf)
        out[b] = (torch.softmax(x, -1) @ v).view(H, D)
    return out


def _exact_prefill(case, s, step=512):
    """Chunks of queries against the keys from the first that any of them sees, and the first tokens, head group by group."""
    H, D = case["heads"], case["dim"]
    KV, W, sinks = case["kv_heads"], case["window"], case["sinks"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, h) in enumerate(zip(_chunks(case), _held(case))):
        k, v = _sequence(case, s, b, h + n)
        for t0 in range(0, n, step):
            t1 = min(n, t0 + step)
            p = torch.arange(h + t0, h + t1, device="cuda")[:, None]
            j = torch.arange(h + t1, device="cuda")
            j = j[(j < sinks) | (j > h + t0 - W)]
            hidden = (j > p) | ((j <= p - W) & (j >= sinks))
            q = s["q"][at + t0:at + t1].double().view(t1 - t0, KV, H // KV, D)
            for g in range(KV):
                x = (torch.einsum("tgd,jd->gtj", q[:, g], k[g, j]) * s["scale"]).masked_fill_(hidden, -torch.inf)
                out[at + t0:at + t1, g * (H // KV):(g + 1) * (H // KV)] = torch.einsum("gtj,jd->tgd", torch.softmax(x, -1), v[g, j])
        at += n
    return out


def exact(case, seed):
    return {"tables": _exact_tables, "norm_rope": _exact_norm_rope, "window_decode": _exact_decode,
            "window_prefill": _exact_prefill}[case["op"]](case, prepare(case, seed))
