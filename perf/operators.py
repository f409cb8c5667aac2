"""Cases of the serving operators around the paged cache: plain torch forms, the library's calls, and 64-bit results.

Two operators, which one layer of a decode step calls one after the other:

- rope: rotate the new tokens' q and K rows by their positions (one position a token, or one on each of several axes
  for image and video tokens) and write K and V into the paged cache at their slots;
- prefix: attention of one query token a sequence over a paged cache in which groups of sequences share the blocks of
  a long prefix, each group's prefix read once for all its members.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}
E4M3 = torch.float8_e4m3fn
# Cached codes are N(0, 56^2) (K) and N(0, 44^2) (V) draws, as in the library's E4M3 workloads.
K_SCALE, V_SCALE = 1.0 / 56.0, 1.0 / 44.0


def _rope(name, tokens, heads, kv_heads, dim, rot, dtype, cache="same", interleaved=False, axes=1, packed=True, block=16, far=4096):
    return {"name": name, "op": "rope", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim, "rot": rot,
            "dtype": dtype, "cache": cache, "interleaved": interleaved, "axes": axes, "packed": packed, "block": block, "far": far}


def _prefix(name, batch, groups, heads, kv_heads, dim, dtype, prefix, suffix, cache="same", block=16, ragged=False, short=0):
    return {"name": name, "op": "prefix", "batch": batch, "groups": groups, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "dtype": dtype, "cache": cache, "prefix": prefix, "suffix": suffix, "block": block, "ragged": ragged, "short": short}


def listed():
    return [
        # One request decoding alone: the call's latency is all there is.
        _rope("rope_one_token", 1, 32, 8, 128, 128, "bf16"),
        # A decode step of a full batch at far positions, rows taken out of the packed projection.
        _rope("rope_decode_256", 256, 32, 8, 128, 128, "bf16", far=131072, block=32),
        # One token budget of chunked prefill (16,384 new tokens), rows out of the packed projection.
        _rope("rope_chunk_16384", 16384, 32, 8, 128, 128, "bf16", far=32768),
        # A chunk quantized into an E4M3 cache on the way, neighbouring elements paired.
        _rope("rope_e4m3", 1023, 20, 4, 128, 128, "bf16", cache="e4m3", interleaved=True),
        # Image and video tokens: positions on three axes (time, height, width), part of each head rotated.
        _rope("rope_three_axes", 4099, 16, 2, 128, 96, "f16", axes=3, packed=False),
        # Heads whose rotated part is no multiple of the vector width, in fp32.
        _rope("rope_odd_heads", 1031, 12, 12, 80, 20, "f32", interleaved=True, packed=False, block=8),
        # A handful of requests behind a short system prompt: the smallest call.
        _prefix("prefix_small", 4, 1, 8, 2, 64, "f16", 256, 48),
        # The batch-32 decode layer with a common 4,096-token prompt.
        _prefix("prefix_b32", 32, 1, 32, 8, 128, "bf16", 4096, 256),
        # The mixed batch of 64 in groups of 8, each with its own 2,048-token prefix, long and short tails; a few
        # sequences end inside the prefix.
        _prefix("prefix_groups_of_8", 64, 8, 32, 8, 128, "f16", 2048, 14336, short=5),
        # Uneven groups and prefixes, 8 query heads a KV head, 64 dims, blocks of 48 tokens.
        _prefix("prefix_ragged", 37, 5, 32, 4, 64, "bf16", 5000, 777, block=48, ragged=True, short=2),
        # An E4M3 cache under a long document that every request asks about.
        _prefix("prefix_e4m3", 48, 1, 32, 8, 128, "bf16", 16384, 512, cache="e4m3", block=32),
        # A wide batch over a 32,768-token prefix: the largest call, bound by the matrix products.
        _prefix("prefix_wide", 256, 1, 32, 8, 128, "bf16", 32768, 512),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, even over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    if rng.random() < 0.5:
        dim, rot = rng.choice([(64, 64), (64, 32), (80, 20), (96, 96), (128, 128), (128, 64), (128, 96), (256, 64)])
        kv = rng.choice([1, 2, 3, 4, 8])
        cache = rng.choice(["same", "same", "same", "e4m3"])
        case = _rope("", _spread(rng, 1, 16384), kv * rng.choice([1, 2, 3, 4]), kv, dim, rot, rng.choice(["bf16", "bf16", "f16", "f32"]),
                     cache, rng.random() < 0.4, rng.choice([1, 1, 2, 3]), rng.random() < 0.6, rng.choice([8, 16, 32, 48]),
                     _spread(rng, 64, 1000000))
        if cache == "e4m3":
            case["tokens"] = min(case["tokens"], 2_500_000 // (kv * dim))
    else:
        dim = rng.choice([64, 128, 128])
        kv = rng.choice([1, 2, 4, 8])
        heads = kv * rng.choice([1, 2, 4, 8])
        batch = _spread(rng, 1, 256)
        prefix = _spread(rng, 16, 65536)
        suffix = _spread(rng, 1, 4096)
        while batch * heads * dim * prefix > 256 * 32 * 128 * 32768:
            prefix //= 2
        while batch * kv * dim * suffix > 256 * 8 * 128 * 512:
            suffix //= 2
        case = _prefix("", batch, rng.randint(1, min(batch, 12)), heads, kv, dim, rng.choice(["f16", "bf16"]), prefix, max(1, suffix),
                       "same" if dim == 64 else rng.choice(["same", "same", "e4m3"]), rng.choice([16, 16, 32, 48, 64, 128]),
                       rng.random() < 0.5, rng.choice([0, 0, 1, 3]))
        while case["groups"] > 1 and case["groups"] * prefix * kv * dim > 1 << 28:
            case["groups"] -= 1
        case["short"] = min(case["short"], batch - 1)
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


def _axis_of(case):
    """Axis of each frequency: sections as even as they come, the first ones longer."""
    n, a = case["rot"] // 2, case["axes"]
    return [min(i * a // n, a - 1) for i in range(n)]


def _prepare_rope(case, seed):
    g = _generator(seed)
    T, H, KV, D, bs = case["tokens"], case["heads"], case["kv_heads"], case["dim"], case["block"]
    dt = DTYPES[case["dtype"]]
    fp8 = case["cache"] == "e4m3"
    if case["packed"]:  # slices of the fused projection's output
        qkv = _normal(g, (T, H + 2 * KV, D), dt)
        q, k, v = qkv[:, :H], qkv[:, H:H + KV], qkv[:, H + KV:]
    else:
        q, k, v = (_normal(g, (T, n, D), dt) for n in (H, KV, KV))
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
    s = {"q": q, "k": k, "v": v, "slots": slots, "ids": ids, "positions": positions, "inv_freq": inv_freq.cuda(),
         "axis": torch.tensor(_axis_of(case), device="cuda"), "interleaved": case["interleaved"], "kc": kc, "vc": vc, "bs": bs,
         "fp8": fp8, "q_out": torch.zeros((T, H, D), dtype=dt, device="cuda"),
         "written": ((slots >= 0) & (ids >= 0)).nonzero()[:, 0], "rotated": (ids >= 0).nonzero()[:, 0]}
    if own:
        import paged_kv_cache_slots_gb300 as pkv

        s["pool"] = pkv.KVPool(1, NB, bs, KV, D, cache_dt, device="cuda", buffer=buffer)
        s["rope"] = pkv.Rope(inv_freq, interleaved=case["interleaved"], axes=_axis_of(case))
    return s


def _group_starts(case):
    return [g * case["batch"] // case["groups"] for g in range(case["groups"] + 1)]


def _prefix_lens(case):
    bs = case["block"]
    return [(case["prefix"] * (g + 1) // case["groups"] if case["ragged"] else case["prefix"]) // bs * bs for g in range(case["groups"])]


def _suffix_lens(case):
    """Tails of 1 to `suffix` tokens, evenly spread (before they are shuffled)."""
    n, b = case["suffix"], case["batch"]
    return [1 + i * (n - 1) // max(1, b - 1) for i in range(b)]


def _prepare_prefix(case, seed):
    g = _generator(seed)
    B, H, KV, D, bs = case["batch"], case["heads"], case["kv_heads"], case["dim"], case["block"]
    dt = DTYPES[case["dtype"]]
    fp8 = case["cache"] == "e4m3"
    starts, plens = _group_starts(case), _prefix_lens(case)
    group = [i for i in range(case["groups"]) for _ in range(starts[i], starts[i + 1])]
    order = torch.randperm(B, generator=g, device="cuda").tolist()
    tails = _suffix_lens(case)
    ctx = [plens[group[s]] + tails[order[s]] for s in range(B)]
    for i in range(case["short"]):  # sequences that end inside their group's prefix, the first of them empty
        s = order[i]
        ctx[s] = plens[group[s]] * i // case["short"]
    mb = max(1, max(-(-c // bs) for c in ctx), max(p // bs for p in plens))
    shared = [p // bs for p in plens]
    private = [max(0, -(-ctx[s] // bs) - shared[group[s]]) for s in range(B)]
    NB = (sum(shared) + sum(private)) * 9 // 8 + 1
    perm = torch.randperm(NB, generator=g, device="cuda", dtype=torch.int32).cpu()
    tables = torch.full((B, mb), -1, dtype=torch.int32)
    at, own_blocks = 0, []
    for n in shared:
        own_blocks.append(perm[at:at + n])
        at += n
    for s in range(B):
        n = shared[group[s]]
        tables[s, :n] = own_blocks[group[s]]
        tables[s, n:n + private[s]] = perm[at:at + private[s]]
        at += private[s]
    shape = (NB, KV, bs, D)
    kc = _codes(g, shape, 56.0) if fp8 else _normal(g, shape, dt)
    vc = _codes(g, shape, 44.0) if fp8 else _normal(g, shape, dt)
    s = {"q": _normal(g, (B, H, D), dt), "kc": kc, "vc": vc, "tables": tables.cuda(), "ctx": torch.tensor(ctx, dtype=torch.int32, device="cuda"),
         "starts": torch.tensor(starts, dtype=torch.int32, device="cuda"), "plens": torch.tensor(plens, dtype=torch.int32, device="cuda"),
         "scale": 1.0 / math.sqrt(D), "fp8": fp8, "group": torch.tensor(group, device="cuda"),
         "longest_prefix": max(plens), "longest_tail": max(max(tails), 1), "out": torch.empty((B, H, D), dtype=dt, device="cuda")}
    if own:
        import paged_kv_cache_slots_gb300 as pkv

        s["workspace"] = pkv.make_shared_prefix_workspace(B, case["groups"], H, KV, D, device="cuda")
    return s


def prepare(case, seed):
    return (_prepare_rope if case["op"] == "rope" else _prepare_prefix)(case, seed)


# ------------------------------------------------------------- plain forms


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


def _plain_rope(s):
    angle = s["positions"][s["axis"]].t().double() * s["inv_freq"]  # far positions need more than 32 bits
    cos, sin = angle.cos().float(), angle.sin().float()
    q = _rotate(s["q"].float(), cos, sin, s["interleaved"]).to(s["q_out"].dtype)
    s["q_out"][s["rotated"]] = q[s["rotated"]]
    w = s["written"]
    k = _rotate(s["k"].float(), cos, sin, s["interleaved"])[w]
    v = s["v"].float()[w]
    at = s["slots"][w].long()
    kc, vc = s["kc"], s["vc"]
    if s["fp8"]:
        k = (k / K_SCALE).clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)
        v = (v / V_SCALE).clamp(-448.0, 448.0).to(E4M3).view(torch.uint8)
        kc, vc = kc.view(torch.uint8), vc.view(torch.uint8)
    kc[at // s["bs"], :, at % s["bs"]] = k.to(kc.dtype)
    vc[at // s["bs"], :, at % s["bs"]] = v.to(vc.dtype)
    return s["q_out"], s["kc"], s["vc"]


def _rows(cache, tables, first, count, scale):
    """Rows first .. first + count - 1 (per table row) of a paged cache in fp32, [n, KV, count, D]; what lies past a table is any row."""
    bs = cache.shape[2]
    pos = first[:, None] + torch.arange(count, device=cache.device)
    blk = tables.gather(1, (pos // bs).clamp(max=tables.shape[1] - 1)).clamp(min=0).long()
    fp8 = cache.dtype == E4M3
    x = (cache.view(torch.uint8) if fp8 else cache)[blk, :, pos % bs]  # [n, count, KV, D]
    x = x.contiguous().view(E4M3).float() * scale if fp8 else x.float()
    return x.transpose(1, 2)


def _plain_prefix(s):
    B, H, D = s["q"].shape
    KV = s["kc"].shape[1]
    G = H // KV
    ks, vs = (K_SCALE, V_SCALE) if s["fp8"] else (1.0, 1.0)
    plens, group, starts = s["plens"].long(), s["group"], s["starts"].long()
    L, S, n = s["longest_prefix"], s["longest_tail"], s["plens"].shape[0]
    ctx = s["ctx"].long()
    plen = plens[group]
    q = s["q"].float().view(B, KV, G, D) * s["scale"]
    # The prefixes: each group's rows taken once, through the table of the member with the longest context.
    best = torch.zeros(n, dtype=torch.long, device=q.device).scatter_reduce(0, group, ctx * B + torch.arange(B, device=q.device), "amax")
    first = torch.zeros(n, dtype=torch.long, device=q.device)
    tables = s["tables"][best % B]
    kp, vp = _rows(s["kc"], tables, first, max(L, 1), ks), _rows(s["vc"], tables, first, max(L, 1), vs)
    rank = torch.arange(B, device=q.device) - starts[group]
    width = -(-B // n)
    qg = torch.zeros((n, KV, width, G, D), device=q.device)
    qg[group, :, rank] = q
    sp = (qg.flatten(2, 3) @ kp.transpose(-1, -2)).view(n, KV, width, G, -1)  # [n, KV, members, G, L]
    limit = torch.zeros((n, width), dtype=torch.long, device=q.device)
    limit[group, rank] = torch.minimum(plen, ctx)
    sp.masked_fill_(torch.arange(max(L, 1), device=q.device) >= limit[:, None, :, None, None], -torch.inf)
    # The tails.
    kt, vt = _rows(s["kc"], s["tables"], plen, S, ks), _rows(s["vc"], s["tables"], plen, S, vs)
    st = q @ kt.transpose(-1, -2)  # [B, KV, G, S]
    st.masked_fill_((plen[:, None] + torch.arange(S, device=q.device) >= ctx[:, None])[:, None, None], -torch.inf)
    # One softmax over both.
    top = torch.maximum(sp.amax(-1)[group, :, rank], st.amax(-1))
    top = torch.where(top == -torch.inf, torch.zeros_like(top), top)[..., None]
    grid = torch.zeros((n, KV, width, G, 1), device=q.device)
    grid[group, :, rank] = top
    ep = (sp - grid).exp_()
    et = (st - top).exp_()
    num = (ep.flatten(2, 3) @ vp).view(n, KV, width, G, D)[group, :, rank] + et @ vt
    den = ep.sum(-1, keepdim=True)[group, :, rank] + et.sum(-1, keepdim=True)
    return (num / torch.where(den == 0, torch.ones_like(den), den)).view(B, H, D).to(s["q"].dtype)


def run(state):
    s = state
    if "rope" in s or "positions" in s:
        if not own:
            return _plain_rope(s)
        scales = {"k_scale": K_SCALE, "v_scale": V_SCALE} if s["fp8"] else {}
        s["pool"].append_rope(0, s["k"], s["v"], s["slots"], s["positions"], s["rope"], q=s["q"], q_out=s["q_out"], seq_ids=s["ids"], **scales)
        return s["q_out"], s["kc"], s["vc"]
    if not own:
        return _plain_prefix(s)
    import paged_kv_cache_slots_gb300 as pkv

    scales = {"k_scale": K_SCALE, "v_scale": V_SCALE} if s["fp8"] else {}
    return pkv.paged_shared_prefix_attention(s["q"], s["kc"], s["vc"], s["tables"], s["ctx"], s["starts"], s["plens"], s["scale"],
                                             out=s["out"], workspace=s["workspace"], **scales)


# ----------------------------------------------------------- work and exact


def work(case):
    e = SIZES[case["dtype"]]
    c = SIZES["e4m3"] if case["cache"] == "e4m3" else e
    H, KV, D = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rope":
        T = case["tokens"]
        kept = T - 3 if T >= 8 else T
        moved = T * (2 * H * D * e) + kept * 2 * KV * D * (e + c) + T * 4 * (2 + case["axes"])
        return {"bytes": moved, "flops": T * (H + KV) * case["rot"] * 3}
    starts, plens, B = _group_starts(case), _prefix_lens(case), case["batch"]
    tails = sorted(_suffix_lens(case))
    tail = sum(tails[case["short"]:])
    sizes = [starts[g + 1] - starts[g] for g in range(case["groups"])]
    keys = sum(plens) + tail
    pairs = sum(n * p for n, p in zip(sizes, plens)) + tail
    return {"bytes": 2 * keys * KV * D * c + 2 * B * H * D * e + 4 * (keys // case["block"] + 2 * B), "flops": 4 * pairs * H * D}


def _exact_rope(case, s):
    T = case["tokens"]
    n = case["rot"] // 2
    pos = s["positions"].double()
    cos, sin = (torch.empty((T, 1, n), dtype=torch.float64, device="cuda") for _ in range(2))
    for i, axis in enumerate(_axis_of(case)):
        angle = pos[axis] * float(s["inv_freq"][i])
        cos[:, 0, i], sin[:, 0, i] = torch.cos(angle), torch.sin(angle)

    def turn(x):
        y = x.double().clone()
        lo = slice(0, 2 * n, 2) if case["interleaved"] else slice(0, n)
        hi = slice(1, 2 * n, 2) if case["interleaved"] else slice(n, 2 * n)
        a, b = x[..., lo].double(), x[..., hi].double()
        y[..., lo] = cos * a - sin * b
        y[..., hi] = sin * a + cos * b
        return y

    live = s["ids"] >= 0
    q = turn(s["q"]) * live[:, None, None]
    ks, vs = (K_SCALE, V_SCALE) if s["fp8"] else (1.0, 1.0)
    kc, vc = (torch.zeros(s["kc"].shape, dtype=torch.float64, device="cuda") for _ in range(2))
    put = live & (s["slots"] >= 0)
    blk, off = s["slots"][put].long() // s["bs"], s["slots"][put].long() % s["bs"]
    top = 448.0 if s["fp8"] else math.inf
    kc[blk, :, off] = (turn(s["k"])[put] / ks).clamp(-top, top)
    vc[blk, :, off] = (s["v"][put].double() / vs).clamp(-top, top)
    return q, kc, vc


def _exact_prefix(case, s):
    """Sequence by sequence over its own whole table: nothing shared."""
    B, H, D = s["q"].shape
    KV, bs = s["kc"].shape[1], s["kc"].shape[2]
    out = torch.zeros((B, H, D), dtype=torch.float64, device="cuda")
    for b, c in enumerate(s["ctx"].tolist()):
        if c == 0:
            continue
        blocks = s["tables"][b, :-(-c // bs)].long()

        def rows(cache, scale):
            x = cache.view(torch.uint8)[blocks].view(E4M3).float().double() * scale if s["fp8"] else cache[blocks].double()
            return x.transpose(0, 1).flatten(1, 2)[:, :c]  # [KV, c, D]

        q = s["q"][b].double().view(KV, H // KV, D)
        p = torch.softmax(q @ rows(s["kc"], K_SCALE if s["fp8"] else 1.0).mT * s["scale"], -1)
        out[b] = (p @ rows(s["vc"], V_SCALE if s["fp8"] else 1.0)).view(H, D)
    return out


def exact(case, seed):
    return (_exact_rope if case["op"] == "rope" else _exact_prefix)(case, prepare(case, seed))
