"""What is measured of the 8-bit paged cache's operators: rotary positions, the
write of new keys and values into a cache of 8-bit floating point (e4m3) with a
scale for each block of tokens and head, reading it back, and the attention of
each request's new tokens over it.

A layer of a serving step with these operators: the projections give queries,
keys and values of the step's new tokens; `rotary` turns the queries by their
positions; `append` turns the keys, quantises both and stores them; `attention`
reads the cache; `gather` hands a stored context to whoever needs it in 16 bits.

Lengths of a case are fixed quantiles of its range in an order that the seed
shuffles, so a case costs the same for every seed.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
E4M3 = torch.float8_e4m3fn
TOP = 448.0  # the largest e4m3 number


def listed():
    return [
        # a decoding step's queries and keys (32 + 8 heads in one tensor): latency
        {"name": "rotate step", "op": "rotary", "tokens": 64, "heads": 40, "D": 128, "rot": 128,
         "pairs": "half", "scaling": "none", "far": 131071, "dtype": "bf16"},
        # prompts' queries and keys, half of each head turned, positions stretched for long contexts
        {"name": "rotate prompts", "op": "rotary", "tokens": 30001, "heads": 40, "D": 128,
         "rot": 64, "pairs": "inter", "scaling": "yarn", "far": 131071, "dtype": "fp16"},
        # the verification step of the headline batch: up to 17 new tokens of 256 requests, which
        # mostly continue a block that holds earlier tokens; keys turned on the way
        {"name": "append step", "op": "append", "B": 256, "new": 17, "Hkv": 8, "D": 128,
         "page": 16, "block": 16, "rot": 128, "pairs": "half", "dtype": "bf16",
         "layout": "token"},
        # prompts enter the cache, heads before tokens inside a page
        {"name": "append prompts", "op": "append", "B": 50, "new": 4000, "Hkv": 8, "D": 128,
         "page": 64, "block": 64, "rot": 0, "pairs": "half", "dtype": "fp16", "layout": "head"},
        # one key head per query head, a scale for every token, part of the head turned
        {"name": "append tokens", "op": "append", "B": 45, "new": 901, "Hkv": 24, "D": 64,
         "page": 32, "block": 1, "rot": 32, "pairs": "inter", "dtype": "bf16",
         "layout": "token"},
        # one request's context read back
        {"name": "gather one", "op": "gather", "B": 1, "new": 1001, "Hkv": 8, "D": 128,
         "page": 16, "block": 16, "dtype": "bf16", "layout": "token"},
        # many contexts read back (moved to another engine)
        {"name": "gather contexts", "op": "gather", "B": 50, "new": 4001, "Hkv": 8, "D": 128,
         "page": 64, "block": 32, "dtype": "fp16", "layout": "head"},
        # one user, one new token, a short context: latency
        {"name": "attend one", "op": "attention", "B": 1, "Hq": 32, "Hkv": 8, "D": 128,
         "page": 16, "block": 16, "lo": 1000, "hi": 1000, "new": 1, "window": 0,
         "dtype": "bf16", "layout": "token"},
        # plain decoding of a mid-sized batch: one new token each, ragged contexts
        {"name": "attend decode 64", "op": "attention", "B": 64, "Hq": 64, "Hkv": 8, "D": 128,
         "page": 64, "block": 64, "lo": 1, "hi": 8191, "new": 1, "window": 0, "dtype": "fp16",
         "layout": "head"},
        # the target's verification forward of the headline batch: up to 1 + 16 new tokens each
        {"name": "attend verify 256", "op": "attention", "B": 256, "Hq": 32, "Hkv": 8, "D": 128,
         "page": 16, "block": 16, "lo": 33, "hi": 4096, "new": 17, "window": 0, "dtype": "bf16",
         "layout": "token"},
        # few users with very long contexts, short draft blocks
        {"name": "attend long", "op": "attention", "B": 3, "Hq": 64, "Hkv": 8, "D": 128,
         "page": 128, "block": 32, "lo": 100001, "hi": 131071, "new": 6, "window": 0,
         "dtype": "bf16", "layout": "token"},
        # a sliding-window layer with one key head per query head, a scale for every token
        {"name": "attend window", "op": "attention", "B": 45, "Hq": 24, "Hkv": 24, "D": 64,
         "page": 32, "block": 1, "lo": 9, "hi": 12000, "new": 9, "window": 1023,
         "dtype": "fp16", "layout": "token"},
    ]


def _log(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "append", "append", "gather", "attention", "attention",
                     "attention"])
    D = rng.choice([64, 128])
    dtype, pairs = rng.choice(["bf16", "fp16"]), rng.choice(["half", "inter"])
    rot = rng.choice([D, D // 2, D // 4, 48])
    if op == "rotary":
        return {"op": op, "tokens": _log(rng, 1, 30001), "heads": rng.choice([1, 6, 12, 40]),
                "D": D, "rot": rot, "pairs": pairs,
                "scaling": rng.choice(["none", "linear", "ntk", "yarn"]),
                "far": _log(rng, 100, 1000000), "dtype": dtype}
    page = rng.choice([8, 16, 32, 64, 128])
    kind = {"page": page, "block": min(page, rng.choice([1, 2, 4, 8, 16, 16, 32, 64, 128])),
            "D": D, "dtype": dtype, "layout": rng.choice(["token", "head"])}
    if op in ("append", "gather"):
        new = rng.choice([1, 5, 17, _log(rng, 18, 4000)])
        c = {"op": op, "B": _log(rng, 1, min(500, 100000 // new)), "new": new,
             "Hkv": rng.choice([1, 2, 4, 5, 8]), **kind}
        if op == "append":
            c.update(rot=rng.choice([0, rot]), pairs=pairs)
        return c
    Hkv = rng.choice([1, 2, 4, 8, 7])
    group = rng.choice([1, 2, 4, 8, 16, 3])
    new = rng.choice([1, 1, 2, 5, 8, 17])
    if group * Hkv > 64:
        group = 64 // Hkv
    hi = _log(rng, max(20, new), 131071)
    # tokens of cache in all: at most what the listed cases have, per key head
    B = _log(rng, 1, max(1, min(256, 300000 // hi)))
    return {"op": op, "B": B, "Hq": group * Hkv, "Hkv": Hkv, "lo": rng.choice([new, hi]),
            "hi": hi, "new": new, "window": rng.choice([0, 0, 0, 1 + hi // 3]), **kind}


def _spread(lo, hi, n):
    """n whole numbers that cover lo..hi evenly."""
    return np.round(np.linspace(lo, hi, n) if n > 1 else np.array([float(hi)])).astype(np.int64)


def _up(a, b):
    return -(-a // b)


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _i32(a):
    return torch.as_tensor(np.ascontiguousarray(a), dtype=torch.int32).cuda()


def _tables(case):
    """Angle per position of every pair, in 64 bits, and the gain of sine and cosine."""
    rot, base, factor, first = case["rot"], 10000.0, 32.0, 4096.0
    kind = case.get("scaling", "none")
    if kind == "ntk":
        base *= factor ** (rot / (rot - 2))
    f = base ** (-2.0 * np.arange(rot // 2) / rot)
    gain = 1.0
    if kind == "linear":
        f = f / factor
    if kind == "yarn":  # pairs that turn often in the first length keep their angle
        turns = first * f / (2 * math.pi)
        keep = np.clip((turns - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        f = keep * f + (1 - keep) * f / factor
        gain = 0.1 * math.log(factor) + 1.0
    return torch.as_tensor(f).cuda(), gain


def _own_table(case):
    from speculative_decoding_verification_41_gb300 import paged_q8
    return paged_q8.RotaryTable(case["rot"], interleaved=case["pairs"] == "inter",
                                scaling=case.get("scaling", "none"),
                                factor=32.0, original_len=4096, device="cuda")


def _paged(counts, width, pages, seed):
    """A block table whose row r names counts[r] of the pages, all different, in random order."""
    ids = torch.randperm(pages, generator=_gen(seed), device="cuda")
    j = torch.arange(width, device="cuda")
    n = torch.as_tensor(counts).cuda()
    at = (torch.cumsum(n, 0) - n)[:, None] + j[None, :]
    return torch.where(j[None, :] < n[:, None], ids[at.clamp(max=pages - 1)], 0).to(torch.int32)


def _cache(pages, case, seed):
    """Codes of the whole cache as [pages, page, heads, D] (with "head" the heads are stored
    before the tokens of a page), about what randn of a block's own size quantises to."""
    shape = [pages, case["page"], case["Hkv"], case["D"]]
    if case["layout"] == "head":
        shape[1], shape[2] = shape[2], shape[1]
    t = torch.randn(shape, generator=_gen(seed), device="cuda",
                    dtype=torch.float32 if math.prod(shape) < 1 << 20 else torch.bfloat16)
    t = t.mul_(90.0).clamp_(-TOP, TOP).to(E4M3)
    return t.transpose(1, 2) if case["layout"] == "head" else t


def _scales(pages, case, seed):
    """A power of two for each block and head."""
    e = torch.randint(-9, -6, (pages, case["page"] // case["block"], case["Hkv"]),
                      generator=_gen(seed), device="cuda")
    return torch.exp2(e.float())


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    s = {"case": case, "op": case["op"]}
    dt = DTYPES[case["dtype"]]
    if case["op"] == "rotary":
        n, H, D = case["tokens"], case["heads"], case["D"]
        # queries and keys of a projection that also makes values
        qkv = torch.randn(n, H + max(1, H // 5), D, generator=_gen(seed), device="cuda").to(dt)
        pos = torch.randint(0, case["far"] + 1, (n,), generator=_gen(seed + 1), device="cuda")
        f, gain = _tables(case)
        s.update(x=qkv[:, :H], positions=pos.to(torch.int32), freq=f, gain=gain,
                 out=torch.empty(n, H, D, dtype=dt, device="cuda"))
        if own:
            s["table"] = _own_table(case)
        return s
    ps, B = case["page"], case["B"]
    if case["op"] in ("append", "gather"):
        new = rng.permutation(_spread(1, case["new"], B))
        ctx = rng.permutation(_spread(0, 2 * ps - 1, B)) if case["op"] == "append" and B > 1 \
            else np.zeros(B, np.int64)
        counts = _up(ctx + new, ps)
        # as many pages whatever tokens the requests hold already
        pages = int(_up(_spread(1, case["new"], B) + 2 * ps, ps).sum()) + 1
        table = _paged(counts, int(counts.max()), pages, seed).cpu().numpy().astype(np.int64)
        req = np.repeat(np.arange(B), new)
        at = np.arange(len(req)) - np.repeat(np.cumsum(new) - new, new) + ctx[req]
        slots = table[req, at // ps] * ps + at % ps
        n = len(slots) + len(slots) // 16  # rows past the last token
        slots = np.concatenate([slots, np.full(n - len(slots), -1)])
        at = np.concatenate([at, np.full(n - len(at), -1)])
        row = [n, case["Hkv"], case["D"]]
        s.update(slot_map=_i32(slots), k_cache=_cache(pages, case, seed + 4),
                 v_cache=_cache(pages, case, seed + 5), k_scale=_scales(pages, case, seed + 6),
                 v_scale=_scales(pages, case, seed + 7))
        if case["op"] == "gather":
            s.update(k=torch.zeros(row, dtype=dt, device="cuda"),
                     v=torch.zeros(row, dtype=dt, device="cuda"))
        else:
            s.update(k=torch.randn(row, generator=_gen(seed + 2), device="cuda").to(dt),
                     v=torch.randn(row, generator=_gen(seed + 3), device="cuda").to(dt))
            if case["rot"]:
                s["positions"] = _i32(at)
                s["freq"], s["gain"] = _tables(case)
        if own:
            s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
            s["table"] = _own_table(case) if case.get("rot") else None
        return s
    new = rng.permutation(_spread(1, case["new"], B))
    ctx = np.maximum(rng.permutation(_spread(case["lo"], case["hi"], B)), new)
    counts = _up(ctx, ps)
    pages = int(counts.sum()) + 1 + seed % 7
    off = np.concatenate([[0], np.cumsum(new)])
    q = 2 * torch.randn(int(off[-1]), case["Hq"], case["D"], generator=_gen(seed + 2),
                        device="cuda")
    s.update(q=q.to(dt), k_cache=_cache(pages, case, seed + 4),
             v_cache=_cache(pages, case, seed + 5), k_scale=_scales(pages, case, seed + 6),
             v_scale=_scales(pages, case, seed + 7),
             table=_paged(counts, _up(case["hi"], ps), pages, seed), context_len=_i32(ctx),
             row_off=torch.as_tensor(off).cuda(), max_new=case["new"], window=case["window"],
             scale=case["D"] ** -0.5)
    if own:
        from speculative_decoding_verification_41_gb300 import paged
        s["buffers"] = paged.AttentionBuffers(int(off[-1]), case["Hq"], case["Hkv"],
                                              case["D"], case["new"], dt, "cuda", with_lse=True)
    return s


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    from speculative_decoding_verification_41_gb300 import paged_q8
    if s["op"] == "rotary":
        return [paged_q8.dspark_rotary(s["x"], s["positions"], s["table"], out=s["out"])["out"]]
    if s["op"] == "append":
        paged_q8.dspark_kv_append_q8(s["k"], s["v"], s["slot_map"], s["k_cache"], s["v_cache"],
                                     s["k_scale"], s["v_scale"], rotary=s["table"],
                                     positions=s.get("positions"), device_status=s["status"])
        return [s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]]
    if s["op"] == "gather":
        paged_q8.dspark_kv_gather_q8(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                     s["slot_map"], k=s["k"], v=s["v"],
                                     device_status=s["status"])
        return [s["k"], s["v"]]
    o = paged_q8.dspark_paged_attention_q8(
        s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
        s["context_len"], s["row_off"], scale=s["scale"], max_new=s["max_new"],
        window=s["window"], with_lse=True, buffers=s["buffers"])
    return [o["out"], o["lse"]]


def _run_plain(s):
    return {"rotary": _rotary, "append": _append, "gather": _gather,
            "attention": _attention}[s["op"]](s)


def _turned(x, positions, freq, gain, pairs):
    """x [n, heads, D] in 32 bits with its first 2 * len(freq) elements turned."""
    rot = 2 * freq.numel()
    angle = positions.double()[:, None] * freq[None, :]
    c, d = ((gain * f(angle)).float()[:, None, :] for f in (torch.cos, torch.sin))
    y = x.float()
    if pairs == "half":
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        return torch.cat([a * c - b * d, b * c + a * d, y[..., rot:]], -1)
    a, b = y[..., 0:rot:2], y[..., 1:rot:2]
    turned = torch.stack([a * c - b * d, b * c + a * d], -1).flatten(-2)
    return torch.cat([turned, y[..., rot:]], -1)


def _rotary(s):
    y = _turned(s["x"], s["positions"], s["freq"], s["gain"], s["case"]["pairs"])
    s["out"].copy_(y)
    return [s["out"]]


def _store(x, slot, cache, scale):
    """Rows x [n, heads, D] (32 bits) into the slots of one cache and its scales, in place."""
    ps, per = cache.shape[1], scale.shape[1]
    b = ps // per
    page, at = slot // ps, slot % ps
    which, place = torch.unique(slot // b, return_inverse=True)       # the blocks written to
    heads = x.shape[1]
    size = torch.where(x.isfinite(), x.abs(), 0.0).amax(-1)           # [n, heads]
    most = torch.zeros(which.numel(), heads, device=x.device)
    most.scatter_reduce_(0, place[:, None].expand(-1, heads), size, "amax")
    m, e = torch.frexp(most)                                          # most = m 2^e, m < 1
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126)          # 448 = 0.875 * 2^9
    need = torch.where(most > 0, torch.exp2(e.float()), 2.0 ** -126)
    first = torch.full((which.numel(),), b, device=x.device)
    first.scatter_reduce_(0, place, at % b, "amin")
    bp, bi = which // per, which % per
    old = scale[bp, bi]
    now = torch.where((first == 0)[:, None], need, torch.maximum(old, need))
    # the tokens that stay, in the blocks whose scale rises
    rises = (first > 0)[:, None] & (now > old)
    t = torch.arange(b, device=x.device)
    there = (bp[:, None], bi[:, None] * b + t[None, :])
    held = cache[there]                                               # [blocks, b, heads, D]
    again = (held.float() * (old / now)[:, None, :, None]).to(E4M3)
    cache[there] = torch.where(rises[:, None, :, None], again.float(), held.float()).to(E4M3)
    scale[bp, bi] = now
    cache[page, at] = (x / now[place][:, :, None]).to(E4M3)


def _append(s):
    t = torch.nonzero(s["slot_map"] >= 0).reshape(-1)
    slot = s["slot_map"][t].long()
    k = s["k"][t]
    k = _turned(k, s["positions"][t], s["freq"], s["gain"], s["case"]["pairs"]) \
        if s["case"]["rot"] else k.float()
    _store(k, slot, s["k_cache"], s["k_scale"])
    _store(s["v"][t].float(), slot, s["v_cache"], s["v_scale"])
    return [s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]]


def _gather(s):
    ps = s["k_cache"].shape[1]
    b = ps // s["k_scale"].shape[1]
    t = torch.nonzero(s["slot_map"] >= 0).reshape(-1)
    slot = s["slot_map"][t].long()
    page, at = slot // ps, slot % ps
    for out, cache, scale in ((s["k"], s["k_cache"], s["k_scale"]),
                              (s["v"], s["v_cache"], s["v_scale"])):
        out[t] = (cache[page, at].float() * scale[page, at // b][:, :, None]).to(out.dtype)
    return [s["k"], s["v"]]


def _held(cache, scale, table):
    """Keys or values of every request's pages in 32 bits: [B, heads, tokens, D]."""
    B, width = table.shape
    _, ps, heads, D = cache.shape
    x = cache[table].float().reshape(B, width, scale.shape[1], -1, heads, D)
    x = x * scale[table][:, :, :, None, :, None]
    return x.reshape(B, width * ps, heads, D).transpose(1, 2)


def _attention(s):
    q, off, ctx, T = s["q"], s["row_off"], s["context_len"].long(), s["max_new"]
    n, Hq, D = q.shape
    B, width = s["table"].shape
    Hkv, L = s["k_cache"].shape[2], width * s["k_cache"].shape[1]
    G = Hq // Hkv
    t = torch.arange(T, device=q.device)[None, :]
    new = (off[1:] - off[:-1])[:, None]
    row = (off[:-1, None] + t).clamp(max=n - 1)                            # [B, T]
    qp = q[row].float().reshape(B, T, Hkv, G, D).permute(0, 2, 3, 1, 4)    # [B, Hkv, G, T, D]
    table = s["table"].long()
    k = _held(s["k_cache"], s["k_scale"], table)
    z = torch.matmul(qp.reshape(B, Hkv, G * T, D), k.transpose(2, 3)) * s["scale"]
    del k
    z = z.reshape(B, Hkv, G, T, L)
    end = (ctx[:, None] - new + t + 1)[:, :, None]                         # [B, T, 1]
    u = torch.arange(L, device=q.device)[None, None, :]
    seen = (u < end) & ((u >= end - s["window"]) if s["window"] else (u >= 0))
    z.masked_fill_(~seen[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = z.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    v = _held(s["v_cache"], s["v_scale"], table)
    o = torch.matmul(p.reshape(B, Hkv, G * T, L), v).reshape(B, Hkv, G, T, D) / total
    lse = (m + total.log()).squeeze(-1)                                    # [B, Hkv, G, T]
    real = (t < new).reshape(-1).nonzero().reshape(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(B * T, Hq, D)[real]
    return [o.to(q.dtype), lse.permute(0, 3, 1, 2).reshape(B * T, Hq)[real]]


def _visible(case):
    """New tokens, cached tokens that some new token sees, and pairs, of a case."""
    new = _spread(1, case["new"], case["B"])
    ctx = np.maximum(_spread(case["lo"], case["hi"], case["B"]), new)
    w = case["window"] or 1 << 40
    span = np.minimum(ctx, w + new - 1).sum()
    pairs = sum(int(np.minimum(c - n + 1 + np.arange(n), w).sum()) for c, n in zip(ctx, new))
    return int(new.sum()), int(span), pairs


def work(case):
    if case["op"] == "rotary":
        n = case["tokens"]
        return {"bytes": n * (4 + 4 * case["heads"] * case["D"]),
                "flops": 3 * n * case["heads"] * case["rot"]}
    if case["op"] in ("append", "gather"):
        n = int(_spread(1, case["new"], case["B"]).sum())
        size = n * case["Hkv"] * case["D"]
        scales = 8 * case["Hkv"] * _up(n, case["block"])
        return {"bytes": 4 * n + 6 * size + scales,
                "flops": 2 * size + 3 * n * case["Hkv"] * case.get("rot", 0)}
    new, span, pairs = _visible(case)
    return {"bytes": 2 * span * case["Hkv"] * case["D"] + 8 * _up(span, case["block"]) * case["Hkv"]
            + 4 * new * case["Hq"] * case["D"] + 4 * new * case["Hq"],
            "flops": 4 * pairs * case["Hq"] * case["D"]}


def _rounded(x):
    """The e4m3 numbers next to x (64 bits, at most 448 in size), ties to even."""
    size = x.abs().clamp(min=2.0 ** -6)
    step = torch.exp2(torch.floor(torch.log2(size)) - 3)
    return torch.round(x / step) * step


def _rotation(case, positions):
    """The turned part of a head as matrices: [n, rot, rot] in 64 bits would be large, so cosine
    and sine of every element, its partner, and the partner's sign."""
    f, gain = _tables(case)
    rot = case["rot"]
    i = torch.arange(rot, device="cuda")
    if case["pairs"] == "half":
        j, partner, sign = i % (rot // 2), (i + rot // 2) % rot, torch.where(i < rot // 2, -1, 1)
    else:
        j, partner, sign = i // 2, i ^ 1, torch.where(i % 2 == 0, -1, 1)
    angle = positions.double()[:, None] * f[j][None, :]
    return gain * torch.cos(angle), gain * torch.sin(angle) * sign, partner


def _exact_turn(case, x, positions):
    c, d, partner = _rotation(case, positions)
    y = x.double().clone()
    head = y[..., :case["rot"]]
    y[..., :case["rot"]] = head * c[:, None] + head[..., partner] * d[:, None]
    return y


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        return [_exact_turn(case, s["x"], s["positions"])]
    ps = case["page"]
    if case["op"] in ("append", "gather"):
        b = case["block"]
        flat = s["slot_map"].cpu().numpy()
        rows = torch.as_tensor(np.flatnonzero(flat >= 0)).cuda()
        page, at = (torch.as_tensor(f(flat[flat >= 0].astype(np.int64), ps)).cuda()
                    for f in (np.floor_divide, np.remainder))
        codes, scales = [], []
        for x, cache, scale in ((s["k"], s["k_cache"], s["k_scale"]),
                                (s["v"], s["v_cache"], s["v_scale"])):
            pages = cache.shape[0]
            each = scale.double().repeat_interleave(b, 1)[..., None]   # [pages, page, heads, 1]
            if case["op"] == "gather":
                y = x.double()
                y.index_copy_(0, rows, (cache.double() * each)[page, at])
                codes.append(y)
                continue
            y = x.index_select(0, rows)
            y = _exact_turn(case, y, s["positions"].index_select(0, rows)) \
                if case["rot"] and x is s["k"] else y.double()
            # the whole cache, block by block: what is new, how large it is, what stays
            new = torch.zeros(pages, ps, dtype=torch.bool, device="cuda")
            new[page, at] = True
            size = torch.zeros(pages, ps, case["Hkv"], dtype=torch.float64, device="cuda")
            size[page, at] = y.abs().amax(-1)
            size = size.reshape(pages, -1, b, case["Hkv"]).amax(2)
            need = torch.exp2(torch.ceil(torch.log2(size / TOP)).clamp(min=-126))
            starts = new[:, ::b, None]
            touched = new.reshape(pages, -1, b).any(2)[..., None]
            kept = torch.maximum(scale.double(), need)
            now = torch.where(touched, torch.where(starts, need, kept), scale.double())
            code = cache.double()
            ratio = torch.where(starts, 1.0, scale.double() / now).repeat_interleave(b, 1)[..., None]
            code = _rounded(code * ratio)
            code[page, at] = _rounded(y / now.repeat_interleave(b, 1)[page, at][..., None])
            codes.append(code)
            scales.append(now)
        return codes + scales
    off, ctx = s["row_off"].tolist(), s["context_len"].tolist()
    table = s["table"].cpu()
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    o = torch.zeros(off[-1], Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((off[-1], Hq), -math.inf, dtype=torch.float64, device="cuda")
    for r, c in enumerate(ctx):
        ids = table[r, :_up(c, ps)].long().cuda()
        T = off[r + 1] - off[r]
        first = 0
        if case["window"]:  # nothing before the first new token's window is seen
            first = max(0, c - T + 1 - case["window"])
        k, v = ((cache.index_select(0, ids).double()
                 * scale.index_select(0, ids).double().repeat_interleave(case["block"], 1)[..., None]
                 ).flatten(0, 1)[first:c] for cache, scale in ((s["k_cache"], s["k_scale"]),
                                                               (s["v_cache"], s["v_scale"])))
        last = torch.arange(c - T, c, device="cuda")[:, None]
        u = torch.arange(first, c, device="cuda")[None, :]
        hidden = u > last
        if case["window"]:
            hidden |= u <= last - case["window"]
        for h in range(Hkv):
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            x = s["q"][off[r]:off[r + 1], heads].double().transpose(0, 1)   # [G, T, D]
            z = x @ k[:, h].T * s["scale"]
            z = z.masked_fill(hidden[None], -math.inf)
            top = torch.logsumexp(z, -1)
            lse[off[r]:off[r + 1], heads] = top.T
            o[off[r]:off[r + 1], heads] = (torch.exp(z - top[..., None]) @ v[:, h]).transpose(0, 1)
    return [o, lse]
