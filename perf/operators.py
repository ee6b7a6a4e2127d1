"""What is measured of the paged-cache operators: the page bookkeeping of a
speculative step (reserve, release), the write of new keys and values into the
cache, and the attention of each request's new tokens over its pages.

A serving step with these operators: the scheduler gives every request a
verify length l_r; `reserve` finds pages for its l_r + 1 new tokens; `append`
stores their keys and values; `attention` reads the cache for them; after the
verification `release` returns the pages of the rejected tokens.

Lengths of a case are fixed quantiles of its range in an order that the seed
shuffles, so a case costs the same for every seed.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


def listed():
    return [
        # one decoding step of a small batch: the smallest bookkeeping call (latency)
        {"name": "reserve step 64", "op": "reserve", "B": 64, "ctx": 4096, "new": 16, "page": 16},
        # a step of the largest batch of the benchmark's workloads, ragged
        {"name": "reserve step 1024", "op": "reserve", "B": 1024, "ctx": 8191, "new": 16,
         "page": 16},
        # prompts enter the cache: hundreds of requests with up to 4,000 tokens each
        {"name": "reserve prompts", "op": "reserve", "B": 500, "ctx": 777, "new": 4000,
         "page": 32},
        # roll back of rejected draft tokens after the headline workload's verification
        {"name": "release step 256", "op": "release", "B": 256, "ctx": 4096, "new": 16,
         "page": 16, "finish": 0},
        # many long requests end in one step (a batch job's tail, preemption)
        {"name": "release long", "op": "release", "B": 1024, "ctx": 32000, "new": 16, "page": 16,
         "finish": 3},
        # new keys and values of one verification step, odd token count
        {"name": "append step", "op": "append", "tokens": 2177, "Hkv": 8, "D": 128, "page": 16,
         "dtype": "bf16", "layout": "token"},
        # prompts' keys and values, heads before tokens inside a page
        {"name": "append prompts", "op": "append", "tokens": 100000, "Hkv": 8, "D": 128,
         "page": 64, "dtype": "fp16", "layout": "head"},
        # one user, one new token, a short context: latency
        {"name": "attend one", "op": "attention", "B": 1, "Hq": 32, "Hkv": 8, "D": 128,
         "page": 16, "lo": 1000, "hi": 1000, "new": 1, "window": 0, "dtype": "bf16",
         "layout": "token"},
        # plain decoding of a mid-sized batch: one new token each, ragged contexts
        {"name": "attend decode 64", "op": "attention", "B": 64, "Hq": 64, "Hkv": 8, "D": 128,
         "page": 64, "lo": 1, "hi": 8191, "new": 1, "window": 0, "dtype": "fp16",
         "layout": "head"},
        # the target's verification forward of the headline batch: up to 1 + 16 new tokens each
        {"name": "attend verify 256", "op": "attention", "B": 256, "Hq": 32, "Hkv": 8, "D": 128,
         "page": 16, "lo": 33, "hi": 4096, "new": 17, "window": 0, "dtype": "bf16",
         "layout": "token"},
        # few users with very long contexts, short draft blocks
        {"name": "attend long", "op": "attention", "B": 3, "Hq": 64, "Hkv": 8, "D": 128,
         "page": 128, "lo": 100001, "hi": 131071, "new": 6, "window": 0, "dtype": "bf16",
         "layout": "token"},
        # a sliding-window layer with one key head per query head
        {"name": "attend window", "op": "attention", "B": 45, "Hq": 24, "Hkv": 24, "D": 64,
         "page": 32, "lo": 9, "hi": 12000, "new": 9, "window": 1023, "dtype": "fp16",
         "layout": "token"},
    ]


def _log(rng, lo, hi):
    """A whole number of lo..hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["reserve", "release", "append", "attention", "attention", "attention"])
    page = rng.choice([8, 16, 32, 64, 128])
    if op in ("reserve", "release"):
        new = rng.choice([0, 4, 16, _log(rng, 1, 32), _log(rng, 33, 4000)])
        if op == "release":
            new = min(new, 32)
        B = _log(rng, 1, 1024 if new <= 32 else 500)
        c = {"op": op, "B": B, "ctx": _log(rng, 16, 32000 if op == "release" else 8191),
             "new": new, "page": max(page, 16)}
        if op == "release":
            c["finish"] = rng.choice([0, 3, 10])
        return c
    D = rng.choice([64, 128])
    kind = {"page": page, "D": D, "dtype": rng.choice(["bf16", "fp16"]),
            "layout": rng.choice(["token", "head"])}
    if op == "append":
        return {"op": op, "tokens": _log(rng, 1, 100000), "Hkv": rng.choice([1, 2, 4, 5, 8]),
                **kind}
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


def _paged(counts, width, pages, seed):
    """A block table whose row r names counts[r] of the pages, all different, in random order,
    and the ids that are left. The rest of a row is 0, as in a table that was allocated once."""
    total = int(counts.sum())
    ids = torch.randperm(pages, generator=_gen(seed), device="cuda")
    j = torch.arange(width, device="cuda")
    n = torch.as_tensor(counts).cuda()
    at = (torch.cumsum(n, 0) - n)[:, None] + j[None, :]
    table = torch.where(j[None, :] < n[:, None], ids[at.clamp(max=pages - 1)], 0)
    return table.to(torch.int32), ids[total:].to(torch.int32)


def _cache(pages, case, seed):
    """Keys or values of the whole cache as [pages, page, heads, D]; with "head" the heads are
    stored before the tokens of a page."""
    shape = [pages, case["page"], case["Hkv"], case["D"]]
    if case["layout"] == "head":
        shape[1], shape[2] = shape[2], shape[1]
    t = torch.randn(shape, generator=_gen(seed), device="cuda",
                    dtype=torch.float32 if math.prod(shape) < 1 << 20 else DTYPES[case["dtype"]])
    t = t.to(DTYPES[case["dtype"]])
    return t.transpose(1, 2) if case["layout"] == "head" else t


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    s = {"case": case, "op": case["op"], "page": case["page"]}
    if case["op"] in ("reserve", "release"):
        B, ps = case["B"], case["page"]
        ctx = rng.permutation(_spread(0, case["ctx"], B))
        new = rng.permutation(_spread(0, case["new"], B))
        after = case["op"] == "release"  # the step's tokens have their pages already
        have = _up(ctx + new + 1, ps) if after else _up(ctx, ps)
        width = _up(case["ctx"] + case["new"] + 1, ps)
        pages = B * width + 1  # a pool that holds the whole batch at its longest
        table, left = _paged(have, width, pages, seed)
        stack = torch.zeros(pages, dtype=torch.int32, device="cuda")
        stack[:left.numel()] = left
        s.update(context_len=_i32(ctx), new_len=_i32(new), table=table, stack=stack,
                 stack_count=_i32([left.numel()]), max_tokens=B * (case["new"] + 1))
        if after:
            kept = np.minimum(rng.permutation(_spread(0, case["new"], B)), new)
            if case["finish"]:
                kept[rng.permutation(B)[:B // case["finish"]]] = -1
            s.update(kept_len=_i32(kept), reserved_len=_i32(ctx + new + 1))
        if own:  # the outputs and scratch that a serving loop allocates once
            from speculative_decoding_verification_41_gb300 import paged
            s["buffers"] = (paged.ReleaseBuffers(B, "cuda") if after else
                            paged.ReserveBuffers(B, s["max_tokens"], "cuda"))
        return s
    if case["op"] == "append":
        n = case["tokens"]
        pages = _up(n + n // 4 + 1, case["page"])
        # runs of whole pages in random order, as a prompt fills them; a few padded rows
        page_order = torch.randperm(pages, generator=_gen(seed + 1), device="cuda")
        t = torch.arange(n, device="cuda")
        slots = page_order[t // case["page"]] * case["page"] + t % case["page"]
        if n > 16:
            slots[n - n // 16:] = -1
        row = [n, case["Hkv"], case["D"]]
        dt = DTYPES[case["dtype"]]
        s.update(slot_map=slots.to(torch.int32),
                 k=torch.randn(row, generator=_gen(seed + 2), device="cuda").to(dt),
                 v=torch.randn(row, generator=_gen(seed + 3), device="cuda").to(dt),
                 k_cache=_cache(pages, case, seed + 4), v_cache=_cache(pages, case, seed + 5))
        if own:
            s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        return s
    B = case["B"]
    new = rng.permutation(_spread(1, case["new"], B))
    ctx = np.maximum(rng.permutation(_spread(case["lo"], case["hi"], B)), new)
    width = _up(case["hi"], case["page"])
    counts = _up(ctx, case["page"])
    pages = int(counts.sum()) + 1 + seed % 7
    table, _ = _paged(counts, width, pages, seed)
    off = np.concatenate([[0], np.cumsum(new)])
    q = 2 * torch.randn(int(off[-1]), case["Hq"], case["D"], generator=_gen(seed + 2),
                        device="cuda")
    s.update(q=q.to(DTYPES[case["dtype"]]), k_cache=_cache(pages, case, seed + 4),
             v_cache=_cache(pages, case, seed + 5), table=table, context_len=_i32(ctx),
             row_off=torch.as_tensor(off).cuda(), max_new=case["new"], window=case["window"],
             scale=case["D"] ** -0.5)
    if own:
        from speculative_decoding_verification_41_gb300 import paged
        s["buffers"] = paged.AttentionBuffers(int(off[-1]), case["Hq"], case["Hkv"],
                                              case["D"], case["new"], DTYPES[case["dtype"]],
                                              "cuda", with_lse=True)
    return s


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    from speculative_decoding_verification_41_gb300 import paged
    if s["op"] == "reserve":
        o = paged.dspark_pages_reserve(s["context_len"], s["new_len"], s["table"], s["stack"],
                                       s["stack_count"], page_size=s["page"],
                                       max_tokens=s["max_tokens"], extra=1, buffers=s["buffers"])
        return [s["table"], o["context_len"], o["row_off"], o["draft_off"], o["slot_map"],
                o["positions"], o["free_count"]]
    if s["op"] == "release":
        o = paged.dspark_pages_release(s["context_len"], s["reserved_len"], s["kept_len"],
                                       s["table"], s["stack"], s["stack_count"],
                                       page_size=s["page"], extra=1, buffers=s["buffers"])
        return [s["stack"], o["context_len"], o["free_count"]]
    if s["op"] == "append":
        paged.dspark_kv_append(s["k"], s["v"], s["slot_map"], s["k_cache"], s["v_cache"],
                               device_status=s["status"])
        return [s["k_cache"], s["v_cache"]]
    o = paged.dspark_paged_attention(s["q"], s["k_cache"], s["v_cache"], s["table"],
                                     s["context_len"], s["row_off"], scale=s["scale"],
                                     max_new=s["max_new"], window=s["window"], with_lse=True,
                                     buffers=s["buffers"])
    return [o["out"], o["lse"]]


def _run_plain(s):
    return {"reserve": _reserve, "release": _release, "append": _append,
            "attention": _attention}[s["op"]](s)


def _reserve(s):
    ps, table, stack = s["page"], s["table"], s["stack"]
    B, width = table.shape
    ctx, draft = s["context_len"].long(), s["new_len"].long()
    n = draft + 1
    have, had = (ctx + ps - 1) // ps, (ctx + n + ps - 1) // ps
    need = had - have
    page0 = torch.cumsum(need, 0) - need
    zero = torch.zeros(1, dtype=torch.int64, device=table.device)
    row_off = torch.cat([zero, torch.cumsum(n, 0)])
    draft_off = torch.cat([zero, torch.cumsum(draft, 0)])
    top = s["stack_count"].long() - 1
    j = torch.arange(width, device=table.device)[None, :]
    fresh = (j >= have[:, None]) & (j < had[:, None])
    pop = (top - page0[:, None] - j + have[:, None]).clamp(0, stack.numel() - 1)
    table = torch.where(fresh, stack[pop], table)
    t = torch.arange(s["max_tokens"], device=table.device)
    r = torch.searchsorted(row_off[1:], t, right=True).clamp(max=B - 1)
    valid = t < row_off[B]
    pos = torch.where(valid, ctx[r] + t - row_off[r], -1)
    page = table[r, (pos // ps).clamp(0, width - 1)].long()
    slot = torch.where(valid, page * ps + pos % ps, -1)
    return [table, (ctx + n).int(), row_off, draft_off, slot.int(), pos.int(),
            s["stack_count"] - need.sum().int()]


def _release(s):
    ps, table, stack = s["page"], s["table"], s["stack"]
    ctx, kept = s["context_len"].long(), s["kept_len"].long()
    keep = torch.where(kept < 0, 0, ctx + kept + 1)
    stay, had = (keep + ps - 1) // ps, (s["reserved_len"].long() + ps - 1) // ps
    gone = had - stay
    first = s["stack_count"].long() + torch.cumsum(gone, 0) - gone
    j = torch.arange(table.shape[1], device=table.device)[None, :]
    back = (j >= stay[:, None]) & (j < had[:, None])
    to = torch.where(back, first[:, None] + j - stay[:, None], stack.numel())
    out = torch.cat([stack, stack.new_zeros(1)])
    out.scatter_(0, to.reshape(-1), table.reshape(-1))
    return [out[:-1], keep.int(), s["stack_count"] + gone.sum().int()]


def _append(s):
    ps = s["page"]
    t = torch.nonzero(s["slot_map"] >= 0).reshape(-1)
    slot = s["slot_map"][t].long()
    s["k_cache"][slot // ps, slot % ps] = s["k"][t]
    s["v_cache"][slot // ps, slot % ps] = s["v"][t]
    return [s["k_cache"], s["v_cache"]]


def _attention(s):
    q, off, ctx, T = s["q"], s["row_off"], s["context_len"].long(), s["max_new"]
    n, Hq, D = q.shape
    B, width = s["table"].shape
    Hkv, L = s["k_cache"].shape[2], width * s["page"]
    G = Hq // Hkv
    t = torch.arange(T, device=q.device)[None, :]
    new = (off[1:] - off[:-1])[:, None]
    row = (off[:-1, None] + t).clamp(max=n - 1)                            # [B, T]
    qp = q[row].float().reshape(B, T, Hkv, G, D).permute(0, 2, 3, 1, 4)    # [B, Hkv, G, T, D]
    table = s["table"].long()
    k = s["k_cache"][table].float().reshape(B, L, Hkv, D).transpose(1, 2)  # [B, Hkv, L, D]
    z = torch.matmul(qp.reshape(B, Hkv, G * T, D), k.transpose(2, 3)) * s["scale"]
    z = z.reshape(B, Hkv, G, T, L)
    end = (ctx[:, None] - new + t + 1)[:, :, None]                         # [B, T, 1]
    u = torch.arange(L, device=q.device)[None, None, :]
    seen = (u < end) & ((u >= end - s["window"]) if s["window"] else (u >= 0))
    z.masked_fill_(~seen[:, None, None], -math.inf)
    m = z.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = z.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    v = s["v_cache"][table].float().reshape(B, L, Hkv, D).transpose(1, 2)
    o = torch.matmul(p.reshape(B, Hkv, G * T, L), v).reshape(B, Hkv, G, T, D) / total
    lse = (m + total.log()).squeeze(-1)                                    # [B, Hkv, G, T]
    real = (t < new).reshape(-1).nonzero().reshape(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(B * T, Hq, D)[real]
    return [o.to(q.dtype), lse.permute(0, 3, 1, 2).reshape(B * T, Hq)[real]]


def _visible(case):
    """New tokens, contexts, cached tokens that some new token sees, and pairs, of a case."""
    new = _spread(1, case["new"], case["B"])
    ctx = np.maximum(_spread(case["lo"], case["hi"], case["B"]), new)
    w = case["window"] or 1 << 40
    span = np.minimum(ctx, w + new - 1).sum()
    pairs = sum(int(np.minimum(c - n + 1 + np.arange(n), w).sum()) for c, n in zip(ctx, new))
    return int(new.sum()), int(ctx.sum()), int(span), pairs


def work(case):
    if case["op"] == "reserve":
        B, new = case["B"], int(_spread(0, case["new"], case["B"]).sum()) + case["B"]
        pages = new // case["page"]
        return {"bytes": 8 * B * (case["new"] + 1) + 8 * pages + 28 * B, "flops": 0}
    if case["op"] == "release":
        B = case["B"]
        ctx, new = _spread(0, case["ctx"], B), _spread(0, case["new"], B)
        pages = int(new.sum()) // case["page"] // 2
        if case["finish"]:
            pages += int(ctx.sum()) // case["page"] // case["finish"]
        return {"bytes": 16 * B + 8 * pages, "flops": 0}
    if case["op"] == "append":
        n = case["tokens"]
        return {"bytes": 4 * n + 8 * (n - n // 16 if n > 16 else n) * case["Hkv"] * case["D"],
                "flops": 0}
    new, _, span, pairs = _visible(case)
    return {"bytes": 4 * span * case["Hkv"] * case["D"] + 4 * new * case["Hq"] * case["D"]
            + 4 * new * case["Hq"], "flops": 4 * pairs * case["Hq"] * case["D"]}


def exact(case, seed):
    s = prepare(case, seed)
    ps = case["page"]
    if case["op"] in ("reserve", "release"):
        return None  # whole numbers: the plain form's are the definition's
    if case["op"] == "append":
        flat = s["slot_map"].cpu().numpy()
        rows = np.flatnonzero(flat >= 0)
        page, at, rows = (torch.as_tensor(a).cuda() for a in (flat[rows] // ps, flat[rows] % ps,
                                                              rows))
        out = []
        for x, cache in ((s["k"], s["k_cache"]), (s["v"], s["v_cache"])):
            c = cache.double()
            c.index_put_((page.long(), at.long()), x.double().index_select(0, rows))
            out.append(c)
        return out
    off, ctx = s["row_off"].tolist(), s["context_len"].tolist()
    table = s["table"].cpu()
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    o = torch.zeros(off[-1], Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.full((off[-1], Hq), -math.inf, dtype=torch.float64, device="cuda")
    for r, c in enumerate(ctx):
        ids = table[r, :_up(c, ps)].long().cuda()
        k = s["k_cache"].index_select(0, ids).flatten(0, 1)[:c]
        v = s["v_cache"].index_select(0, ids).flatten(0, 1)[:c]
        T = off[r + 1] - off[r]
        first = 0
        if case["window"]:  # nothing before the first new token's window is seen
            first = max(0, c - T + 1 - case["window"])
        last = torch.arange(c - T, c, device="cuda")[:, None]
        u = torch.arange(first, c, device="cuda")[None, :]
        hidden = u > last
        if case["window"]:
            hidden |= u <= last - case["window"]
        for h in range(Hkv):
            heads = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            x = s["q"][off[r]:off[r + 1], heads].double().transpose(0, 1)   # [G, T, D]
            z = x @ k[first:, h].double().T * s["scale"]
            z = z.masked_fill(hidden[None], -math.inf)
            top = torch.logsumexp(z, -1)
            lse[off[r]:off[r + 1], heads] = top.T
            o[off[r]:off[r + 1], heads] = (torch.exp(z - top[..., None])
                                           @ v[first:, h].double()).transpose(0, 1)
    return [o, lse]
