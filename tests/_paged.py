"""Plain statements of the paged-cache calls (include/dspark_paged.h) in numpy,
64 bits, and the inputs of their tests. Nothing here uses the library."""
from __future__ import annotations

import math
from dataclasses import dataclass

import numpy as np
import torch

OK, BAD_DATA, TOO_LARGE, NO_PAGES = 0, 5, 6, 7


def up(a: int, b: int) -> int:
    return -(-a // b)


def reserve(ctx, new, extra, table, stack, count, page_size, num_pages, max_tokens):
    """dspark_pages_reserve, request by request. Returns a dict of its outputs."""
    table = table.copy()
    width = table.shape[1]
    ok_count = 0 <= count <= num_pages
    avail = count if ok_count else 0
    status = set() if ok_count else {BAD_DATA}
    ctx_out, row_off, draft_off, slots, pos = list(ctx), [0], [0], [], []
    tokens = drafts = popped = 0
    closed = False
    for r, (c, d) in enumerate(zip(ctx.tolist(), new.tolist())):
        n = d + extra
        if c < 0 or d < 0 or c + n > width * page_size:
            status.add(BAD_DATA)
            n = 0
        elif n > 0 and not closed:
            need = up(c + n, page_size) - up(c, page_size)
            if tokens + n > max_tokens:
                status.add(TOO_LARGE)
                closed = True
            if popped + need > avail:
                status.add(NO_PAGES)
                closed = True
        if closed or n == 0:
            row_off.append(tokens)
            draft_off.append(drafts)
            continue
        first = up(c, page_size)
        for j in range(first, up(c + n, page_size)):
            table[r, j] = stack[avail - 1 - popped]
            popped += 1
            if not 0 <= table[r, j] < num_pages:
                status.add(BAD_DATA)
        if c % page_size and not 0 <= table[r, c // page_size] < num_pages:
            status.add(BAD_DATA)
        for p in range(c, c + n):
            page = int(table[r, p // page_size])
            good = 0 <= page < num_pages
            slots.append(page * page_size + p % page_size if good else num_pages * page_size)
            pos.append(p)
        tokens += n
        drafts += d
        ctx_out[r] = c + n
        row_off.append(tokens)
        draft_off.append(drafts)
    pad = [-1] * (max_tokens - len(slots))
    st = next((s for s in (BAD_DATA, TOO_LARGE, NO_PAGES) if s in status), OK)
    return {"block_table": table, "context_len": np.array(ctx_out, np.int32),
            "row_off": np.array(row_off, np.int64), "draft_off": np.array(draft_off, np.int64),
            "slot_map": np.array(slots + pad, np.int32), "positions": np.array(pos + pad, np.int32),
            "free_count": np.array([count - popped], np.int32), "status": st}


def release(ctx, reserved, kept, extra, table, stack, count, page_size, num_pages):
    """dspark_pages_release, request by request."""
    stack = stack.copy()
    ok_count = 0 <= count <= num_pages
    top = count if ok_count else num_pages
    bad, out = not ok_count, []
    room = table.shape[1] * page_size
    for r, (c, e, k) in enumerate(zip(ctx.tolist(), reserved.tolist(), kept.tolist())):
        if c < 0 or e < c or e > room or k < -1 or (k >= 0 and e > c and k + extra > e - c):
            bad = True
            out.append(e)
            continue
        keep = 0 if k < 0 else c + k + extra if e > c else e
        for j in range(up(keep, page_size), up(e, page_size)):
            if top < num_pages:
                stack[top] = table[r, j]
            else:
                bad = True
            top += 1
        out.append(keep)
    now = min(top, num_pages) if ok_count else count
    return {"free_pages": stack, "context_len": np.array(out, np.int32),
            "free_count": np.array([now], np.int32), "status": BAD_DATA if bad else OK}


@dataclass
class Attention:
    """Inputs of dspark_paged_attention on one device."""
    q: torch.Tensor
    k_cache: torch.Tensor
    v_cache: torch.Tensor
    table: torch.Tensor
    context_len: torch.Tensor
    row_off: torch.Tensor
    scale: float
    max_new: int
    window: int


def make_attention(lens, news, Hq, Hkv, D, page_size, dtype, *, layout="token", window=0,
                   q_gain=1.0, seed=0, device="cpu", max_new=None, poison=True,
                   table_pad=0) -> Attention:
    """Requests of these cached lengths and new-token counts with their pages in random order.
    Everything in the cache that no row may see is NaN (poison): the rest of last pages, pages
    that nobody holds and, with a window, what lies before it (whose table entries are -1)."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    counts = [up(n, page_size) for n in lens]
    width = max(1, max(counts)) + 1
    pages = sum(counts) + 3
    ids = rng.permutation(pages)
    shape = [pages, page_size, Hkv, D]
    fill = math.nan if poison else 0.0
    k, v = torch.full(shape, fill, dtype=dtype), torch.full(shape, fill, dtype=dtype)
    table = np.full((len(lens), width + table_pad), -1, np.int32)
    at = 0
    for r, (n, T) in enumerate(zip(lens, news)):
        first = max(0, n - T + 1 - window) if window else 0
        for j in range(counts[r]):
            page = int(ids[at])
            at += 1
            lo, hi = max(first - j * page_size, 0), min(n - j * page_size, page_size)
            if lo >= page_size:
                continue  # before the window: page given back
            table[r, j] = page
            m = hi - lo
            k[page, lo:hi] = torch.randn(m, Hkv, D, generator=g).to(dtype)
            v[page, lo:hi] = torch.randn(m, Hkv, D, generator=g).to(dtype)
    if layout == "head":
        k, v = (x.transpose(1, 2).contiguous().transpose(1, 2) for x in (k, v))
    off = np.concatenate([[0], np.cumsum(news)])
    q = (q_gain * torch.randn(max(int(off[-1]), 1), Hq, D, generator=g)).to(dtype)
    put = lambda x: _put(x, device)
    return Attention(put(q), put(k), put(v), torch.from_numpy(table).to(device)[:, :width],
                     torch.tensor(list(lens), dtype=torch.int32, device=device),
                     torch.from_numpy(off.astype(np.int64)).to(device), D ** -0.5,
                     max_new or max(max(news), 1), window)


def _put(x, device):
    """x on `device` with its strides (a dense permutation of its dimensions)."""
    out = torch.empty_strided(x.shape, x.stride(), dtype=x.dtype, device=device)
    out.copy_(x)
    return out


def attention(a: Attention, u: float):
    """out and lse in 64 bits, and how far a computation in the call's precision may be off.
    u: half a step of the inputs' type.

    The bound. Scores: D products in 16 bits are exact in binary32, their sum is off by at most
    D 2^-23 sum|q||k| (an adder that truncates); scaling and the reference add 2^-22 |score| + 2^-22,
    the exponential 2^-21. Call that relative error of a weight e. Weights are rounded to 16 bits for
    the second product (u each; half precision below 2^-14: 2^-25 of the largest), not in their
    sum. The sum of n products is off by at most n 2^-23 of the sum of their magnitudes. The
    result is rounded once more (u)."""
    q = a.q.double().cpu().numpy()
    n_tokens, Hq, D = q.shape
    ps, Hkv = a.k_cache.shape[1], a.k_cache.shape[2]
    table = a.table.cpu().numpy()
    off, ctx = a.row_off.cpu().numpy(), a.context_len.cpu().numpy()
    out, lse = np.zeros((n_tokens, Hq, D)), np.full((n_tokens, Hq), -np.inf)
    tol, lse_tol = np.zeros((n_tokens, Hq, D)), np.zeros((n_tokens, Hq))
    half = a.q.dtype == torch.float16
    for r in range(len(ctx)):
        T, n = int(off[r + 1] - off[r]), int(ctx[r])
        first = max(0, n - T + 1 - a.window) if a.window else 0
        if T == 0 or n == 0:
            continue
        pos = np.arange(first, n)
        page = torch.from_numpy(table[r][pos // ps].astype(np.int64)).to(a.k_cache.device)
        at = torch.from_numpy(pos % ps).to(a.k_cache.device)
        K = a.k_cache[page, at].double().cpu().numpy()   # [n - first, Hkv, D]
        V = a.v_cache[page, at].double().cpu().numpy()
        for t in range(T):
            end = n - T + t + 1
            lo = max(0, end - a.window) if a.window else 0
            if end <= lo:
                continue
            row = int(off[r]) + t
            for h in range(Hq):
                kk, vv = K[lo - first:end - first, h // (Hq // Hkv)], V[lo - first:end - first, h // (Hq // Hkv)]
                with np.errstate(all="ignore"):
                    z = kk @ q[row, h] * a.scale
                    top = z.max()
                    w = np.exp(z - top)
                    total = w.sum()
                    w /= total
                    out[row, h] = w @ vv
                    lse[row, h] = top + np.log(total)
                    mag = w @ np.abs(vv)
                    e = (D * 2.0 ** -23 * (np.abs(kk) @ np.abs(q[row, h])).max() * a.scale
                         + 2.0 ** -22 * np.abs(z).max() + 2.0 ** -21 + 2.0 ** -22)
                    m = end - lo
                    tol[row, h] = (u * np.abs(out[row, h]) * 1.01
                                   + (u + 2 * e + 2 * m * 2.0 ** -23) * mag
                                   + (m * 2.0 ** -25 * np.abs(vv).max() if half else 0) + 2.0 ** -25)
                    lse_tol[row, h] = e + m * 2.0 ** -23 + 2.0 ** -22 * abs(lse[row, h])
    return out, lse, tol, lse_tol
