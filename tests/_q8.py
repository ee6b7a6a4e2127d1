"""Plain statements of the 8-bit cache's calls (include/dspark_q8.h) in 64 bits, and the
inputs of their tests. Nothing here uses the library."""
from __future__ import annotations

import math
from dataclasses import dataclass

import numpy as np
import torch

from tests import _paged

E4M3 = torch.float8_e4m3fn
# the numbers of the 256 codes, from the format's definition
_c = np.arange(256)
_sign, _e, _m = np.where(_c & 128, -1.0, 1.0), (_c >> 3) & 15, _c & 7
CODES = _sign * np.where(_e == 0, _m * 2.0 ** -9, (1 + _m / 8) * 2.0 ** (_e - 7.0))
CODES[(_c & 127) == 127] = math.nan


def numbers(codes: torch.Tensor) -> np.ndarray:
    """What a tensor of codes stands for, without its scales."""
    return CODES[codes.cpu().contiguous().view(torch.uint8).numpy()]


def rounded(x: np.ndarray) -> np.ndarray:
    """The nearest e4m3 numbers, ties to even; |x| <= 448. NaN and infinities: NaN."""
    with np.errstate(all="ignore"):
        e = np.floor(np.log2(np.maximum(np.abs(x), 2.0 ** -6)))
        step = 2.0 ** (e - 3)
        return np.where(np.isfinite(x), np.round(x / step) * step, np.nan)


def needed(a: float) -> float:
    """The smallest 2^e, e >= -126, with a <= 448 * 2^e."""
    e = -126
    if a > 0:
        e = max(-126, math.frexp(a / 448)[1])
        while e > -126 and a <= 448 * 2.0 ** (e - 1):
            e -= 1
        while a > 448 * 2.0 ** e:
            e += 1
    return 2.0 ** e


def turned(x: np.ndarray, positions: np.ndarray, angles, gain=1.0, interleaved=False,
           inverse=False) -> np.ndarray:
    """Rows x [n, heads, D] turned by their positions."""
    rot = 2 * len(angles)
    th = positions.astype(np.float64)[:, None] * np.asarray(angles)[None, :] * (-1 if inverse else 1)
    c, s = gain * np.cos(th)[:, None], gain * np.sin(th)[:, None]
    y = x.astype(np.float64).copy()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, b * c + a * s
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * c - b * s, b * c + a * s
    return y


def append(rows, slots, numbers_, scale, block):
    """One cache (its numbers [pages, page, heads, D], changed in place) and its scales
    ([pages, page / block, heads]) with rows [n, heads, D] in their slots."""
    ps, n_slots = numbers_.shape[1], numbers_.shape[0] * numbers_.shape[1]
    taken = {}
    for i, s in enumerate(slots):
        if 0 <= s < n_slots:
            taken.setdefault(s // block, []).append((int(s), i))
    for b, got in taken.items():
        page, at, index = b * block // ps, b * block % ps, b * block % ps // block
        fresh = any(s % block == 0 for s, _ in got)
        for h in range(numbers_.shape[2]):
            v = np.abs(np.concatenate([rows[i, h] for _, i in got]))
            a = v[np.isfinite(v)].max(initial=0.0)
            old, now = scale[page, index, h], needed(a)
            if not fresh and 0 < old < math.inf:
                if a <= 448 * float(old):
                    now = float(old)
                else:
                    numbers_[page, at:at + block, h] = rounded(
                        numbers_[page, at:at + block, h] * (float(old) / now))
            scale[page, index, h] = now
            for s, i in got:
                numbers_[page, s % ps, h] = rounded(rows[i, h] / now)


@dataclass
class Attention(_paged.Attention):
    """Inputs of dspark_paged_attention_q8; k_cache and v_cache are codes."""
    k_scale: torch.Tensor = None
    v_scale: torch.Tensor = None


def make_attention(lens, news, Hq, Hkv, D, page_size, dtype, *, block=16, layout="token", window=0,
                   q_gain=1.0, seed=0, device="cpu", max_new=None, poison=True, table_pad=0,
                   spread=2, exact_scales=True) -> Attention:
    """_paged.make_attention's requests, their cache in codes with scales of their blocks within
    2^spread of each other. What no row may see is NaN, code and scale."""
    block = min(block, page_size)
    a = _paged.make_attention(lens, news, Hq, Hkv, D, page_size, dtype, window=window,
                              q_gain=q_gain, seed=seed, max_new=max_new, poison=poison,
                              table_pad=table_pad)
    g = torch.Generator().manual_seed(seed + 1)
    codes, scales = [], []
    for x in (a.k_cache, a.v_cache):
        x = x.float()
        pages = x.shape[0]
        e = torch.randint(-spread, 1, (pages, page_size // block, Hkv), generator=g)
        s = 2.0 ** (e - 7)
        if not exact_scales:
            s = s * (1 + torch.rand(s.shape, generator=g))
        seen = ~x[..., 0].isnan()  # [pages, page, heads]
        c = (x * 100).clamp(-448, 448).to(E4M3)
        c.view(torch.uint8)[x.isnan()] = 0x7F if poison else 0
        any_seen = seen.reshape(pages, -1, block, Hkv).any(2)
        s = torch.where(any_seen, s, math.nan if poison else 1.0)
        if layout == "head":
            c = c.transpose(1, 2).contiguous().transpose(1, 2)
            s = s.transpose(1, 2).contiguous().transpose(1, 2)
        codes.append(_paged._put(c, device))
        scales.append(_paged._put(s, device))
    put = lambda t: _paged._put(t, device)
    # the table keeps the padding behind its rows
    table = a.table.new_full((a.table.shape[0], a.table.shape[1] + table_pad), -1)
    table[:, :a.table.shape[1]] = a.table
    return Attention(put(a.q), codes[0], codes[1], table.to(device)[:, :a.table.shape[1]],
                     put(a.context_len), put(a.row_off), a.scale, a.max_new, a.window, scales[0],
                     scales[1])


def attention(a: Attention):
    """out and lse in 64 bits, and how far a computation in the call's precision may be off.

    The bound. Queries: the parts miss at most 2^-17 of the row's largest element (2^-10 where it
    is scaled to 2^7 or more) of each. Scores: the parts' products with 4-bit codes are exact in
    binary32, their sum (QP * D products of at most 1.1 |q| |k| in all) is off by at most
    QP D 2^-23 1.1 sum|q||k| (an adder that truncates); two factors, a product and the reference
    add 2^-22 + 2^-22 |score|, the exponential 2^-21. Call that relative error of a weight e.
    Weights for the second product: times two factors (2^-23); cut to 9 bits after being made
    larger by 2^-9.47, so off by at most 2^-8 (bf16), or rounded to 11 bits, 2^-11 (half
    precision); small ones by 2^-19 where the largest is 2^9 vs / 2^r or more and 2^r is at most
    4 max vs: 2^-28 of the largest weight times 4 max vs and the code, at most 448.
    The sum of n products in PP parts is off by at most PP n 2^-23 of the sum of their
    magnitudes. The result is rounded once more: half a step, u."""
    q = a.q.double().cpu().numpy()
    n_tokens, Hq, D = q.shape
    half = a.q.dtype == torch.float16
    u = torch.finfo(a.q.dtype).eps / 2
    QP, PP, uw = (3, 4, 2.0 ** -11) if half else (2, 3, 2.0 ** -8)
    ps, Hkv = a.k_cache.shape[1], a.k_cache.shape[2]
    block = ps // a.k_scale.shape[1]
    k, v = numbers(a.k_cache), numbers(a.v_cache)
    ks, vs = a.k_scale.double().cpu().numpy(), a.v_scale.double().cpu().numpy()
    table = a.table.cpu().numpy()
    off, ctx = a.row_off.cpu().numpy(), a.context_len.cpu().numpy()
    out, lse = np.zeros((n_tokens, Hq, D)), np.full((n_tokens, Hq), -np.inf)
    tol, lse_tol = np.zeros((n_tokens, Hq, D)), np.zeros((n_tokens, Hq))
    for r in range(len(ctx)):
        T, n = int(off[r + 1] - off[r]), int(ctx[r])
        first = max(0, n - T + 1 - a.window) if a.window else 0
        if T == 0 or n == 0:
            continue
        pos = np.arange(first, n)
        page, at = table[r][pos // ps], pos % ps
        K = k[page, at] * ks[page, at // block][..., None]   # [n - first, Hkv, D]
        S = vs[page, at // block]
        V = v[page, at] * S[..., None]
        for t in range(T):
            end = n - T + t + 1
            lo = max(0, end - a.window) if a.window else 0
            if end <= lo:
                continue
            row, sl = int(off[r]) + t, slice(lo - first, end - first)
            for h in range(Hq):
                kk, vv, x = K[sl, h // (Hq // Hkv)], V[sl, h // (Hq // Hkv)], q[row, h]
                with np.errstate(all="ignore"):
                    z = kk @ x * a.scale
                    top = z.max()
                    w = np.exp(z - top)
                    total = w.sum()
                    w /= total
                    out[row, h] = w @ vv
                    lse[row, h] = top + np.log(total)
                    mag = w @ np.abs(vv)
                    size = np.abs(kk)
                    e = (2.0 ** -17 * size.sum(1).max() * np.abs(x).max() * a.scale
                         + QP * D * 2.0 ** -23 * 1.1 * (size @ np.abs(x)).max() * a.scale
                         + 2.0 ** -22 * np.abs(z).max() + 2.0 ** -22 + 2.0 ** -21)
                    m = end - lo
                    tol[row, h] = (u * np.abs(out[row, h]) * 1.01
                                   + (uw + 2 * e + 2.0 ** -22 + 2 * PP * m * 2.0 ** -23) * mag
                                   + m * 2.0 ** -28 * 4 * S[sl].max() * 448 + 2.0 ** -25)
                    lse_tol[row, h] = e + m * 2.0 ** -23 + 2.0 ** -22 * abs(lse[row, h])
    return out, lse, tol, lse_tol
