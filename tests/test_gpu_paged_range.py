"""dspark_paged_attention where a row's weights span a wide range, against softmax
attention in 64 bits: one token far above a long tail (whose value is zero, so
that the tail alone makes the result)."""
import math

import numpy as np
import pytest
import torch

from speculative_decoding_verification_41_gb300 import build as cuda_build
from speculative_decoding_verification_41_gb300 import paged

pytestmark = pytest.mark.gpu

# rows per key head (query heads of a group, new tokens): every row block
BLOCKS = [(1, 1), (8, 1), (16, 2), (8, 6), (8, 10), (8, 17)]


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    cuda_build.build()
    return torch.device("cuda:0")


def attend(dev, q, k, v, B, ps, scale):
    """B requests with the same queries q [T, Hq, D] over the same tokens k, v [L, Hkv, D] (their
    block tables name the same pages): requests enough that a CTA has whole ones."""
    L, H, D = k.shape
    T, Hq, _ = q.shape
    pages = -(-L // ps)
    cache = torch.full((2, pages * ps, H, D), math.nan, dtype=k.dtype, device=dev)
    cache[0, :L], cache[1, :L] = k.to(dev), v.to(dev)
    kc, vc = cache.view(2, pages, ps, H, D)
    table = torch.arange(pages, dtype=torch.int32, device=dev).repeat(B, 1)
    o = paged.dspark_paged_attention(
        q.to(dev).repeat(B, 1, 1), kc, vc, table, torch.full((B,), L, dtype=torch.int32, device=dev),
        torch.arange(B + 1, device=dev) * T, scale=scale, max_new=T, with_lse=True, check=True)
    return (o["out"].double().cpu().numpy().reshape(B, T, Hq, D),
            o["lse"].double().cpu().numpy().reshape(B, T, Hq))


def exact(q, k, v, scale, floor):
    """out and lse in 64 bits and how far they may be off. The bound: scores are off by D 2^-23 of
    the sum of their products' magnitudes (an adder that truncates), 2^-22 of themselves for scaling
    and reference, 2^-21 and 2^-22 for the exponential (e, relative to a weight); a weight is
    rounded to the type (half a step u), or, below the type's normal range, by floor of the
    largest; sums of n in binary32 by n 2^-23 each; the result once more by u, or 2^-25."""
    T, Hq, D = q.shape
    L, H, _ = k.shape
    u = torch.finfo(q.dtype).eps / 2
    qq, kk, vv = (x.double().numpy() for x in (q, k, v))
    out, lse, tol, lse_tol = (np.zeros((T, Hq, D)), np.zeros((T, Hq)), np.zeros((T, Hq, D)),
                              np.zeros((T, Hq)))
    for t in range(T):
        n = L - T + t + 1
        for h in range(Hq):
            K, V = kk[:n, h // (Hq // H)], vv[:n, h // (Hq // H)]
            z = K @ qq[t, h] * scale
            w = np.exp(z - z.max())
            lse[t, h] = z.max() + np.log(w.sum())
            w /= w.sum()
            out[t, h] = w @ V
            e = (D * 2.0 ** -23 * (np.abs(K) @ np.abs(qq[t, h])).max() * scale
                 + 2.0 ** -22 * np.abs(z).max() + 2.0 ** -21 + 2.0 ** -22)
            tol[t, h] = (u * np.abs(out[t, h]) * 1.01 + (u + 2 * e + 2 * n * 2.0 ** -23) * (w @ np.abs(V))
                         + n * floor * w.max() * np.abs(V).max() + 2.0 ** -25)
            lse_tol[t, h] = e + n * 2.0 ** -23 + 2.0 ** -22 * abs(lse[t, h])
    return out, lse, tol, lse_tol


def sink(L, G, T, D, dtype, at, drop, seed, H=1):
    """Token `at` is `drop` nats above the others, which differ by some tenths; its value is 0."""
    g = torch.Generator().manual_seed(seed)
    q, k = torch.randn(T, H * G, D, generator=g) * 0.3, torch.randn(L, H, D, generator=g)
    q[:, :, 0], k[:, :, 0] = 1.0, 0.0
    k[at], v = 0.0, 1.0 + 0.25 * torch.randn(L, H, D, generator=g)
    k[at, :, 0], v[at] = drop * D ** 0.5, 0.0
    return q.to(dtype), k.to(dtype), v.to(dtype), D ** -0.5


# What half precision rounds away below its normal range: half of 2^-24, where the largest weight is
# at least 2^12 (a row with a peak), or 2^9 (any row).
FLOOR = {torch.float16: 2.0 ** -37, torch.bfloat16: 0.0}
ANY_FLOOR = {torch.float16: 2.0 ** -34, torch.bfloat16: 0.0}


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("G,T", BLOCKS)
@pytest.mark.parametrize("L,at,drop", [(2200, 3, 12.0), (2200, 3, 17.0), (2200, 1000, 17.0),
                                       (2200, 2150, 17.0), (900, 400, 15.0), (900, 0, 21.0)])
def test_one_token_far_above_the_rest(dev, dtype, G, T, L, at, drop):
    D = 64 if G == 16 or T == 10 else 128
    q, k, v, scale = sink(L, G, T, D, dtype, at, drop, seed=L + at, H=2)
    want, lse, tol, lse_tol = exact(q, k, v, scale, FLOOR[dtype])
    got, got_lse = attend(dev, q, k, v, 160, 16, scale)
    off = np.abs(got - want)
    assert (off <= tol).all(), f"off by {(off / tol).max():.2f} of the bound"
    assert (np.abs(got_lse - lse) <= lse_tol).all()


@pytest.mark.parametrize("G,T", [(1, 1), (8, 6)])
@pytest.mark.parametrize("drop", [12.5, 18.0])
def test_one_token_far_above_a_long_tail(dev, G, T, drop):
    """110,000 tokens of half precision; a CTA has some 23,000 of them."""
    q, k, v, scale = sink(110000, G, T, 64, torch.float16, 5, drop, seed=G)
    want, lse, tol, lse_tol = exact(q, k, v, scale, FLOOR[torch.float16])
    got, got_lse = attend(dev, q, k, v, 64, 64, scale)
    off = np.abs(got - want)
    assert (off <= tol).all(), f"off by {(off / tol).max():.2f} of the bound"
    assert (np.abs(got_lse - lse) <= lse_tol).all()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("G,T", BLOCKS)
@pytest.mark.parametrize("L,first,drop", [(2200, 0, 15.0), (2200, 0, 17.0), (2200, 1024, 17.0),
                                          (900, 640, 18.0)])
def test_peaks_everywhere_in_a_tile(dev, dtype, G, T, L, first, drop):
    """Eight tokens of one tile, 16 apart, far above the rest."""
    D = 64 if G == 16 or T == 10 else 128
    at = torch.arange(first, first + 128, 16) + 5
    q, k, v, scale = sink(L, G, T, D, dtype, at, drop, seed=L + first, H=2)
    want, lse, tol, lse_tol = exact(q, k, v, scale, ANY_FLOOR[dtype])
    got, got_lse = attend(dev, q, k, v, 160, 16, scale)
    off = np.abs(got - want)
    assert (off <= tol).all(), f"off by {(off / tol).max():.2f} of the bound"
    assert (np.abs(got_lse - lse) <= lse_tol).all()


@pytest.mark.parametrize("G,T", BLOCKS)
@pytest.mark.parametrize("L,rise", [(700, 40.0), (2300, 40.0), (2300, 9.0)])
def test_values_near_the_end_of_the_range(dev, G, T, L, rise):
    """bf16 values of 2^110 and scores that rise along the context (from nothing to `rise` nats past
    the first half): every partial sum in the formula's order of magnitude is in binary32's range."""
    D = 128
    g = torch.Generator().manual_seed(L)
    q, k = torch.randn(T, G, D, generator=g) * 0.1, torch.randn(L, 1, D, generator=g)
    q[:, :, 0], k[:, :, 0] = 1.0, 0.0
    k[L // 2:, :, 0] = rise * D ** 0.5
    v = (torch.randn(L, 1, D, generator=g) * 0.25 + 1.0) * 2.0 ** 110
    q, k, v = (x.to(torch.bfloat16) for x in (q, k, v))
    want, lse, tol, lse_tol = exact(q, k, v, D ** -0.5, 0.0)
    got, got_lse = attend(dev, q, k, v, 320, 16, D ** -0.5)
    assert np.isfinite(got).all()
    off = np.abs(got - want)
    assert (off <= tol).all(), f"off by {(off / tol).max():.2f} of the bound"
    assert (np.abs(got_lse - lse) <= lse_tol).all()
