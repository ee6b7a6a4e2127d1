"""dspark_paged_attention on the GPU against softmax attention in 64 bits.

Everything in the cache that no row may see holds NaN, so a read of it shows.
The bound of every comparison is _paged.attention's, derived there from the
call's arithmetic before its first run."""
import math

import numpy as np
import pytest
import torch

from speculative_decoding_verification_41_gb300 import build as cuda_build
from speculative_decoding_verification_41_gb300 import paged
from tests import _paged

pytestmark = pytest.mark.gpu

HALF_STEP = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16)}


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    cuda_build.build()
    return torch.device("cuda:0")


def call(a, buffers=None, **kw):
    """With buffers of its own unless given some: the usual path of the binding."""
    n, Hq, D = a.q.shape
    buffers = buffers or paged.AttentionBuffers(n, Hq, a.k_cache.shape[2], D, a.max_new, a.q.dtype,
                                                a.q.device, with_lse=True)
    return paged.dspark_paged_attention(a.q, a.k_cache, a.v_cache, a.table, a.context_len,
                                        a.row_off, scale=a.scale, max_new=a.max_new,
                                        window=a.window, with_lse=True, buffers=buffers, **kw)


def check(a, o=None, rows=None):
    if o is None:
        o = call(a)
    torch.cuda.synchronize()
    assert int(o["device_status"].item()) == 0
    out, lse, tol, lse_tol = _paged.attention(a, HALF_STEP[a.q.dtype])
    n = int(a.row_off[-1].item())
    rows = np.arange(n) if rows is None else rows
    got, got_lse = o["out"].double().cpu().numpy(), o["lse"].double().cpu().numpy()
    off = np.abs(got - out)[rows]
    assert not np.isnan(got[rows]).any()
    worst = (off / tol[rows].clip(1e-300)).max() if off.size else 0.0
    assert (off <= tol[rows]).all(), f"off by {worst:.2f} of the bound"
    seen = np.isfinite(lse[rows])
    assert np.array_equal(np.isneginf(got_lse[rows]), ~seen)
    d = np.abs(got_lse[rows][seen] - lse[rows][seen])
    assert (d <= lse_tol[rows][seen]).all()
    return o


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128])
def test_one_tile(dev, dtype, D):
    """The smallest call: one request, one key head, one new token, 20 cached tokens."""
    check(_paged.make_attention([20], [1], 1, 1, D, 16, dtype, device=dev))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("layout,ps", [("token", 8), ("head", 16), ("token", 64), ("head", 128),
                                       ("token", 256), ("head", 1024)])
def test_lengths_and_pages(dev, dtype, D, layout, ps):
    """Single new tokens over contexts around the borders of pages and tiles."""
    lens = [1, 2, 7, 8, 15, 16, 17, 127, 128, 129, 255, 256, 257, 300, 511, 640, 1000, 1025]
    check(_paged.make_attention(lens, [1] * len(lens), 8, 2, D, ps, dtype, layout=layout,
                                seed=ps + D, device=dev))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,T", [
    (1, 1, 1), (16, 1, 1), (17, 1, 1), (8, 8, 5), (12, 4, 5), (32, 1, 1), (33, 1, 1), (64, 1, 1),
    (10, 5, 17), (8, 1, 8), (8, 1, 17), (24, 8, 33), (5, 1, 32), (65, 1, 1), (16, 2, 18),
    (160, 1, 1), (161, 1, 1), (322, 2, 2), (7, 7, 160), (7, 1, 33), (16, 1, 33)])
def test_heads_and_new_tokens(dev, Hq, Hkv, T, D):
    """Head layouts and draft lengths, over every row block and more rows than one holds; news
    of zero tokens among them."""
    rng = np.random.default_rng(Hq * 100 + T)
    news = [T, 0, max(1, T // 2), 1, T]
    lens = [int(n + rng.integers(0, 300)) for n in news]
    dtype = torch.bfloat16 if (Hq + T) % 2 else torch.float16
    check(_paged.make_attention(lens, news, Hq, Hkv, D, 16, dtype, seed=Hq + T, device=dev))


@pytest.mark.parametrize("T,G,D,window", [(1, 1, 64, 1), (1, 8, 128, 5), (5, 4, 128, 128),
                                          (9, 1, 64, 100), (17, 8, 128, 3), (17, 4, 64, 129),
                                          (4, 2, 128, 100000), (33, 2, 64, 257)])
def test_window(dev, T, G, D, window):
    """Sliding windows; pages wholly before one have been given back (table entries -1)."""
    rng = np.random.default_rng(T + window)
    news = [T, 1, max(1, T - 1), T, T]
    lens = [max(n, int(x)) for n, x in zip(news, [T, 700, 129, 1000, 263])]
    check(_paged.make_attention(lens, news, 2 * G, 2, D, 16, torch.bfloat16, window=window,
                                seed=int(rng.integers(1000)), device=dev))


@pytest.mark.parametrize("D", [64, 128])
def test_rows_that_see_nothing(dev, D):
    """More new tokens than cached ones, and no cached token at all: zeros and lse -inf."""
    a = _paged.make_attention([3, 0, 9, 0, 140], [8, 5, 9, 1, 8], 8, 2, D, 16, torch.bfloat16,
                              device=dev)
    o = check(a)
    assert float(o["out"][:5].float().abs().max()) == 0.0
    assert bool((o["lse"][:5] == -math.inf).all())
    assert float(o["out"][8:13].float().abs().max()) == 0.0


@pytest.mark.parametrize("G,T,D", [(4, 1, 128), (1, 1, 64), (8, 5, 128), (8, 17, 128), (8, 17, 64)])
def test_long_contexts_split(dev, G, T, D):
    """Contexts that many CTAs share, next to short ones."""
    a = _paged.make_attention([20011, 1 + T, 7777, T], [T] * 4, 2 * G, 2, D, 64, torch.bfloat16,
                              seed=G + T, device=dev)
    first = check(a)
    again = call(a)
    torch.cuda.synchronize()
    assert torch.equal(first["out"], again["out"]) and torch.equal(first["lse"], again["lse"])


@pytest.mark.parametrize("gain", [0.0, 8.0, 60.0])
def test_flat_and_steep_scores(dev, gain):
    """All scores equal; scores whose maximum keeps rising; single weights near one."""
    for dtype in (torch.bfloat16, torch.float16):
        check(_paged.make_attention([900, 130, 3000], [3, 1, 2], 8, 2, 128, 16, dtype,
                                    q_gain=gain, seed=5, device=dev))


def test_rising_maximum(dev):
    """Keys that grow along the context: every tile raises the reference."""
    a = _paged.make_attention([2000], [2], 4, 1, 128, 16, torch.bfloat16, seed=2, device=dev)
    ps, table = 16, a.table.cpu().numpy()
    q = a.q[0, 0].float()
    for p in range(2000):
        a.k_cache[int(table[0, p // ps]), p % ps, 0] = (q * (p / 40.0)).to(torch.bfloat16) / 8
    check(a)


@pytest.mark.parametrize("B,T", [(700, 1), (300, 9)])
def test_many_requests(dev, B, T):
    """More requests than threads of a CTA, most of them short."""
    rng = np.random.default_rng(B)
    news = rng.integers(0, T + 1, B).tolist()
    lens = [int(n + (0 if rng.random() < 0.1 else rng.integers(0, 200))) for n in news]
    check(_paged.make_attention(lens, news, 4, 2, 64, 16, torch.float16, seed=B, max_new=T,
                                device=dev))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("value", [math.nan, math.inf, -math.inf])
def test_values_that_later_rows_alone_see(dev, dtype, D, value):
    """Infinite or NaN keys and values of a draft token reach the rows that see it and no other."""
    T, n, ps = 6, 131, 16
    a = _paged.make_attention([n, 40], [T, T], 8, 2, D, ps, dtype, seed=9, device=dev)
    clean = call(a)["out"].clone()
    u = n - 3  # seen by the rows t >= 3
    page = int(a.table[0, u // ps])
    a.v_cache[page, u % ps, 1, 5] = value
    a.v_cache[page, u % ps, 1, D - 1] = value
    o = call(a)["out"]
    torch.cuda.synchronize()
    hit = torch.zeros(o.shape, dtype=torch.bool, device=dev)
    hit[3:T, 4:, 5] = hit[3:T, 4:, D - 1] = True  # heads 4.. share key head 1
    assert torch.equal(o[~hit], clean[~hit])
    bad = o[hit].float()
    assert bool(torch.isnan(bad).all() if math.isnan(value) else (bad == value).all())
    a.v_cache[page, u % ps, 1] = 0
    a.k_cache[page, u % ps, 1] = math.nan
    o = call(a)["out"]
    torch.cuda.synchronize()
    rows = torch.zeros(o.shape, dtype=torch.bool, device=dev)
    rows[3:T, 4:] = True
    assert torch.equal(o[~rows], clean[~rows])
    assert bool(torch.isnan(o[rows]).all())


def test_values_before_some_windows(dev):
    """An infinite value that the first new tokens' windows still hold and the later ones' not."""
    T, n, w, ps = 5, 400, 50, 16
    a = _paged.make_attention([n], [T], 2, 1, 64, ps, torch.bfloat16, window=w, seed=4, device=dev)
    clean = call(a)["out"].clone()
    u = n - T + 1 - w + 2  # the windows of rows 0..2 begin at or before it
    a.v_cache[int(a.table[0, u // ps]), u % ps, 0, 7] = math.inf
    o = call(a)["out"]
    torch.cuda.synchronize()
    assert bool(torch.isinf(o[:3, :, 7]).all())
    o[:3, :, 7] = clean[:3, :, 7]
    assert torch.equal(o, clean)


def test_infinite_scores(dev):
    """A score of -inf weighs nothing; rows of nothing else, or of +inf, are NaN as the formula's."""
    a = _paged.make_attention([200, 30], [1, 1], 2, 1, 64, 16, torch.bfloat16, seed=4, device=dev)
    a.q[:, :, 0] = 1.0
    for p in range(150):  # whole first tile and more
        a.k_cache[int(a.table[0, p // 16]), p % 16, 0, 0] = -math.inf
    o = call(a)
    torch.cuda.synchronize()
    keep = _paged.make_attention([200, 30], [1, 1], 2, 1, 64, 16, torch.bfloat16, seed=4)
    tab = a.table.cpu().numpy()
    pos = np.arange(150, 200)
    K = a.k_cache.cpu()[tab[0][pos // 16], pos % 16, 0].double().numpy()
    V = keep.v_cache[tab[0][pos // 16], pos % 16, 0].double().numpy()
    z = K @ a.q[0].double().cpu().numpy().T * a.scale
    w = np.exp(z - z.max(0))
    want = (w / w.sum(0)).T @ V
    assert np.abs(o["out"][0].double().cpu().numpy() - want).max() < 2.0 ** -7 * np.abs(V).max()
    for p in range(30):
        a.k_cache[int(tab[1, p // 16]), p % 16, 0, 0] = -math.inf
    o = call(a)
    torch.cuda.synchronize()
    assert bool(torch.isnan(o["out"][1]).all()) and not bool(torch.isnan(o["out"][0]).any())
    for p in range(30):
        a.k_cache[int(tab[1, p // 16]), p % 16, 0, 0] = math.inf if p == 3 else 0.0
    o = call(a)
    torch.cuda.synchronize()
    assert bool(torch.isnan(o["out"][1]).all()) and not bool(torch.isnan(o["out"][0]).any())


def test_strides_streams_and_graphs(dev):
    """q inside wider rows, a block table with longer rows, a side stream, a captured call."""
    a = _paged.make_attention([300, 17, 900], [2, 1, 2], 8, 2, 128, 32, torch.bfloat16, seed=8,
                              table_pad=5, device=dev)
    want = check(a)
    wide = torch.full((5, 24, 128), math.nan, dtype=torch.bfloat16, device=dev)
    wide[:, 8:16] = a.q
    a.q = wide[:, 8:16]
    torch.cuda.synchronize()
    side = torch.cuda.Stream(dev)
    o = call(a, stream=side)
    side.synchronize()
    assert torch.equal(o["out"], want["out"])
    o = paged.dspark_paged_attention(a.q, a.k_cache, a.v_cache, a.table, a.context_len, a.row_off,
                                     scale=a.scale, max_new=a.max_new, with_lse=True, stream=side)
    side.synchronize()
    assert torch.equal(o["out"], want["out"]) and torch.equal(o["lse"], want["lse"])
    buf = paged.AttentionBuffers(5, 8, 2, 128, a.max_new, torch.bfloat16, dev, with_lse=True)
    call(a, buffers=buf)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(a, buffers=buf)
    for _ in range(3):
        buf.out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(buf.out, want["out"])
    # lengths are read on the device: the same graph serves other ones
    a.context_len -= 1
    a.context_len[1] = 17
    graph.replay()
    torch.cuda.synchronize()
    check(a, {"out": buf.out, "lse": buf.lse, "device_status": buf.device_status})


def test_rows_outside_requests_are_left(dev):
    """Padded rows of q, before the first request's and after the last's, are not written."""
    a = _paged.make_attention([50, 60], [2, 3], 4, 2, 64, 16, torch.bfloat16, seed=1, device=dev)
    q = torch.zeros(12, 4, 64, dtype=torch.bfloat16, device=dev)
    q[4:9] = a.q
    want = check(a)["out"]
    a.q, a.row_off = q, a.row_off + 4
    buf = paged.AttentionBuffers(12, 4, 2, 64, 3, torch.bfloat16, dev, with_lse=True)
    buf.out.fill_(3.0)
    buf.lse.fill_(3.0)
    o = call(a, buffers=buf)
    torch.cuda.synchronize()
    assert torch.equal(o["out"][4:9], want)
    assert bool((o["out"][:4] == 3).all() and (o["out"][9:] == 3).all())
    assert bool((o["lse"][:4] == 3).all() and (o["lse"][9:] == 3).all())


def test_bad_data(dev):
    """Lengths and offsets that do not fit set the status and leave the other requests right;
    page ids outside the pool set it too."""
    a = _paged.make_attention([50, 300, 60], [2, 2, 2], 4, 2, 64, 16, torch.bfloat16, seed=1,
                              device=dev)
    want = check(a)["out"]
    good = a.context_len.clone()
    for v in (-1, a.table.shape[1] * 16 + 1, 2 ** 31 - 1):
        a.context_len[1] = v
        o = call(a)
        torch.cuda.synchronize()
        assert int(o["device_status"].item()) == _paged.BAD_DATA
        assert torch.equal(o["out"][:2], want[:2]) and torch.equal(o["out"][4:], want[4:])
    a.context_len.copy_(good)
    off = a.row_off.clone()
    for v in ([0, 2, 6, 6], [0, 2, 1, 6], [0, 2, 2 ** 40, 6], [0, 2, -5, 6]):
        a.row_off.copy_(torch.tensor(v))
        o = call(a)
        torch.cuda.synchronize()
        assert int(o["device_status"].item()) == _paged.BAD_DATA
        assert torch.equal(o["out"][:2], want[:2])
    a.row_off.copy_(off)
    for v in (-1, a.k_cache.shape[0], 2 ** 31 - 1):
        a.table[1, 3] = v
        o = call(a)
        torch.cuda.synchronize()
        assert int(o["device_status"].item()) == _paged.BAD_DATA
        assert torch.equal(o["out"][:2], want[:2]) and torch.equal(o["out"][4:], want[4:])


def test_past_32_bit_offsets(dev):
    """Pages whose element offsets pass 2^32 (the end of a 9 GB cache)."""
    pages, ps, H, D = 270000, 16, 8, 128
    big = torch.empty(pages, ps, H, D, dtype=torch.bfloat16, device=dev)
    assert big.numel() > 2 ** 32
    big[-20:] = torch.randn(20, ps, H, D, device=dev).to(torch.bfloat16)
    table = torch.arange(pages - 20, pages, dtype=torch.int32, device=dev).flip(0)[None]
    q = torch.randn(3, 32, D, device=dev).to(torch.bfloat16)
    a = _paged.Attention(q, big, big, table, torch.tensor([311], dtype=torch.int32, device=dev),
                         torch.tensor([0, 3], device=dev), D ** -0.5, 3, 0)
    check(a)


def test_binding(dev):
    """Outputs that the call allocates itself are the ones of given buffers, and tensors that are
    not the call's are refused on either path before anything is launched."""
    a = _paged.make_attention([50, 300], [2, 1], 4, 2, 64, 16, torch.bfloat16, seed=1, device=dev)
    want = call(a)
    args = [a.q, a.k_cache, a.v_cache, a.table, a.context_len, a.row_off]
    opts = dict(scale=a.scale, max_new=a.max_new, with_lse=True)
    o = paged.dspark_paged_attention(*args, **opts)
    torch.cuda.synchronize()
    assert torch.equal(o["out"], want["out"]) and torch.equal(o["lse"], want["lse"])
    buf = paged.AttentionBuffers(3, 4, 2, 64, 2, torch.bfloat16, dev, with_lse=True)
    marks = buf.out.fill_(7.0)
    bad = [(0, a.q.half()), (0, a.q.cpu()), (0, a.q[:, :3]), (0, a.q.transpose(1, 2)), (0, None),
           (1, a.k_cache.half()), (1, a.k_cache.transpose(2, 3)), (2, a.v_cache[:-1]),
           (2, a.v_cache.clone().transpose(1, 2).contiguous().transpose(1, 2)),
           (3, a.table.long()), (3, a.table[:1]), (3, a.table.cpu()), (4, a.context_len[:1]),
           (4, a.context_len.long()), (5, a.row_off[:2]), (5, a.row_off.int())]
    for i, x in bad:
        for given in (None, buf):
            with pytest.raises(ValueError):
                paged.dspark_paged_attention(*args[:i], x, *args[i + 1:], **opts, buffers=given)
    for given in (paged.AttentionBuffers(2, 4, 2, 64, 2, torch.bfloat16, dev, with_lse=True),
                  paged.AttentionBuffers(3, 4, 2, 64, 2, torch.float16, dev, with_lse=True),
                  paged.AttentionBuffers(3, 4, 2, 64, 2, torch.bfloat16, dev)):
        with pytest.raises(ValueError):
            paged.dspark_paged_attention(*args, **opts, buffers=given)
    for wrong in (dict(scale=0.0), dict(window=-1)):
        for given in (None, buf):
            with pytest.raises(paged.DsparkError):
                paged.dspark_paged_attention(*args, **{**opts, **wrong}, buffers=given)
    torch.cuda.synchronize()
    assert bool((marks == 7.0).all())


def test_nothing_to_do(dev):
    a = _paged.make_attention([5], [0], 4, 2, 64, 16, torch.bfloat16, device=dev, max_new=1)
    o = call(a)
    torch.cuda.synchronize()
    assert int(o["device_status"].item()) == 0
    empty = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device=dev)
    o = paged.dspark_paged_attention(empty, a.k_cache, a.v_cache, a.table, a.context_len,
                                     a.row_off, scale=1.0, max_new=1, check=True)
    assert o["out"].shape == (0, 4, 64)
