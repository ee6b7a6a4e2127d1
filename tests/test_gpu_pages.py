"""dspark_pages_reserve, dspark_pages_release and dspark_kv_append on the GPU,
against their plain statements: whole numbers, so every output is equal."""
import numpy as np
import pytest
import torch

from speculative_decoding_verification_41_gb300 import build as cuda_build
from speculative_decoding_verification_41_gb300 import paged
from tests import _paged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    cuda_build.build()
    return torch.device("cuda:0")


def t32(a, dev):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=dev)


def make(B, ps, ctx_max, new_max, seed, extra, spare=0, width_pad=0):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, ctx_max + 1, B).astype(np.int32)
    new = rng.integers(0, new_max + 1, B).astype(np.int32)
    width = _paged.up(ctx_max + new_max + extra, ps) + 1
    have = [_paged.up(int(c), ps) for c in ctx]
    need = [_paged.up(int(c + n) + extra, ps) - h for c, n, h in zip(ctx, new, have)]
    pages = sum(have) + sum(need) + spare + 1
    ids = rng.permutation(pages).astype(np.int32)
    table = np.full((B, width + width_pad), -5, np.int32)
    at = 0
    for r, h in enumerate(have):
        table[r, :h] = ids[at:at + h]
        at += h
    stack = np.full(pages, -9, np.int32)
    stack[:pages - at] = ids[at:]
    return ctx, new, table, stack, pages - at, pages, width


def run_reserve(dev, ctx, new, table, stack, count, ps, max_tokens, extra, width=None, **kw):
    tab = t32(table, dev)
    view = tab if width is None else tab[:, :width]
    o = paged.dspark_pages_reserve(t32(ctx, dev), t32(new, dev), view, t32(stack, dev),
                                   t32([count], dev), page_size=ps, max_tokens=max_tokens,
                                   extra=extra, **kw)
    torch.cuda.synchronize()
    o = {k: v.cpu().numpy() for k, v in o.items()}
    o["block_table"] = tab.cpu().numpy()
    return o


def same(o, ref, keys=("block_table", "context_len", "row_off", "draft_off", "slot_map",
                       "positions", "free_count")):
    assert int(o["device_status"][0]) == ref["status"]
    for k in keys:
        assert np.array_equal(o[k], ref[k]), k


@pytest.mark.parametrize("B,ps,ctx_max,new_max,extra,pad", [
    (1, 16, 0, 0, 1, 0), (1, 8, 100, 0, 0, 5), (3, 16, 50, 16, 1, 3), (64, 16, 4096, 16, 1, 7),
    (33, 1024, 5000, 3000, 1, 0), (255, 32, 1, 1, 0, 1), (1023, 8, 40, 9, 1, 4100),
    (1024, 64, 300, 33, 1, 2), (1025, 16, 64, 17, 2, 3), (3000, 16, 90, 5, 1, 11),
    (40, 128, 700, 9000, 1, 4097)])
def test_reserve(dev, B, ps, ctx_max, new_max, extra, pad):
    ctx, new, table, stack, count, pages, width = make(B, ps, ctx_max, new_max, B + ps, extra,
                                                       width_pad=3)
    tokens = int(new.sum()) + extra * B + pad
    ref = _paged.reserve(ctx, new, extra, table[:, :width], stack, count, ps, pages, tokens)
    assert ref["status"] == _paged.OK
    o = run_reserve(dev, ctx, new, table, stack, count, ps, tokens, extra, width=width)
    assert np.array_equal(o["block_table"][:, width:], table[:, width:])
    o["block_table"] = o["block_table"][:, :width]
    same(o, ref)


def test_reserve_without_requests_or_rows(dev):
    o = run_reserve(dev, [], [], np.zeros((0, 4), np.int32), np.arange(5), 3, 16, 6, 1)
    assert o["row_off"].tolist() == [0] and o["free_count"].tolist() == [3]
    assert o["slot_map"].tolist() == [-1] * 6 and int(o["device_status"][0]) == 0
    o = run_reserve(dev, [3, 16], [0, 0], np.zeros((2, 4), np.int32), np.arange(5), 3, 16, 0, 0)
    assert o["row_off"].tolist() == [0, 0, 0] and o["context_len"].tolist() == [3, 16]
    assert int(o["device_status"][0]) == 0


@pytest.mark.parametrize("seed", range(12))
def test_reserve_that_does_not_fit(dev, seed):
    """Too few free pages, too few rows, or both: the first request that does not fit ends it."""
    rng = np.random.default_rng(900 + seed)
    B = int(rng.choice([1, 5, 70, 1030, 2100]))
    ctx, new, table, stack, count, pages, width = make(B, 16, 60, 40, seed, 1)
    need = int(_paged.reserve(ctx, new, 1, table, stack, count, 16, pages, 1 << 20)
               ["row_off"][-1])
    short = int(rng.integers(0, max(1, count))) if seed % 3 != 1 else count
    tokens = int(rng.integers(0, need)) if seed % 3 != 0 else need
    ref = _paged.reserve(ctx, new, 1, table, stack, short, 16, pages, tokens)
    assert ref["status"] in (_paged.TOO_LARGE, _paged.NO_PAGES, _paged.OK)
    same(run_reserve(dev, ctx, new, table, stack, short, 16, tokens, 1), ref)


def test_reserve_bad_data(dev):
    ctx, new, table, stack, count, pages, width = make(9, 16, 60, 40, 5, 1, spare=20)
    room = width * 16
    for change in ("ctx", "new", "long", "huge"):
        c, n = ctx.copy(), new.copy()
        if change == "ctx":
            c[2] = -1
        elif change == "new":
            n[0] = -7
        elif change == "long":
            n[8] = room
        else:
            c[4], n[4] = 2 ** 31 - 1, 2 ** 31 - 1
        ref = _paged.reserve(c, n, 1, table, stack, count, 16, pages, 500)
        assert ref["status"] == _paged.BAD_DATA
        same(run_reserve(dev, c, n, table, stack, count, 16, 500, 1), ref)
    for bad in (-1, pages, 2 ** 31 - 1, -2 ** 31):  # page ids outside the pool
        s = stack.copy()
        s[count - 2] = bad
        t = table.copy()
        r = int(np.flatnonzero(ctx % 16)[0])
        t[r, ctx[r] // 16] = bad
        ref = _paged.reserve(ctx, new, 1, t, s, count, 16, pages, 500)
        assert ref["status"] == _paged.BAD_DATA and (ref["slot_map"] == pages * 16).any()
        same(run_reserve(dev, ctx, new, t, s, count, 16, 500, 1), ref)
    for n_free in (-1, pages + 1, 2 ** 31 - 1):
        ref = _paged.reserve(ctx, new, 1, table, stack, n_free, 16, pages, 500)
        assert ref["status"] == _paged.BAD_DATA
        same(run_reserve(dev, ctx, new, table, stack, n_free, 16, 500, 1), ref)


def test_buffers_and_refusals(dev):
    """Given buffers hold what allocated ones do; what is not the calls' is refused either way."""
    B, tokens = 70, 3000
    ctx, new, table, stack, count, pages, width = make(B, 16, 200, 40, 9, 1, spare=9)
    args = [t32(ctx, dev), t32(new, dev), t32(table, dev), t32(stack, dev), t32([count], dev)]
    opts = dict(page_size=16, max_tokens=tokens, extra=1)
    want = paged.dspark_pages_reserve(*args, **opts)
    buf = paged.ReserveBuffers(B, tokens, dev)
    got = paged.dspark_pages_reserve(*args, **opts, buffers=buf)
    torch.cuda.synchronize()
    assert all(torch.equal(want[k], got[k]) for k in want)
    kept = torch.zeros(B, dtype=torch.int32, device=dev)
    rel = [args[0], want["context_len"], kept, args[2]]
    a, b = args[3].clone(), args[3].clone()
    want_r = paged.dspark_pages_release(*rel, a, want["free_count"], page_size=16, extra=1)
    got_r = paged.dspark_pages_release(*rel, b, want["free_count"], page_size=16, extra=1,
                                       buffers=paged.ReleaseBuffers(B, dev))
    torch.cuda.synchronize()
    assert torch.equal(a, b) and all(torch.equal(want_r[k], got_r[k]) for k in want_r)
    for i, x in [(0, args[0].long()), (0, args[0].cpu()), (1, args[1][1:]), (2, args[2].long()),
                 (2, args[2][:, ::2]), (2, args[2][1:]), (3, args[3].float()), (4, args[3]),
                 (4, None)]:
        for given in (None, buf):
            with pytest.raises(ValueError):
                paged.dspark_pages_reserve(*args[:i], x, *args[i + 1:], **opts, buffers=given)
    for given in (paged.ReserveBuffers(B + 1, tokens, dev), paged.ReserveBuffers(B, 5, dev)):
        with pytest.raises(ValueError):
            paged.dspark_pages_reserve(*args, **opts, buffers=given)
    with pytest.raises(ValueError):
        paged.dspark_pages_release(*rel, a, want["free_count"], page_size=16,
                                   buffers=paged.ReleaseBuffers(B - 1, dev))
    for given in (None, buf):
        with pytest.raises(paged.DsparkError):
            paged.dspark_pages_reserve(*args, **{**opts, "page_size": 24}, buffers=given)
    cache = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device=dev)
    k = torch.ones(3, 2, 64, dtype=torch.bfloat16, device=dev)
    slots, st = t32([1, 2, 3], dev), t32([9], dev)
    assert paged.dspark_kv_append(k, k, slots, cache, cache, device_status=st)["device_status"] is st
    assert int(st.item()) == 0
    for bad in [(k.half(), k, slots, cache, cache), (k, k[:2], slots, cache, cache),
                (k, k, slots[:2], cache, cache), (k, k, slots.long(), cache, cache),
                (k, k, slots, cache, cache[:3]), (k[:, :1], k[:, :1], slots, cache, cache),
                (k, None, slots, cache, cache), (k.cpu(), k.cpu(), slots, cache, cache)]:
        for given in (None, st):
            with pytest.raises(ValueError):
                paged.dspark_kv_append(*bad, device_status=given)


@pytest.mark.parametrize("B", [3, 1500])
def test_in_place_lengths(dev, B):
    """context_out over context_len and the count over itself: the outputs of separate buffers."""
    ctx, new, table, stack, count, pages, width = make(B, 16, 200, 40, B, 1, spare=9)
    tokens = int(new.sum()) + B
    ref = _paged.reserve(ctx, new, 1, table, stack, count, 16, pages, tokens)
    buf = paged.ReserveBuffers(B, tokens, dev)
    buf.context_len, buf.free_count = t32(ctx, dev), t32([count], dev)
    tab, st = t32(table, dev), t32(stack, dev)
    o = paged.dspark_pages_reserve(buf.context_len, t32(new, dev), tab, st, buf.free_count,
                                   page_size=16, max_tokens=tokens, extra=1, buffers=buf)
    torch.cuda.synchronize()
    o = {k: v.cpu().numpy() for k, v in o.items()}
    o["block_table"] = tab.cpu().numpy()
    same(o, ref)
    kept = np.minimum(np.random.default_rng(3).integers(-1, 41, B), new).astype(np.int32)
    before = t32(ctx, dev)
    rel = paged.ReleaseBuffers(B, dev)
    rel.context_len, rel.free_count = buf.context_len, buf.free_count
    q = paged.dspark_pages_release(before, buf.context_len, t32(kept, dev), tab, st,
                                   buf.free_count, page_size=16, extra=1, buffers=rel)
    torch.cuda.synchronize()
    want = _paged.release(ctx, ref["context_len"], kept, 1, ref["block_table"], stack,
                          int(ref["free_count"][0]), 16, pages)
    assert int(q["device_status"].item()) == want["status"] == _paged.OK
    assert np.array_equal(st.cpu().numpy(), want["free_pages"])
    assert np.array_equal(q["context_len"].cpu().numpy(), want["context_len"])
    assert q["free_count"].item() == want["free_count"][0]


def run_release(dev, ctx, res, kept, table, stack, count, ps, extra):
    st = t32(stack, dev)
    o = paged.dspark_pages_release(t32(ctx, dev), t32(res, dev), t32(kept, dev), t32(table, dev),
                                   st, t32([count], dev), page_size=ps, extra=extra)
    torch.cuda.synchronize()
    return {"free_pages": st.cpu().numpy(), **{k: v.cpu().numpy() for k, v in o.items()}}


@pytest.mark.parametrize("B,ps,ctx_max,new_max,extra", [
    (1, 8, 0, 0, 1), (5, 16, 90, 16, 1), (256, 16, 400, 16, 1), (1024, 8, 70, 30, 0),
    (1025, 64, 900, 9, 1), (2600, 16, 60, 4, 1)])
def test_release(dev, B, ps, ctx_max, new_max, extra):
    rng = np.random.default_rng(B)
    ctx, new, table, stack, count, pages, width = make(B, ps, ctx_max, new_max, B, extra)
    o = _paged.reserve(ctx, new, extra, table, stack, count, ps, pages, 1 << 20)
    left = int(o["free_count"][0])
    kept = np.minimum(rng.integers(-1, new_max + 1, B), new).astype(np.int32)
    kept[rng.integers(0, B, 1 + B // 7)] = -1
    ref = _paged.release(ctx, o["context_len"], kept, extra, o["block_table"], stack, left, ps,
                         pages)
    got = run_release(dev, ctx, o["context_len"], kept, o["block_table"], stack, left, ps, extra)
    same(got, ref, ("free_pages", "context_len", "free_count"))
    assert ref["status"] == _paged.OK


def test_release_after_a_refusal_keeps_what_was_there(dev):
    """Requests that got nothing hold no new pages, whatever their draft lengths say."""
    ctx, new, table, stack, count, pages, width = make(50, 16, 60, 40, 7, 1)
    o = _paged.reserve(ctx, new, 1, table, stack, count // 2, 16, pages, 1 << 20)
    assert o["status"] == _paged.NO_PAGES
    kept = new // 2
    left = int(o["free_count"][0])
    ref = _paged.release(ctx, o["context_len"], kept, 1, o["block_table"], stack, left, 16, pages)
    got = run_release(dev, ctx, o["context_len"], kept, o["block_table"], stack, left, 16, 1)
    same(got, ref, ("free_pages", "context_len", "free_count"))
    assert ref["status"] == _paged.OK


def test_release_bad_data(dev):
    ctx, new, table, stack, count, pages, width = make(9, 16, 60, 40, 5, 1)
    o = _paged.reserve(ctx, new, 1, table, stack, count, 16, pages, 1 << 20)
    res, tab, left = o["context_len"], o["block_table"], int(o["free_count"][0])
    for change in ("more", "less", "back", "long", "negative", "full", "count"):
        c, e, k, n = ctx.copy(), res.copy(), new.copy(), left
        k[3] = -1
        if change == "more":
            k[1] = new[1] + 1
        elif change == "less":
            k[1] = -2
        elif change == "back":
            e[2] = c[2] - 1
        elif change == "long":
            e[2] = width * 16 + 1
        elif change == "negative":
            c[5] = -1
        elif change == "full":  # a stack that has no room for what comes back
            k[:] = -1
            n = pages - 2
        else:
            n = pages + 1
        ref = _paged.release(c, e, k, 1, tab, stack, n, 16, pages)
        assert ref["status"] == _paged.BAD_DATA
        same(run_release(dev, c, e, k, tab, stack, n, 16, 1), ref,
             ("free_pages", "context_len", "free_count"))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("n,Hkv,D,ps,layout", [
    (1, 1, 64, 8, "token"), (1, 8, 128, 16, "head"), (7, 3, 64, 16, "head"),
    (130, 8, 128, 16, "token"), (999, 5, 64, 128, "head"), (4097, 2, 128, 1024, "token"),
    (50, 128, 128, 16, "token"), (0, 4, 64, 16, "token")])
def test_append(dev, dtype, n, Hkv, D, ps, layout):
    g = torch.Generator().manual_seed(n + Hkv)
    pages = _paged.up(n, ps) + 3
    shape = [pages, ps, Hkv, D]
    base = [torch.randn(shape, generator=g).to(dtype) for _ in range(2)]
    rows = torch.randn(n, 3 * Hkv, D, generator=g).to(dtype)  # keys and values inside wider rows
    k, v = rows[:, :Hkv], rows[:, 2 * Hkv:]
    slots = torch.randperm(pages * ps, generator=g)[:n + 5].to(torch.int32)
    slots[torch.rand(n + 5, generator=g) < 0.2] = -1
    if n > 2:
        slots[1] = -2 ** 31
    want = [x.clone() for x in base]
    for x, y in zip(want, (k, v)):
        for i in range(n):
            s = int(slots[i])
            if s >= 0:
                x[s // ps, s % ps] = y[i]
    caches = [x.transpose(1, 2).contiguous().to(dev).transpose(1, 2) if layout == "head"
              else x.to(dev) for x in base]
    kd = rows.to(dev)
    o = paged.dspark_kv_append(kd[:, :Hkv], kd[:, 2 * Hkv:], slots.to(dev), *caches, check=True)
    assert int(o["device_status"].item()) == 0
    for x, y in zip(caches, want):
        assert torch.equal(x.cpu().view(torch.int16), y.view(torch.int16))


def test_append_slots_outside_the_pool(dev):
    cache = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device=dev)
    v = cache.clone()
    k = torch.ones(3, 2, 64, dtype=torch.bfloat16, device=dev)
    slots = torch.tensor([5, 64, 2 ** 31 - 1], dtype=torch.int32, device=dev)
    o = paged.dspark_kv_append(k, k, slots, cache, v)
    assert int(o["device_status"].item()) == _paged.BAD_DATA
    assert float(cache.float().sum()) == float(v.float().sum()) == 128.0
    o = paged.dspark_kv_append(k, k, slots[:1].repeat(3), cache, v)  # the status starts anew
    assert int(o["device_status"].item()) == 0


def test_append_past_32_bit_offsets(dev):
    """Slots whose element offsets pass 2^32: the last pages of a 9 GB cache."""
    pages, ps, H, D = 270000, 16, 8, 128
    cache = torch.empty(pages, ps, H, D, dtype=torch.bfloat16, device=dev)
    assert cache.numel() > 2 ** 32
    v = cache
    k = torch.randn(40, H, D, device=dev).to(torch.bfloat16)
    slots = torch.arange(pages * ps - 40, pages * ps, dtype=torch.int32, device=dev)
    paged.dspark_kv_append(k, k, slots, cache, v, check=True)
    got = cache.view(-1, H, D)[-40:]
    assert torch.equal(got, k)
