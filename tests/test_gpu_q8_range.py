"""The 8-bit cache's calls at the ends of their ranges: elements of any size, blocks longer than a
CTA's window, slots past 4 GB, keys and values in one tensor, two streams at once."""
import math

import numpy as np
import pytest
import torch

from speculative_decoding_verification_41_gb300 import build as cuda_build
from speculative_decoding_verification_41_gb300 import paged, paged_q8
from tests import test_gpu_q8_cache as cache_tests
from tests.test_gpu_q8_cache import BOTH, check_append, make_cache, runs_to_slots

pytestmark = pytest.mark.gpu
dev = cache_tests.dev


@BOTH
@pytest.mark.parametrize("block", [1, 8, 32])
@pytest.mark.parametrize("D", [64, 128])
def test_append_elements_of_any_size(dev, dtype, block, D):
    """Rows from the smallest numbers to the largest of the type, alone and with others."""
    g = torch.Generator().manual_seed(D + block)
    n, heads = 150, 3
    low, high = (-24, 15) if dtype == torch.float16 else (-133, 127)
    x = [torch.rand(n, heads, D, generator=g) * 2 - 1 for _ in range(2)]
    # exponents of rows and heads, and of single elements below them
    k, v = ((y.double() * 2.0 ** torch.randint(low, high + 1, (n, heads, 1), generator=g).double()
             * 2.0 ** -torch.randint(0, 12, (n, heads, D), generator=g).double()).to(dtype).to(dev)
            for y in x)
    slots, _ = runs_to_slots([(0, 70), (3, 40), (31, 1), (5, 39)], 64, 30, 3)
    check_append(dev, k, v, slots, make_cache(30, 64, heads, D, block, 4, dev), block)


@BOTH
@pytest.mark.parametrize("block", [1, 16])
@pytest.mark.parametrize("inter", [False, True])
def test_append_turned_values_that_are_not_finite(dev, dtype, block, inter):
    g = torch.Generator().manual_seed(31)
    x = torch.randn(40, 2, 128, generator=g)
    x[0, 0, 3], x[9, 1, 100], x[17, 0, 64], x[33, 1, 127] = math.inf, math.nan, -math.inf, math.nan
    x[38] = math.nan
    k = x.to(dtype).to(dev)
    v = torch.randn(40, 2, 128, generator=g).to(dtype).to(dev)
    slots, pos = runs_to_slots([(0, 20), (7, 20)], 64, 4, 2)
    t = paged_q8.RotaryTable(112, interleaved=inter, device=dev)
    check_append(dev, k, v, slots, make_cache(4, 64, 2, 128, block, 6, dev), block, t, pos)


@BOTH
@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("heads,D", [(2, 128), (20, 64)])
def test_append_blocks_longer_than_a_window(dev, dtype, turned, heads, D):
    runs = [(0, 1000), (1000, 20), (100, 900), (1, 1), (500, 300)]
    n = sum(r[1] for r in runs)
    slots, pos = runs_to_slots(runs, 1024, 6, 1)
    slots[::97] = -1
    slots[300:640] = -1
    g = torch.Generator().manual_seed(12)
    k, v = ((torch.randn(n, heads, D, generator=g) * 2.0 ** (torch.arange(n) % 7)[:, None, None])
            .to(dtype).to(dev) for _ in range(2))
    t = paged_q8.RotaryTable(D, device=dev) if turned else None
    check_append(dev, k, v, slots, make_cache(6, 1024, heads, D, 1024, 3, dev), 1024, t,
                 pos if turned else None)


def attend(q, cache, table, ctx, off, max_new, buffers=None):
    return paged_q8.dspark_paged_attention_q8(q, *cache, table, ctx, off, scale=0.088,
                                              max_new=max_new, with_lse=True, buffers=buffers)


def test_slots_past_4_gb_in_a_tensor_of_keys_and_values(dev):
    """The last pages of a cache of 9.2 GB, K and V in one tensor, against a small cache."""
    pages, ps, heads, D, block, few = 70_000, 64, 8, 128, 16, 40
    big = torch.empty(pages, 2, ps, heads, D, dtype=torch.uint8, device=dev).view(paged_q8.E4M3)
    scales = torch.empty(pages, 2, ps // block, heads, device=dev)
    small = make_cache(few, ps, heads, D, block, 1, dev)
    large = (big[:, 0], big[:, 1], scales[:, 0], scales[:, 1])
    for a, b in zip(large, small):
        a[-few:].copy_(b)
    runs = [(0, 300), (63, 70), (5, 900)]
    n = sum(r[1] for r in runs)
    slots, pos = runs_to_slots(runs, ps, few, 9)
    g = torch.Generator().manual_seed(2)
    k, v = (torch.randn(n, heads, D, generator=g).bfloat16().to(dev) for _ in range(2))
    t = paged_q8.RotaryTable(128, device=dev)
    p = torch.from_numpy(pos).to(dev)
    s = torch.from_numpy(slots).to(dev)
    got = []
    for cache, add in ((small, 0), (large, (pages - few) * ps)):
        paged_q8.dspark_kv_append_q8(k, v, s + add, *cache, rotary=t, positions=p, check=True)
        back = paged_q8.dspark_kv_gather_q8(*cache, s + add, check=True)
        # the last request, whose pages follow the others'
        ids = torch.from_numpy(slots[370:][::1]).to(dev)
        first = torch.unique_consecutive(ids // ps)
        table = torch.zeros(1, 16, dtype=torch.int32, device=dev)
        table[0, :first.numel()] = first + add // ps
        q = torch.randn(3, 16, D, generator=torch.Generator().manual_seed(4)).bfloat16().to(dev)
        o = attend(q, cache, table, torch.tensor([900], dtype=torch.int32, device=dev),
                   torch.tensor([0, 3], device=dev), 3)
        assert int(o["device_status"].item()) == 0
        got.append([back["k"], back["v"], o["out"], o["lse"]]
                   + [x[-few:].view(torch.uint8) if x.dtype != torch.float32 else x[-few:]
                      for x in cache])
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert not got[0][2].isnan().any()


def test_two_streams_at_once(dev):
    """Append and attention of two caches on two streams, again and again, as one after the other."""
    g = torch.Generator().manual_seed(7)
    t = paged_q8.RotaryTable(64, device=dev)
    work = []
    for seed in range(2):
        runs = [(0, 400), (0, 33), (0, 1)]
        slots, pos = runs_to_slots(runs, 32, 20, seed)
        k, v = (torch.randn(434, 4, 64, generator=g).half().to(dev) for _ in range(2))
        q = torch.randn(9, 12, 64, generator=g).half().to(dev)
        table = torch.zeros(3, 13, dtype=torch.int32, device=dev)
        at = 0
        for r, (_, n) in enumerate(runs):
            ids = slots[at:at + n:32] // 32
            table[r, :len(ids)] = torch.from_numpy(ids).to(dev)
            at += n
        work.append((torch.from_numpy(slots).to(dev), torch.from_numpy(pos).to(dev), k, v, q, table))
    ctx = torch.tensor([400, 33, 1], dtype=torch.int32, device=dev)
    off = torch.tensor([0, 5, 8, 9], device=dev)

    def run(w, cache, buffers):
        slots, pos, k, v, q, table = w
        paged_q8.dspark_kv_append_q8(k, v, slots, *cache, rotary=t, positions=pos)
        return attend(q, cache, table, ctx, off, 5, buffers)

    def fresh(seed):
        return (make_cache(20, 32, 4, 64, 8, seed, dev),
                paged.AttentionBuffers(9, 12, 4, 64, 5, torch.float16, dev, with_lse=True))

    want = []
    for i, w in enumerate(work):
        cache, buffers = fresh(i)
        o = run(w, cache, buffers)
        want.append((o["out"].clone(), o["lse"].clone(), [x.clone() for x in cache]))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(dev) for _ in range(2)]
    state = [fresh(i) for i in range(2)]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, w in enumerate(work):
            with torch.cuda.stream(streams[i]):
                run(w, *state[i])
    torch.cuda.synchronize()
    for (cache, buffers), (out, lse, codes) in zip(state, want):
        assert int(buffers.device_status.item()) == 0
        assert torch.equal(buffers.out, out) and torch.equal(buffers.lse, lse)
        for a, b in zip(cache, codes):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert np.isfinite(want[0][0].float().cpu().numpy()).all()
