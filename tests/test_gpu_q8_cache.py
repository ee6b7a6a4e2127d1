"""dspark_rotary, dspark_kv_append_q8 and dspark_kv_gather_q8 on the GPU against their plain
statements in 64 bits (_q8)."""
import math

import numpy as np
import pytest
import torch

from speculative_decoding_verification_41_gb300 import build as cuda_build
from speculative_decoding_verification_41_gb300 import paged, paged_q8
from tests import _q8

pytestmark = pytest.mark.gpu

BOTH = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    cuda_build.build()
    return torch.device("cuda:0")


# ---- rotary
def rotary_bound(x, want, dtype, gain=1.0):
    """Angles are right to 2^-25 + 2^-32 of a half turn (2^-23 with pi), sine and cosine to two
    steps of binary32 (2^-22), the sum of two products to 2^-23 of each: less than 2^-20 of |a| +
    |b| in all. Then half a step of the output (and of half precision's smallest number)."""
    u = torch.finfo(dtype).eps / 2
    size = np.abs(x).max(-1, keepdims=True) * 2 * abs(gain)
    return 1.01 * u * np.abs(want) + 2.0 ** -20 * size + 2.0 ** -25


@BOTH
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 64), (128, 112)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n,heads", [(1, 1), (3, 5), (70, 3), (33, 40)])
def test_rotary(dev, dtype, D, rot, inter, n, heads):
    g = torch.Generator().manual_seed(rot + n)
    x = torch.randn(n, heads, D, generator=g).to(dtype)
    pos = torch.randint(0, 1 << 20, (n,), generator=g, dtype=torch.int32)
    pos[0] = 0
    t = paged_q8.RotaryTable(rot, interleaved=inter, device=dev)
    out = torch.empty(n, heads, D, dtype=dtype, device=dev)
    paged_q8.dspark_rotary(x.to(dev), pos.to(dev), t, out=out)
    want = _q8.turned(x.double().numpy(), pos.numpy(), t.angles, interleaved=inter)
    off = np.abs(out.double().cpu().numpy() - want)
    assert (off <= rotary_bound(x.double().numpy(), want, dtype)).all()
    assert torch.equal(out[0].cpu(), x[0])  # position 0


@pytest.mark.parametrize("pos", [1, 4095, 131071, 16777217, 2 ** 31 - 1])
def test_rotary_far_positions(dev, pos):
    x = torch.randn(1, 2, 128, generator=torch.Generator().manual_seed(1)).half()
    t = paged_q8.RotaryTable(128, base=500000.0, device=dev)
    p = torch.tensor([pos], dtype=torch.int32)
    out = paged_q8.dspark_rotary(x.to(dev), p.to(dev), t)["out"]
    want = _q8.turned(x.double().numpy(), p.numpy(), t.angles)
    # the statement's own angles: pos * 2^-53 radians
    bound = rotary_bound(x.double().numpy(), want, torch.float16) + pos * 2.0 ** -52
    assert (np.abs(out.double().cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("scaling", ["linear", "ntk", "yarn"])
def test_rotary_scaled(dev, scaling):
    t = paged_q8.RotaryTable(64, scaling=scaling, factor=8.0, original_len=2048, device=dev)
    x = torch.randn(20, 2, 128, generator=torch.Generator().manual_seed(2)).bfloat16()
    pos = torch.arange(20, dtype=torch.int32) * 777
    out = paged_q8.dspark_rotary(x.to(dev), pos.to(dev), t)["out"]
    want = _q8.turned(x.double().numpy(), pos.numpy(), t.angles, t.gain)
    assert (np.abs(out.double().cpu().numpy() - want)
            <= rotary_bound(x.double().numpy(), want, torch.bfloat16, t.gain)).all()


def test_rotary_strides_in_place_padding_and_negative_positions(dev):
    g = torch.Generator().manual_seed(3)
    qkv = torch.randn(50, 9, 128, generator=g).bfloat16()
    pos = torch.randint(0, 999, (60,), generator=g, dtype=torch.int32)
    pos[[4, 30]] = -1
    t = paged_q8.RotaryTable(128, device=dev)
    d = qkv.to(dev)
    paged_q8.dspark_rotary(d[:, :6], pos.to(dev), t, out=d[:, :6])
    want = qkv.double().numpy()
    turned = _q8.turned(want[:, :6], pos.numpy()[:50], t.angles)
    keep = pos.numpy()[:50] < 0
    turned[keep] = want[keep, :6]
    got = d.double().cpu().numpy()
    assert (np.abs(got[:, :6] - turned) <= rotary_bound(want[:, :6], turned, torch.bfloat16)).all()
    assert np.array_equal(got[keep], want[keep]) and np.array_equal(got[:, 6:], want[:, 6:])


@BOTH
@pytest.mark.parametrize("inter", [False, True])
def test_rotary_inverse_is_the_gradient(dev, dtype, inter):
    """<g, turn(x)> = <inverse(g), x>, and against differences of the 64-bit statement."""
    gen = torch.Generator().manual_seed(4)
    x = torch.randn(7, 3, 64, generator=gen).to(dtype)
    g = torch.randn(7, 3, 64, generator=gen).to(dtype)
    pos = torch.randint(0, 5000, (7,), generator=gen, dtype=torch.int32)
    t = paged_q8.RotaryTable(32, interleaved=inter, gain=1.25, device=dev)
    back = paged_q8.dspark_rotary(g.to(dev), pos.to(dev), t, inverse=True)["out"]
    f = lambda y: float((g.double().numpy() * _q8.turned(y, pos.numpy(), t.angles, t.gain, inter)).sum())
    x64 = x.double().numpy()
    got, u = back.double().cpu().numpy(), torch.finfo(dtype).eps / 2
    for i, h, d in ((0, 0, 0), (3, 1, 5), (6, 2, 17), (2, 0, 31), (5, 2, 40), (1, 1, 63)):
        step = np.zeros_like(x64)
        step[i, h, d] = 0.5
        diff = f(x64 + step) - f(x64 - step)  # linear: exact but for rounding
        bound = rotary_bound(g.double().numpy(), got, dtype, 1.25)
        assert abs(got[i, h, d] - diff) <= bound[i, h, d] + 2 * u * abs(diff)


# ---- append
def make_cache(pages, ps, heads, D, block, seed, dev, layout="token"):
    """Codes of every kind (but NaN) and scales that are powers of two."""
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in range(2):
        c = torch.randint(0, 256, (pages, ps, heads, D), generator=g, dtype=torch.uint8)
        c[(c & 127) == 127] = 3
        s = 2.0 ** torch.randint(-12, -5, (pages, ps // block, heads), generator=g).float()
        c = c.view(_q8.E4M3)
        if layout == "head":
            c = c.transpose(1, 2).contiguous().transpose(1, 2)
        out += [_q8._paged._put(c, dev), _q8._paged._put(s, dev)]
    return out[0], out[2], out[1], out[3]


def runs_to_slots(runs, ps, pages, seed):
    """(first position, tokens) of every request; their pages in random order."""
    ids = np.random.default_rng(seed).permutation(pages)
    slots, pos, at = [], [], 0
    for first, n in runs:
        need = -(-(first + n) // ps)
        mine = ids[at:at + need]
        at += need
        p = np.arange(first, first + n)
        slots += (mine[p // ps] * ps + p % ps).tolist()
        pos += p.tolist()
    assert at <= pages
    return np.array(slots, np.int32), np.array(pos, np.int32)


def check_append(dev, k, v, slots, cache, block, table=None, pos=None, status=0):
    kc, vc, ks, vs = cache
    want = []
    for x, c, s in ((k, kc, ks), (v, vc, vs)):
        rows = x.double().cpu().numpy()
        sl = slots.copy()
        if table is not None and x is k:
            rows = _q8.turned(rows, pos, table.angles, table.gain, table.interleaved)
        if table is not None:
            sl[pos < 0] = -1
        num, sc = _q8.numbers(c), s.cpu().numpy().copy()
        _q8.append(rows, sl, num, sc, block)
        want.append((num, sc))
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    paged_q8.dspark_kv_append_q8(k, v, torch.from_numpy(slots).to(dev), kc, vc, ks, vs,
                                 rotary=table,
                                 positions=None if table is None else torch.from_numpy(pos).to(dev),
                                 device_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == status
    for (num, sc), c, s, turned in ((want[0], kc, ks, table is not None), (want[1], vc, vs, False)):
        got = _q8.numbers(c)
        assert np.array_equal(s.cpu().numpy(), sc.astype(np.float32), equal_nan=True)
        assert np.array_equal(np.isnan(got), np.isnan(num))
        if not turned:
            assert np.array_equal(np.nan_to_num(got), np.nan_to_num(num))
        else:
            # binary32 rotation: a code may be the other neighbour where 64 bits lie within
            # 2^-20 of the row's largest element of a border; scales as above
            differ = got != num
            differ &= ~np.isnan(num)
            size = np.maximum(np.abs(np.nan_to_num(num)), 2.0 ** -6)  # (NaN: compared above)
            step = np.maximum(2.0 ** np.floor(np.log2(size)) / 8, 2.0 ** -9)
            assert (np.abs(np.nan_to_num(got - num)) <= step).all()
            assert differ.mean() < 2.0 ** -10


RUNS = [[(0, 1)], [(0, 40)], [(3, 1), (17, 17), (15, 2), (0, 5)], [(31, 1), (5, 11), (0, 16), (16, 16)],
        [(i * 7 % 33, 1 + i % 18) for i in range(30)]]


@BOTH
@pytest.mark.parametrize("D,heads", [(64, 3), (128, 2), (128, 9)])
@pytest.mark.parametrize("page,block", [(16, 16), (16, 1), (32, 4), (64, 64), (128, 32)])
@pytest.mark.parametrize("runs", RUNS)
def test_append(dev, dtype, D, heads, page, block, runs):
    n = sum(r[1] for r in runs)
    slots, _ = runs_to_slots(runs, page, 300, n)
    g = torch.Generator().manual_seed(n)
    k, v = ((torch.randn(n, heads, D, generator=g) * 2.0 ** torch.randint(-6, 3, (n, 1, 1), generator=g))
            .to(dtype).to(dev) for _ in range(2))
    cache = make_cache(300, page, heads, D, block, n, dev, "head" if heads == 9 else "token")
    check_append(dev, k, v, slots, cache, block)


@BOTH
@pytest.mark.parametrize("D,rot", [(64, 64), (64, 32), (128, 128), (128, 48)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("block", [1, 16, 64])
def test_append_turned(dev, dtype, D, rot, inter, block):
    runs = [(i * 11 % 70, 1 + i * 5 % 80) for i in range(9)]
    n = sum(r[1] for r in runs)
    slots, pos = runs_to_slots(runs, 64, 40, rot)
    g = torch.Generator().manual_seed(rot)
    k, v = (torch.randn(n, 3, D, generator=g).to(dtype).to(dev) for _ in range(2))
    pos[5] = -1  # skipped, like a negative slot
    t = paged_q8.RotaryTable(rot, interleaved=inter, gain=0.9, device=dev)
    check_append(dev, k, v, slots, make_cache(40, 64, 3, D, block, 5, dev), block, t, pos)


@BOTH
def test_append_padding_order_and_bad_slots(dev, dtype):
    g = torch.Generator().manual_seed(6)
    slots = np.array([-1, 5, 4, 3, -7, 17, -1, 63, 62, 64, 10 ** 6, 2 ** 31 - 1, 33], np.int32)
    k, v = (torch.randn(len(slots), 2, 64, generator=g).to(dtype).to(dev) for _ in range(2))
    check_append(dev, k, v, slots, make_cache(4, 16, 2, 64, 8, 7, dev), 8, status=5)


@BOTH
def test_append_values_that_are_not_finite_zeros_and_ends(dev, dtype):
    g = torch.Generator().manual_seed(8)
    x = torch.randn(24, 2, 128, generator=g)
    x[0, 0, 3], x[1, 1, 9], x[2, 0, 0] = math.inf, -math.inf, math.nan
    x[8:16] = 0
    x[16, 0] = torch.finfo(dtype).max
    x[17, 1] = torch.finfo(dtype).tiny * 0.25
    k = x.to(dtype).to(dev)
    v = torch.full((24, 2, 128), math.nan, dtype=dtype, device=dev)
    slots = np.arange(24, dtype=np.int32)
    check_append(dev, k, v, slots, make_cache(4, 32, 2, 128, 8, 9, dev), 8)


def test_append_scales_at_their_borders(dev):
    """Largest magnitudes of exactly 448 * 2^e, and the next number above."""
    k = torch.zeros(8, 1, 64)
    for i, m in enumerate((448.0, 450.0, 224.0, 225.0, 7.0, 7.03125, 1.75, 1.7578125)):
        k[i, 0, i] = -m if i % 2 else m
    k = k.bfloat16().to(dev)
    check_append(dev, k, k.clone(), np.arange(8, dtype=np.int32),
                 make_cache(1, 8, 1, 64, 1, 10, dev), 1)


def test_append_keeps_scales_that_are_no_powers_of_two(dev):
    g = torch.Generator().manual_seed(11)
    kc, vc, ks, vs = make_cache(3, 16, 2, 64, 16, 12, dev)
    ks.mul_(1.37), vs.mul_(100.3)
    k, v = (torch.randn(5, 2, 64, generator=g).half().to(dev) for _ in range(2))
    kk = k.clone()
    before = vs.clone()
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    paged_q8.dspark_kv_append_q8(kk, v, torch.arange(4, 9, dtype=torch.int32, device=dev), kc, vc,
                                 ks, vs, device_status=st)
    torch.cuda.synchronize()
    assert torch.equal(vs, before)
    got = _q8.numbers(vc)[0, 4:9]
    exact = v.double().cpu().numpy() / vs[0, 0].double().cpu().numpy()[:, None]
    # a division in binary32 before the rounding: half a step and 2^-23
    step = 2.0 ** np.maximum(np.floor(np.log2(np.maximum(np.abs(exact), 1e-30))), -6) / 8
    assert (np.abs(got - exact) <= step * 0.5 + 2.0 ** -22 * np.abs(exact)).all()


def test_append_starts_a_block_with_no_scale_yet(dev):
    """Scales of a pool that was never written: not positive, not finite."""
    for bad in (0.0, -3.0, math.nan, math.inf):
        kc, vc, ks, vs = make_cache(2, 16, 1, 64, 16, 13, dev)
        ks.fill_(bad), vs.fill_(bad)
        k = torch.randn(3, 1, 64, generator=torch.Generator().manual_seed(1)).half().to(dev)
        check_append(dev, k, k.clone(), np.array([5, 6, 7], np.int32), (kc, vc, ks, vs), 16)


# ---- gather
@BOTH
@pytest.mark.parametrize("D,heads,page,block", [(64, 1, 8, 8), (64, 5, 16, 1), (128, 3, 64, 16),
                                                (128, 8, 32, 32)])
@pytest.mark.parametrize("n", [1, 7, 300])
def test_gather(dev, dtype, D, heads, page, block, n):
    kc, vc, ks, vs = make_cache(20, page, heads, D, block, n, dev, "head" if n == 7 else "token")
    g = torch.Generator().manual_seed(n)
    slots = torch.randint(-3, 20 * page, (n + 2,), generator=g, dtype=torch.int32)  # some twice
    k, v = (torch.full((n, heads, D), 7.0, dtype=dtype, device=dev) for _ in range(2))
    st = torch.zeros(1, dtype=torch.int32, device=dev)
    paged_q8.dspark_kv_gather_q8(kc, vc, ks, vs, slots.to(dev), k=k, v=v, device_status=st)
    torch.cuda.synchronize()
    assert int(st.item()) == 0
    s = slots.numpy()[:n]
    for out, c, sc in ((k, kc, ks), (v, vc, vs)):
        want = _q8.numbers(c)[s // page, s % page] * \
            sc.double().cpu().numpy()[s // page, s % page // block][..., None]
        want[s < 0] = 7.0
        assert torch.equal(out.cpu(), torch.from_numpy(want).to(dtype))
    o = paged_q8.dspark_kv_gather_q8(kc, vc, ks, vs, slots.to(dev), dtype=dtype, check=True)
    keep = torch.from_numpy(s >= 0)
    assert torch.equal(o["k"].cpu()[:n][keep], k.cpu()[keep]) and (o["v"].cpu()[:n][~keep] == 0).all()


def test_gather_bad_slot(dev):
    kc, vc, ks, vs = make_cache(2, 16, 1, 64, 16, 1, dev)
    with pytest.raises(paged.DsparkError):
        paged_q8.dspark_kv_gather_q8(kc, vc, ks, vs,
                                     torch.tensor([0, 32], dtype=torch.int32, device=dev), check=True)


def test_no_rows(dev):
    kc, vc, ks, vs = make_cache(2, 16, 1, 64, 16, 1, dev)
    none = torch.zeros(0, dtype=torch.int32, device=dev)
    k = torch.zeros(0, 1, 64, dtype=torch.float16, device=dev)
    before = kc.view(torch.uint8).clone()
    t = paged_q8.RotaryTable(64, device=dev)
    paged_q8.dspark_kv_append_q8(k, k, none, kc, vc, ks, vs, rotary=t, positions=none, check=True)
    assert torch.equal(kc.view(torch.uint8), before)
    assert paged_q8.dspark_kv_gather_q8(kc, vc, ks, vs, none, check=True)["k"].shape == (0, 1, 64)
    assert paged_q8.dspark_rotary(k, none, t)["out"].shape == (0, 1, 64)


@pytest.mark.parametrize("page,block", [(32, 1), (32, 16), (512, 512)])
def test_append_of_rows_with_one_slot_leaves_the_last(dev, page, block):
    """All rows of a block are as large, so the scale is the same whichever rows count."""
    g = torch.Generator().manual_seed(11)
    n = 2 * block + 600 if block > 256 else 300
    k, v = ((torch.randint(1, 8, (n, 3, 64), generator=g) / 4).to(torch.float16) for _ in range(2))
    k[..., 0] = v[..., 0] = 7.0
    slots = (torch.arange(n) // 3 * 2).to(torch.int32)
    slots[torch.randperm(n, generator=g)[:n // 5]] = -1
    slots[200:240] = -1
    pages = int(slots.max()) // page + 1
    cache = make_cache(pages, page, 3, 64, block, 5, dev)
    last = {int(x): i for i, x in enumerate(slots.tolist()) if x >= 0}
    out = paged_q8.dspark_kv_append_q8(k.to(dev), v.to(dev), slots.to(dev), *cache)
    assert int(out["device_status"]) == 0
    rows = torch.tensor(list(last.values()))
    got = paged_q8.dspark_kv_gather_q8(*cache, torch.tensor(list(last), dtype=torch.int32, device=dev),
                                       dtype=torch.float16)
    assert torch.equal(got["k"].cpu(), k[rows]) and torch.equal(got["v"].cpu(), v[rows])
