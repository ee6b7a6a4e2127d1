"""dspark_paged_attention_q8 on the GPU against softmax attention in 64 bits over what the
codes and scales stand for.

Everything in the cache that no row may see, codes and scales, is NaN, so a read of it shows.
The bound of every comparison is _q8.attention's, derived there from the call's arithmetic
before its first run."""
import math

import numpy as np
import pytest
import torch

from speculative_decoding_verification_41_gb300 import build as cuda_build
from speculative_decoding_verification_41_gb300 import paged, paged_q8
from tests import _q8

pytestmark = pytest.mark.gpu


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
    return paged_q8.dspark_paged_attention_q8(
        a.q, a.k_cache, a.v_cache, a.k_scale, a.v_scale, a.table, a.context_len, a.row_off,
        scale=a.scale, max_new=a.max_new, window=a.window, with_lse=True, buffers=buffers, **kw)


def check(a, o=None, rows=None):
    if o is None:
        o = call(a)
    torch.cuda.synchronize()
    assert int(o["device_status"].item()) == 0
    out, lse, tol, lse_tol = _q8.attention(a)
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


BOTH = pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])


@BOTH
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 31, 32, 33, 127, 128, 129, 1000])
def test_one_request(dev, dtype, D, n):
    check(_q8.make_attention([n], [1], 4, 2, D, 16, dtype, seed=n, device=dev))


@BOTH
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("group,new", [(1, 1), (1, 16), (3, 5), (4, 17), (8, 4), (8, 10), (16, 6),
                                       (5, 19), (16, 12), (100, 1), (7, 30)])
def test_rows_of_a_pass(dev, dtype, D, group, new):
    """Every row block, and more rows than one holds."""
    lens, news = [300, new, 131, 700], [new, new, max(1, new // 2), 1]
    check(_q8.make_attention(lens, news, 2 * group, 2, D, 32, dtype, seed=group + new, device=dev))


@BOTH
@pytest.mark.parametrize("page,block", [(8, 1), (8, 8), (16, 2), (32, 32), (64, 16), (128, 64),
                                        (128, 128), (256, 1), (256, 256), (1024, 512)])
@pytest.mark.parametrize("layout", ["token", "head"])
def test_pages_and_blocks(dev, dtype, page, block, layout):
    check(_q8.make_attention([1, 77, 517, 260], [1, 3, 2, 5], 6, 3, 128, page, dtype, block=block,
                             layout=layout, seed=page + block, device=dev, table_pad=3))


@BOTH
@pytest.mark.parametrize("window", [1, 2, 31, 128, 200, 5000])
def test_window(dev, dtype, window):
    check(_q8.make_attention([5, 640, 333, 90], [3, 9, 1, 9], 8, 2, 64, 16, dtype, block=4,
                             window=window, seed=window, device=dev))


@BOTH
def test_no_rows_no_tokens(dev, dtype):
    """Requests without new tokens, without a cached one, and rows that see none."""
    a = _q8.make_attention([0, 40, 2, 0, 150], [2, 0, 4, 0, 1], 4, 2, 128, 16, dtype, seed=3,
                           device=dev)
    o = check(a)
    out = o["out"].float()
    assert (out[:4] == 0).all() and (out[4:6].abs().sum(-1) > 0).all()


@BOTH
def test_long_context_many_ctas(dev, dtype):
    """A request cut among all the CTAs, and joined."""
    check(_q8.make_attention([20011], [2], 8, 2, 128, 64, dtype, seed=5, device=dev))


@BOTH
def test_many_ragged_requests(dev, dtype):
    rng = np.random.default_rng(1)
    lens = rng.integers(0, 400, 190).tolist()
    news = [min(int(rng.integers(0, 4)), n) for n in lens]
    check(_q8.make_attention(lens, news, 4, 2, 64, 8, dtype, block=2, seed=6, device=dev))


@BOTH
@pytest.mark.parametrize("gain", [0.0, 6.0, 40.0])
def test_sharp_and_flat_scores(dev, dtype, gain):
    """From equal weights to one weight that is all."""
    check(_q8.make_attention([700, 260], [3, 1], 8, 2, 128, 16, dtype, q_gain=gain, seed=7,
                             device=dev))


@BOTH
@pytest.mark.parametrize("spread", [8, 40])
def test_scales_far_apart(dev, dtype, spread):
    check(_q8.make_attention([900, 300], [2, 5], 4, 2, 128, 16, dtype, spread=spread, seed=spread,
                             device=dev, q_gain=1.0 if spread < 10 else 0.02))


@BOTH
def test_scales_that_are_no_powers_of_two(dev, dtype):
    check(_q8.make_attention([900, 300], [2, 5], 4, 2, 128, 16, dtype, exact_scales=False, seed=8,
                             device=dev))


@BOTH
def test_rising_scores(dev, dtype):
    """Scores that grow along the context: the reference is raised tile by tile."""
    a = _q8.make_attention([2000], [1], 2, 1, 64, 16, dtype, seed=9, spread=0, device=dev)
    pos = torch.arange(2000, device=dev)
    page = a.table[0, pos // 16].long()
    k = torch.zeros(2000, 64, device=dev)
    k[:, 0] = pos / 5.0
    a.k_cache[page, pos % 16, 0] = k.to(_q8.E4M3)
    a.k_scale[page, pos % 16 // 16, 0] = 0.25
    a.q.zero_()
    a.q[..., 0] = 8.0
    check(a)


@BOTH
def test_a_sink_does_not_cost_the_others_their_bits(dev, dtype):
    """One token 12 nats above all others, whose value is nothing: the output is the others'."""
    a = _q8.make_attention([2000], [1], 4, 1, 128, 16, dtype, seed=10, spread=0, q_gain=0.0,
                           device=dev)
    a.q[..., 0] = 1.0
    p0 = int(a.table[0, 0])
    a.k_cache[:, :, :, 0] = 0
    a.k_cache[p0, 0, 0, 0] = 256.0
    a.k_scale[p0, 0, 0] = 12 / (256.0 * a.scale)
    a.v_cache[p0, 0, 0] = 0
    o = call(a)
    torch.cuda.synchronize()
    out, _, _, _ = _q8.attention(a)
    got = o["out"].double().cpu().numpy()
    err = np.linalg.norm(got - out) / np.linalg.norm(out)
    # weights of 9 bits cut about their middle (2^-9 at most, but for the low end's own) and
    # the output's rounding
    assert err < (2.0 ** -7 if dtype == torch.bfloat16 else 2.0 ** -9)


@BOTH
@pytest.mark.parametrize("code", [0x7F, 0xFF])
def test_nan_of_a_value_reaches_those_who_see_it(dev, dtype, code):
    """A NaN in the last tokens' values belongs to the new tokens that see it."""
    a = _q8.make_attention([200], [4], 2, 1, 128, 16, dtype, seed=11, device=dev)
    at = 198  # seen by the last two
    page = int(a.table[0, at // 16])
    a.v_cache.view(torch.uint8)[page, at % 16, 0, 5] = code
    o = call(a)
    torch.cuda.synchronize()
    out = o["out"].float().cpu()
    nan = out.isnan()
    assert nan[2:, :, 5].all() and int(nan.sum()) == 4
    a.v_cache.view(torch.uint8)[page, at % 16, 0, 5] = 0
    clean = call(a)
    torch.cuda.synchronize()
    assert torch.equal(out[:2], clean["out"].float().cpu()[:2])


@BOTH
def test_nan_of_a_key_and_a_query(dev, dtype):
    a = _q8.make_attention([200], [4], 2, 1, 64, 16, dtype, seed=12, device=dev)
    at = 198
    page = int(a.table[0, at // 16])
    a.k_cache.view(torch.uint8)[page, at % 16, 0, 7] = 0x7F
    a.q[0, 1, 3] = math.inf
    o = call(a)
    torch.cuda.synchronize()
    out = o["out"].float().cpu()
    assert out[2:].isnan().all() and out[0, 1].isnan().all()
    assert not out[0, 0].isnan().any() and not out[1].isnan().any()


@pytest.mark.parametrize("bad", [0.0, -1.0, math.nan, math.inf])
@pytest.mark.parametrize("which", ["k_scale", "v_scale"])
def test_bad_scale_is_reported(dev, bad, which):
    a = _q8.make_attention([100, 50], [1, 1], 2, 1, 64, 16, torch.bfloat16, seed=13, device=dev)
    getattr(a, which)[int(a.table[0, 2]), 0, 0] = bad
    o = call(a)
    torch.cuda.synchronize()
    assert int(o["device_status"].item()) == 5
    good, _, tol, _ = _q8.attention(a)
    assert (np.abs(o["out"][1].double().cpu().numpy() - good[1]) <= tol[1]).all()


def test_bad_page_is_reported(dev):
    a = _q8.make_attention([100, 50], [1, 1], 2, 1, 64, 16, torch.bfloat16, seed=14, device=dev)
    for page in (-1, a.k_cache.shape[0]):
        a.table[0, 3] = page
        o = call(a)
        torch.cuda.synchronize()
        assert int(o["device_status"].item()) == 5


def test_bad_lengths_are_reported(dev):
    a = _q8.make_attention([100, 50], [1, 1], 2, 1, 64, 16, torch.bfloat16, seed=15, device=dev)
    for n in (-1, 10 ** 6):
        a.context_len[1] = n
        o = call(a)
        torch.cuda.synchronize()
        assert int(o["device_status"].item()) == 5


@BOTH
def test_same_every_time_and_captured(dev, dtype):
    a = _q8.make_attention([5000, 300, 77], [2, 9, 1], 8, 2, 128, 16, dtype, seed=16, device=dev)
    n, Hq, D = a.q.shape
    b = paged.AttentionBuffers(n, Hq, 2, D, a.max_new, a.q.dtype, dev, with_lse=True)
    o = call(a, b)
    first, lse = o["out"].clone(), o["lse"].clone()
    for _ in range(3):
        call(a, b)
        torch.cuda.synchronize()
        assert torch.equal(first, b.out) and torch.equal(lse, b.lse)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(a, b)
    b.out.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(first, b.out) and torch.equal(lse, b.lse)


def test_strided_queries_and_other_streams(dev):
    a = _q8.make_attention([150, 90], [2, 3], 4, 2, 64, 16, torch.bfloat16, seed=17, device=dev)
    wide = torch.full((5, 12, 64), math.nan, dtype=torch.bfloat16, device=dev)
    wide[:, 2:6] = a.q
    want = call(a)["out"].clone()
    a.q = wide[:, 2:6]
    side = torch.cuda.Stream(device=dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    o = paged_q8.dspark_paged_attention_q8(
        a.q, a.k_cache, a.v_cache, a.k_scale, a.v_scale, a.table, a.context_len, a.row_off,
        scale=a.scale, max_new=a.max_new, stream=side, check=True)
    assert torch.equal(o["out"], want) and o["lse"] is None


def test_rows_outside_requests_stay(dev):
    a = _q8.make_attention([150, 90], [2, 3], 4, 2, 64, 16, torch.bfloat16, seed=18, device=dev)
    more = torch.zeros(9, 4, 64, dtype=torch.bfloat16, device=dev)
    more[2:7] = a.q
    a.q, a.row_off = more, a.row_off + 2
    b = paged.AttentionBuffers(9, 4, 2, 64, a.max_new, torch.bfloat16, dev, with_lse=True)
    b.out.fill_(7.0)
    call(a, b)
    torch.cuda.synchronize()
    assert (b.out[:2] == 7).all() and (b.out[7:] == 7).all()
    check(a, {"out": b.out, "lse": b.lse, "device_status": b.device_status}, np.arange(2, 7))
