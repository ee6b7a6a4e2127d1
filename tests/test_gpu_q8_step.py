"""The serving step on the 8-bit cache with rotary positions (paged_step.py): reservation, append,
rotary, attention, verification and roll back together, eager and as a replayed graph."""
import numpy as np
import pytest
import torch

from speculative_decoding_verification_41_gb300 import paged_q8, paged_step
from speculative_decoding_verification_41_gb300 import build as cuda_build
from tests import _q8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    cuda_build.build()
    return torch.device("cuda:0")


@pytest.mark.parametrize("block", [1, 8, 16])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_steps_against_the_whole_history(dev, block, dtype):
    """Every step: the stored tokens against the turned keys and the values of the whole history,
    the attention against 64 bits over what is stored."""
    B, gamma, V, ps, D = 6, 4, 512, 16, 64
    g = torch.Generator(device=dev).manual_seed(3)
    table = paged_q8.RotaryTable(48, interleaved=block == 8, device=dev)
    target = paged_step.ToyTarget(V, 8, 2, D, dtype=dtype, device=dev)
    cache = paged_step.PagedCache(B, 64, ps, 8, 2, D, gamma + 1, device=dev, block=block,
                                  rotary=table)
    anchors = torch.randint(0, V, (B,), generator=g, device=dev, dtype=torch.int32)
    history = [[] for _ in range(B)]
    taken = {}
    attend = cache.attend

    def spy(q):
        out = attend(q)
        taken.update(out=out.clone(), q=q.clone(), pos=cache.rows.positions.clone(),
                     a=_q8.Attention(cache._turned.clone(), cache.k.clone(), cache.v.clone(),
                                     cache.block_table.clone(), cache.rows.context_len.clone(),
                                     cache.rows.row_off.clone(), D ** -0.5, gamma + 1, 0,
                                     *(s.clone() for s in cache.scales)))
        return out

    cache.attend = spy
    u = torch.finfo(dtype).eps / 2
    for step in range(8):
        draft = torch.randint(0, V, (B, gamma), generator=g, device=dev, dtype=torch.int32)
        dl = torch.randn(B, gamma, V, generator=g, device=dev).to(torch.bfloat16)
        ell = torch.randint(0, gamma + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        uni = torch.rand(B, gamma + 1, generator=g, device=dev)
        def logits(attended):
            # (the verification takes bf16)
            return (attended.flatten(1) @ target.head).to(torch.bfloat16)

        target.logits = logits
        out = paged_step.speculative_step(cache, target, anchors, draft, dl, ell, uni, 1.0)
        torch.cuda.synchronize()
        assert cache.statuses() == [0, 0, 0, 0]
        a = taken["a"]
        n = int(a.row_off[-1])
        # the queries, turned: binary32, rounded once
        pos = taken["pos"].cpu().numpy()
        q = taken["q"].double().cpu().numpy()[:n]
        want = _q8.turned(q, pos[:n], table.angles, interleaved=table.interleaved)
        size = np.abs(q).max(-1, keepdims=True)
        off = np.abs(a.q.double().cpu().numpy()[:n] - want)
        assert (off <= 1.01 * u * np.abs(want) + 2.0 ** -19 * size + 2.0 ** -25).all()
        # the attention
        want, _, tol, _ = _q8.attention(a)
        off = np.abs(taken["out"].double().cpu().numpy() - want)[:n]
        assert (off <= tol[:n]).all()
        # What is stored. A token is rounded once, half a step of 2^-4 of it, and again when its
        # block's scale rises: to powers of two, so that only codes below the normal ones lose,
        # half of 2^-9 of each scale, twice that of the last in all. Turning: 2^-19 of the head.
        ctx, row_off = a.context_len.cpu().tolist(), a.row_off.cpu().tolist()
        bt = a.table.cpu().numpy()
        l, m = ell.cpu().numpy(), out["accepted_len"].cpu().numpy()
        for r in range(B):
            seq = history[r] + [int(anchors[r])] + draft[r, :l[r]].tolist()
            assert ctx[r] == len(seq) and row_off[r + 1] - row_off[r] == l[r] + 1
            p = np.arange(len(seq))
            assert (pos[row_off[r]:row_off[r + 1]] == p[len(history[r]):]).all()
            _, k, v = (x.double().cpu().numpy() for x in target.qkv(torch.tensor(seq, device=dev)))
            k = _q8.turned(k, p, table.angles, interleaved=table.interleaved)
            for x, codes, scale in ((k, a.k_cache, a.k_scale), (v, a.v_cache, a.v_scale)):
                page = bt[r][p // ps]
                s = scale.double().cpu().numpy()[page, p % ps // block][..., None]
                got = _q8.numbers(codes)[page, p % ps] * s
                big = np.abs(x).max(-1, keepdims=True)
                bound = 2.0 ** -4 * np.abs(x) + 2.0 ** -9 * s + 2.0 ** -18 * big
                assert (np.abs(got - x) <= bound).all()
            history[r] += [int(anchors[r])] + draft[r, :m[r]].tolist()
        assert cache.context_len.cpu().tolist() == [len(h) for h in history]
        anchors = out["next_anchors"].contiguous()
    # what is stored, read back by slots
    r = int(np.argmax([len(h) for h in history]))
    p = np.arange(len(history[r]))
    slots = torch.from_numpy((cache.block_table[r].cpu().numpy()[p // ps] * ps + p % ps)
                             .astype(np.int32)).to(dev)
    k, v = cache.stored(slots, dtype)
    for got, codes, scale in ((k, cache.k, cache.scales[0]), (v, cache.v, cache.scales[1])):
        page = slots.cpu().numpy() // ps
        want = (_q8.numbers(codes)[page, p % ps]
                * scale.double().cpu().numpy()[page, p % ps // block][..., None])
        assert np.array_equal(got.double().cpu().numpy(),
                              torch.from_numpy(want).to(dtype).double().numpy())


def test_a_captured_step_replays(dev):
    """One step captured in a CUDA graph, replayed on new drafts and lengths: the outputs, codes and
    scales of the same steps run one by one."""
    B, gamma, V = 5, 3, 256
    table = paged_q8.RotaryTable(64, scaling="yarn", factor=4.0, original_len=512, device=dev)

    def fresh():
        target = paged_step.ToyTarget(V, 4, 2, 64, seed=4, device=dev)
        return target, paged_step.PagedCache(B, 40, 8, 8, 2, 64, gamma + 1, device=dev, block=8,
                                             rotary=table)

    g = torch.Generator(device=dev).manual_seed(5)
    steps = [dict(anchors=torch.randint(0, V, (B,), generator=g, device=dev, dtype=torch.int32),
                  draft_tokens=torch.randint(0, V, (B, gamma), generator=g, device=dev,
                                             dtype=torch.int32),
                  draft_logits=torch.randn(B, gamma, V, generator=g, device=dev).to(torch.bfloat16),
                  verify_len=torch.randint(0, gamma + 1, (B,), generator=g, device=dev,
                                           dtype=torch.int32),
                  uniforms=torch.rand(B, gamma + 1, generator=g, device=dev)) for _ in range(6)]

    def state(cache):
        return [cache.context_len, cache.free_pages, cache.free_count, cache.block_table,
                cache.k.view(torch.uint8), cache.v.view(torch.uint8), *cache.scales]

    target, cache = fresh()
    want = []
    for s in steps:
        o = paged_step.speculative_step(cache, target, temperature=1.0, **s)
        torch.cuda.synchronize()
        assert cache.statuses() == [0, 0, 0, 0]
        want.append([o["emitted_tokens"].clone()] + [t.clone() for t in state(cache)])
    target, cache = fresh()
    slots = {k: v.clone() for k, v in steps[0].items()}
    side = torch.cuda.Stream(dev)
    side.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(side):  # first calls, cuBLAS's among them, outside the capture
        paged_step.speculative_step(cache, target, temperature=1.0, **slots)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = paged_step.speculative_step(cache, target, temperature=1.0, **slots)
    for t, s in zip(state(cache), state(fresh()[1])):
        t.copy_(s)
    for s, w in zip(steps, want):
        for k, v in s.items():
            slots[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        for got, x in zip([out["emitted_tokens"]] + state(cache), w):
            assert torch.equal(got, x)


def test_rotary_on_the_16_bit_cache(dev):
    """The same turned keys and attention through the calls of their own."""
    table = paged_q8.RotaryTable(64, device=dev)
    g = torch.Generator(device=dev).manual_seed(6)
    q, k, v = (torch.randn(6, h, 64, generator=g, device=dev).to(torch.bfloat16) for h in (8, 2, 2))
    caches = [paged_step.PagedCache(2, 8, 16, 4, 2, 64, 3, device=dev, rotary=r)
              for r in (table, None)]
    new = torch.tensor([2, 1], dtype=torch.int32, device=dev)
    outs = []
    for c in caches:
        rows = c.reserve(new)
        if c.rotary is None:
            kk, qq = (paged_q8.dspark_rotary(x, rows["positions"], table)["out"] for x in (k, q))
        else:
            kk, qq = k, q
        c.append(kk, v)
        outs.append((c.attend(qq)[:5].clone(), c.stored(c.rows.slot_map[:5])))
        assert c.statuses() == [0, 0, 0, 0]
    assert torch.equal(outs[0][0], outs[1][0])
    assert all(torch.equal(a, b) for a, b in zip(outs[0][1], outs[1][1]))


def test_demo(dev):
    got = paged_step.demo(steps=4, block=16, rotary=paged_q8.RotaryTable(64, device=dev))
    assert got["statuses"] == [0, 0, 0, 0]
    assert got["tokens"] == got["cached"] >= 4 * 32
    assert got["pages_held"] + got["pages_free"] == 32 * 8


def test_refusals(dev):
    for block in (-1, 3, 32):
        with pytest.raises(ValueError, match="block"):
            paged_step.PagedCache(1, 4, 16, 2, 2, 64, 2, device=dev, block=block)
