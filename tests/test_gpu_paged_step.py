"""The serving step on a paged cache (paged_step.py): the calls together, as a
serving loop uses them. Every step's logits are checked against attention over
the whole kept history in 64 bits, the verification against the oracle on those
logits, and the pages' books after every step."""
import numpy as np
import pytest
import torch

import oracle
from speculative_decoding_verification_41_gb300 import binding, paged_step, workloads
from speculative_decoding_verification_41_gb300 import build as cuda_build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    cuda_build.build()
    return torch.device("cuda:0")


def books(cache, page_size):
    """Every page is held once or free once."""
    ctx = cache.context_len.cpu().numpy()
    table = cache.block_table.cpu().numpy()
    held = [int(table[r, j]) for r in range(len(ctx)) for j in range(-(-int(ctx[r]) // page_size))]
    free = cache.free_pages[:int(cache.free_count.item())].cpu().tolist()
    assert sorted(held + free) == list(range(cache.k.shape[0]))


def history_logits(target, tokens):
    """Logits of the last position of `tokens` in 64 bits, with the layer's roundings of q, k, v
    to bf16 (they are what the cache holds)."""
    q, k, v = (x.double().cpu() for x in target.qkv(torch.tensor(tokens, device="cuda")))
    G = target.Hq // target.Hkv
    o = []
    for h in range(target.Hq):
        z = k[:, h // G] @ q[-1, h] * target.D ** -0.5
        o.append(torch.softmax(z, 0) @ v[:, h // G])
    return torch.stack(o).flatten().numpy()


def test_steps_against_the_whole_history(dev):
    B, gamma, V, ps = 6, 4, 512, 16
    g = torch.Generator(device=dev).manual_seed(3)
    target = paged_step.ToyTarget(V, 8, 2, 64, device=dev)
    cache = paged_step.PagedCache(B, 64, ps, 8, 2, 64, gamma + 1, device=dev)
    anchors = torch.randint(0, V, (B,), generator=g, device=dev, dtype=torch.int32)
    history = [[] for _ in range(B)]
    taken = {}
    attend = cache.attend

    def spy(q):
        out = attend(q)
        taken["out"] = out.clone()
        taken["row_off"] = cache.rows.row_off.clone()
        return out

    cache.attend = spy
    half_step = torch.finfo(torch.bfloat16).eps / 2
    for step in range(7):
        draft = torch.randint(0, V, (B, gamma), generator=g, device=dev, dtype=torch.int32)
        dl = torch.randn(B, gamma, V, generator=g, device=dev).to(torch.bfloat16)
        ell = torch.randint(0, gamma + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        u = torch.rand(B, gamma + 1, generator=g, device=dev)
        out = paged_step.speculative_step(cache, target, anchors, draft, dl, ell, u, 1.0)
        torch.cuda.synchronize()
        assert cache.statuses() == [0, 0, 0, 0]
        off = taken["row_off"].cpu().numpy()
        attended = taken["out"].double().cpu().numpy()
        logits = target.logits(taken["out"])
        l, m = ell.cpu().numpy(), out["accepted_len"].cpu().numpy()
        vmax = float(cache.v.float().abs().max())
        for r in range(B):
            seq = history[r] + [int(anchors[r])] + draft[r, :l[r]].tolist()
            for j in range(l[r] + 1):
                want = history_logits(target, seq[:len(history[r]) + 1 + j])
                got = attended[off[r] + j].ravel()
                # weights and the result are rounded to bf16 once each; binary32 sums: far less
                assert np.abs(got - want).max() <= 2.1 * half_step * vmax
        t_off = torch.from_numpy(off).to(dev)
        ref = oracle.verify(workloads.bf16_bits(logits.cpu()),
                            workloads.bf16_bits(dl.reshape(B * gamma, V).cpu()),
                            draft.cpu().numpy(), l, u.cpu().numpy(), 1.0, off,
                            np.arange(B + 1, dtype=np.int64) * gamma)
        sure = ~ref["flags"].any(axis=1)
        assert np.array_equal(m[sure], ref["accepted_len"][sure])
        assert np.array_equal(out["emitted_tokens"].cpu().numpy()[sure], ref["emitted"][sure])
        for r in range(B):
            history[r] += [int(anchors[r])] + draft[r, :m[r]].tolist()
        assert cache.context_len.cpu().tolist() == [len(h) for h in history]
        books(cache, ps)
        anchors = out["emitted_tokens"].gather(1, out["accepted_len"].long()[:, None])[:, 0].contiguous()
    finish = torch.full((B,), -1, dtype=torch.int32, device=dev)
    cache.reserve(torch.zeros(B, dtype=torch.int32, device=dev), extra=0)
    cache.release(finish, extra=0)
    torch.cuda.synchronize()
    assert int(cache.free_count.item()) == 64 and cache.context_len.abs().sum().item() == 0
    del t_off


def test_a_captured_step_replays(dev):
    """One step captured in a CUDA graph, replayed on new drafts and lengths: the outputs and the
    books of the same steps run one by one."""
    B, gamma, V = 5, 3, 256

    def fresh():
        target = paged_step.ToyTarget(V, 4, 2, 64, seed=4, device=dev)
        return target, paged_step.PagedCache(B, 40, 8, 8, 2, 64, gamma + 1, device=dev)

    g = torch.Generator(device=dev).manual_seed(5)
    steps = [dict(anchors=torch.randint(0, V, (B,), generator=g, device=dev, dtype=torch.int32),
                  draft_tokens=torch.randint(0, V, (B, gamma), generator=g, device=dev,
                                             dtype=torch.int32),
                  draft_logits=torch.randn(B, gamma, V, generator=g, device=dev).to(torch.bfloat16),
                  verify_len=torch.randint(0, gamma + 1, (B,), generator=g, device=dev,
                                           dtype=torch.int32),
                  uniforms=torch.rand(B, gamma + 1, generator=g, device=dev)) for _ in range(6)]
    target, cache = fresh()
    want = []
    for s in steps:
        o = paged_step.speculative_step(cache, target, temperature=1.0, **s)
        torch.cuda.synchronize()
        want.append((o["emitted_tokens"].clone(), cache.context_len.clone(),
                     cache.free_pages.clone(), cache.free_count.clone()))
    target, cache = fresh()
    slots = {k: v.clone() for k, v in steps[0].items()}
    side = torch.cuda.Stream(dev)
    with torch.cuda.stream(side):  # first calls, cuBLAS's among them, outside the capture
        paged_step.speculative_step(cache, target, temperature=1.0, **slots)
    side.synchronize()
    state = [cache.context_len, cache.free_pages, cache.free_count, cache.block_table]
    start = paged_step.PagedCache(B, 40, 8, 8, 2, 64, gamma + 1, device=dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = paged_step.speculative_step(cache, target, temperature=1.0, **slots)
    for t, s in zip(state, [start.context_len, start.free_pages, start.free_count,
                            start.block_table]):
        t.copy_(s)
    for s, (em, ctx, free, count) in zip(steps, want):
        for k, v in s.items():
            slots[k].copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out["emitted_tokens"], em) and torch.equal(cache.context_len, ctx)
        assert torch.equal(cache.free_pages, free) and torch.equal(cache.free_count, count)


def test_demo(dev):
    got = paged_step.demo(steps=4)
    assert got["statuses"] == [0, 0, 0, 0]
    assert got["tokens"] == got["cached"] >= 4 * 32
    assert got["pages_held"] + got["pages_free"] == 32 * 8
