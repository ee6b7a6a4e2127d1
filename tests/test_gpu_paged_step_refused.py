"""Serving steps on a pool that is too small: requests that the reservation refuses keep their place
(anchor, history, pages) and go on from it when pages are free again."""
import numpy as np
import pytest
import torch

import oracle
from speculative_decoding_verification_41_gb300 import build as cuda_build
from speculative_decoding_verification_41_gb300 import paged, paged_step, workloads
from tests.test_gpu_paged_step import books, history_logits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    cuda_build.build()
    return torch.device("cuda:0")


def test_refused_requests_keep_their_place(dev):
    B, gamma, V, ps, pages = 4, 4, 512, 8, 7
    g = torch.Generator(device=dev).manual_seed(11)
    target = paged_step.ToyTarget(V, 8, 2, 64, device=dev)
    cache = paged_step.PagedCache(B, pages, ps, 6, 2, 64, gamma + 1, device=dev)
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
    waiting, came_back = set(), 0
    for _ in range(24):
        draft = torch.randint(0, V, (B, gamma), generator=g, device=dev, dtype=torch.int32)
        dl = torch.randn(B, gamma, V, generator=g, device=dev).to(torch.bfloat16)
        ell = torch.randint(0, gamma + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        u = torch.rand(B, gamma + 1, generator=g, device=dev)
        before = anchors.cpu().tolist()
        out = paged_step.speculative_step(cache, target, anchors, draft, dl, ell, u, 1.0)
        torch.cuda.synchronize()
        off = taken["row_off"].cpu().numpy()
        served = out["served"].cpu().numpy()
        l, m = ell.cpu().numpy(), out["accepted_len"].cpu().numpy()
        assert np.array_equal(np.diff(off), np.where(served, l + 1, 0))
        assert int(out["reserve_status"].item()) == (0 if served.all() else paged.DSPARK_ERR_NO_PAGES)
        anchors = out["next_anchors"]
        nxt, emitted = anchors.cpu().tolist(), out["emitted_tokens"].cpu().numpy()
        attended = taken["out"].double().cpu().numpy()
        vmax = float(cache.v.float().abs().max())
        for r in np.flatnonzero(served):
            seq = history[r] + [before[r]] + draft[r, :l[r]].tolist()
            for j in range(l[r] + 1):
                want = history_logits(target, seq[:len(history[r]) + 1 + j])
                # weights and the result are rounded to bf16 once each; binary32 sums: far less
                assert np.abs(attended[off[r] + j].ravel() - want).max() <= 2.1 * half_step * vmax
            assert nxt[r] == emitted[r, m[r]] >= 0
            history[r] += [before[r]] + draft[r, :m[r]].tolist()
        idx = np.flatnonzero(served)
        if len(idx):
            ref = oracle.verify(
                workloads.bf16_bits(target.logits(taken["out"]).cpu()),
                workloads.bf16_bits(dl[torch.from_numpy(idx).to(dev)].reshape(-1, V).cpu()),
                draft.cpu().numpy()[idx], l[idx], u.cpu().numpy()[idx], 1.0,
                np.append(off[idx], off[-1]), np.arange(len(idx) + 1, dtype=np.int64) * gamma)
            sure = ~ref["flags"].any(axis=1)
            assert np.array_equal(m[idx][sure], ref["accepted_len"][sure])
            assert np.array_equal(emitted[idx][sure], ref["emitted"][sure])
        for r in np.flatnonzero(~served):
            assert nxt[r] == before[r] and m[r] == 0 and (emitted[r] == -1).all()
        came_back += len(waiting & set(idx.tolist()))
        waiting = set(np.flatnonzero(~served).tolist())
        assert cache.context_len.cpu().tolist() == [len(h) for h in history]
        books(cache, ps)
        if waiting:  # the longest request ends, and another takes its place
            r = max(range(B), key=lambda i: len(history[i]))
            kept = torch.zeros(B, dtype=torch.int32, device=dev)
            kept[r] = -1
            cache.reserve(torch.zeros(B, dtype=torch.int32, device=dev), extra=0)
            cache.release(kept, extra=0)
            history[r] = []
            books(cache, ps)
    assert came_back >= 3
