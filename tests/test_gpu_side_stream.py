"""Calls on another stream than the current one that allocate for themselves: nothing that is still
queued on the current stream writes their outputs, workspace or status after them."""
import numpy as np
import pytest
import torch

from speculative_decoding_verification_41_gb300 import build as cuda_build
from speculative_decoding_verification_41_gb300 import binding, paged, workloads
from tests import _paged

pytestmark = pytest.mark.gpu

CYCLES = 100_000_000  # some 50 ms of work on the current stream


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    cuda_build.build()
    return torch.device("cuda:0")


def behind(dev, call, sizes=()):
    """call(side) while the current stream is busy: behind a long kernel it has still to write to
    blocks of `sizes` bytes that the allocator has back already. The call's results once all of it
    is done."""
    side = torch.cuda.Stream(dev)
    call(side)  # what a first call sets up
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    freed = [torch.zeros(n, dtype=torch.uint8, device=dev) for n in sizes]
    torch.cuda.synchronize()
    torch.cuda._sleep(CYCLES)
    for t in freed:
        t.fill_(0x55)
    del freed, t
    out = call(side)
    side.synchronize()
    torch.cuda.synchronize()
    return out


def test_paged_statuses_survive(dev):
    """Bad data, found on the side stream, is not zeroed by the current one."""
    i32 = dict(dtype=torch.int32, device=dev)
    ctx, new = torch.tensor([5, -1], **i32), torch.tensor([2, 2], **i32)
    table, stack, count = torch.zeros(2, 4, **i32), torch.arange(8, **i32), torch.tensor([8], **i32)
    cache = torch.zeros(8, 16, 2, 64, dtype=torch.bfloat16, device=dev)
    rows = torch.ones(2, 2, 64, dtype=torch.bfloat16, device=dev)
    q = torch.ones(2, 4, 64, dtype=torch.bfloat16, device=dev)
    bad_slots, off = torch.tensor([3, 8 * 16], **i32), torch.tensor([0, 1, 2], device=dev)
    calls = [
        lambda s: paged.dspark_pages_reserve(ctx, new, table, stack, count, page_size=16,
                                             max_tokens=8, stream=s),
        lambda s: paged.dspark_pages_release(ctx, ctx, new, table, stack, count,
                                             page_size=16, stream=s),
        lambda s: paged.dspark_kv_append(rows, rows, bad_slots, cache, cache, stream=s),
        lambda s: paged.dspark_paged_attention(q, cache, cache, table, ctx, off, scale=0.125,
                                               max_new=1, stream=s)]
    for call in calls:
        o = behind(dev, call, [512] * 6)
        assert int(o["device_status"].item()) == _paged.BAD_DATA


def test_paged_outputs_survive(dev):
    a = _paged.make_attention([300, 17, 900], [2, 1, 2], 8, 2, 128, 32, torch.bfloat16, seed=8,
                              device=dev)
    args = (a.q, a.k_cache, a.v_cache, a.table, a.context_len, a.row_off)
    opts = dict(scale=a.scale, max_new=a.max_new, with_lse=True)
    want = paged.dspark_paged_attention(*args, **opts)
    ws = paged.paged_attention_workspace_bytes(8, 2, a.max_new, 128)
    o = behind(dev, lambda s: paged.dspark_paged_attention(*args, **opts, stream=s),
               [ws, want["out"].numel() * 2, want["lse"].numel() * 4])
    assert torch.equal(o["out"], want["out"]) and torch.equal(o["lse"], want["lse"])

    rng = np.random.default_rng(2)
    B, ps = 50, 16
    ctx = torch.tensor(rng.integers(0, 90, B), dtype=torch.int32, device=dev)
    new = torch.tensor(rng.integers(0, 17, B), dtype=torch.int32, device=dev)
    table = torch.zeros(B, 8, dtype=torch.int32, device=dev)
    stack = torch.arange(400, dtype=torch.int32, device=dev)
    count = torch.tensor([400], dtype=torch.int32, device=dev)
    call = lambda s: paged.dspark_pages_reserve(ctx, new, table, stack, count, page_size=ps,
                                                max_tokens=900, extra=1, stream=s)
    want = call(None)
    torch.cuda.synchronize()
    o = behind(dev, call, [4 * B, 8 * B + 8, 8 * B + 8, 3600, 3600, 4, 4])
    assert all(torch.equal(o[k], want[k]) for k in want)


def test_the_method_s_calls(dev):
    """The verification, its rates, the scheduler's calls and the drafter: on sound inputs the
    outputs of the same call on the current stream, on bad ones its status."""
    t = workloads.make_tiny(dev)
    bad_len = t.verify_len.clone()
    bad_len[1] = t.gamma + 3
    conf = torch.from_numpy(workloads.make_confidences(8, 4, seed=3)).to(dev)
    bad_conf = conf.clone()
    bad_conf[2, 1] = float("nan")
    T = torch.from_numpy(workloads.step_time_profile(8 * 5 + 1, base_ms=1.0, slope_ms=0.05)).to(dev)
    d = workloads.make_markov_draft(3, 4, 1000, 64, temperature=0.7, seed=1, device=dev)
    bad_anchors = d.anchors.clone()
    bad_anchors[0] = -1
    K = torch.tensor([9], dtype=torch.int32, device=dev)

    def verify(ell):
        return lambda s: binding.dspark_verify(t.target_logits, t.draft_logits, t.draft_tokens,
                                               ell, t.uniforms, t.temperature, stream=s)

    def rates(ell):
        return lambda s: binding.dspark_acceptance(t.target_logits, t.draft_logits, ell,
                                                   t.temperature, t.gamma, stream=s)

    def draft(anchors):
        return lambda s: binding.dspark_draft_markov(d.base_logits, d.w1, d.w2t, anchors,
                                                     d.uniforms, d.temperature, stream=s)

    pairs = [(verify(t.verify_len), verify(bad_len)), (rates(t.verify_len), rates(bad_len)),
             (draft(d.anchors), draft(bad_anchors))]
    pairs += [(lambda s, c=c: c(conf, s), lambda s, c=c: c(bad_conf, s)) for c in (
        lambda x, s: binding.dspark_schedule(x, T, stream=s),
        lambda x, s: binding.dspark_schedule_capacity(x, T, stream=s),
        lambda x, s: binding.dspark_schedule_topk(x, K, stream=s),
        lambda x, s: binding.dspark_schedule_threshold(x, 0.5, stream=s))]
    sizes = [512] * 8 + [binding.verify_workspace_bytes(t.B, t.gamma, 32),
                         binding.acceptance_workspace_bytes(t.B, t.gamma, 32),
                         binding.draft_workspace_bytes(3, 64, 1000), 24000]
    written = {"accepted_len", "emitted_tokens", "probs", "rates", "draft_logits", "draft_tokens",
               "verify_len"}
    for good, bad in pairs:
        want = good(None)
        torch.cuda.synchronize()
        o = behind(dev, good, sizes)
        assert int(o["device_status"].item()) == 0
        assert any(k in written for k in o)
        assert all(torch.equal(o[k], want[k]) for k in o if k in written)
        want = int(bad(None)["device_status"].item())
        assert want != 0
        assert int(behind(dev, bad, sizes)["device_status"].item()) == want
