"""Tensors of another shape than the paged calls', with as many elements: refused with given buffers
as without, before anything is launched."""
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


def others(t):
    """t's elements in other shapes."""
    return [t[None], t[..., None]] + ([t.flatten(), t.transpose(0, 1).contiguous()]
                                      if t.dim() > 1 else [t.reshape(2, -1)] if t.numel() % 2 == 0
                                      else [t[0]] if t.numel() == 1 else [])


def test_inputs(dev):
    B, tokens = 4, 40
    i32 = dict(dtype=torch.int32, device=dev)
    ctx, new, table = torch.tensor([3, 0, 20, 16], **i32), torch.full((B,), 3, **i32), torch.zeros(B, 3, **i32)
    stack, count = torch.arange(20, **i32), torch.tensor([14], **i32)
    reserve, release = [ctx, new, table, stack, count], [ctx, ctx + 3, new, table, stack, count]
    a = _paged.make_attention([50, 300], [2, 1], 4, 2, 64, 16, torch.bfloat16, seed=1, device=dev)
    attend = [a.q, a.k_cache, a.v_cache, a.table, a.context_len, a.row_off]
    for fn, args, which, opts, make in (
            (paged.dspark_pages_reserve, reserve, (0, 1, 2, 4),
             dict(page_size=16, max_tokens=tokens), lambda: paged.ReserveBuffers(B, tokens, dev)),
            (paged.dspark_pages_release, release, (0, 1, 2, 3, 5), dict(page_size=16),
             lambda: paged.ReleaseBuffers(B, dev)),
            (paged.dspark_paged_attention, attend, (0, 1, 3, 4, 5),
             dict(scale=a.scale, max_new=2),
             lambda: paged.AttentionBuffers(3, 4, 2, 64, 2, torch.bfloat16, dev))):
        fn(*args, **opts, buffers=make())
        for i in which:
            for x in others(args[i]):
                for given in (None, make()):
                    with pytest.raises(ValueError):
                        fn(*args[:i], x, *args[i + 1:], **opts, buffers=given)


def test_buffers(dev):
    B, tokens = 4, 40
    i32 = dict(dtype=torch.int32, device=dev)
    ctx, new, table = torch.tensor([3, 0, 20, 16], **i32), torch.full((B,), 3, **i32), torch.zeros(B, 3, **i32)
    stack, count = torch.arange(20, **i32), torch.tensor([14], **i32)
    a = _paged.make_attention([50, 300], [2, 1], 4, 2, 64, 16, torch.bfloat16, seed=1, device=dev)
    calls = [
        (lambda b: paged.dspark_pages_reserve(ctx, new, table, stack, count, page_size=16,
                                              max_tokens=tokens, buffers=b),
         lambda: paged.ReserveBuffers(B, tokens, dev),
         ("context_len", "row_off", "draft_off", "slot_map", "positions", "free_count",
          "device_status")),
        (lambda b: paged.dspark_pages_release(ctx, ctx + 3, new, table, stack, count, page_size=16,
                                              buffers=b),
         lambda: paged.ReleaseBuffers(B, dev), ("context_len", "free_count", "device_status")),
        (lambda b: paged.dspark_paged_attention(a.q, a.k_cache, a.v_cache, a.table, a.context_len,
                                                a.row_off, scale=a.scale, max_new=2, with_lse=True,
                                                buffers=b),
         lambda: paged.AttentionBuffers(3, 4, 2, 64, 2, torch.bfloat16, dev, with_lse=True),
         ("out", "lse", "device_status"))]
    for call, make, names in calls:
        call(make())
        for name in names:
            for x in others(getattr(make(), name)):
                b = make()
                setattr(b, name, x)
                with pytest.raises(ValueError):
                    call(b)
    cache = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device=dev)
    rows, slots = torch.ones(3, 2, 64, dtype=torch.bfloat16, device=dev), torch.zeros(3, **i32)
    for x in others(torch.zeros(1, **i32)):
        with pytest.raises(ValueError):
            paged.dspark_kv_append(rows, rows, slots, cache, cache, device_status=x)
