"""dspark_pages_reserve at the largest step: max_tokens = 2^30 rows, and steps of more than that."""
import pytest
import torch

from speculative_decoding_verification_41_gb300 import build as cuda_build
from speculative_decoding_verification_41_gb300 import paged
from tests import _paged

pytestmark = pytest.mark.gpu

MOST = 1 << 30
PS = 1024


@pytest.fixture(scope="module")
def dev():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    cuda_build.build()
    return torch.device("cuda:0")


@pytest.fixture(scope="module")
def buffers(dev):
    made = {}

    def get(B):
        made.clear()
        made[B] = paged.ReserveBuffers(B, MOST, dev)
        return made[B]
    return get


def reserve(dev, buffers, new, pages, width):
    i32 = dict(dtype=torch.int32, device=dev)
    B = len(new)
    table = torch.full((B, width), -3, **i32)
    buf = buffers(B)
    buf.slot_map.fill_(-7)
    o = paged.dspark_pages_reserve(
        torch.zeros(B, **i32), torch.tensor(new, **i32), table, torch.arange(pages, **i32),
        torch.tensor([pages], **i32), page_size=PS, max_tokens=MOST, buffers=buf)
    torch.cuda.synchronize()
    return o, table


@pytest.mark.parametrize("past", [0, 1])
def test_a_step_of_2_to_the_30_rows(dev, buffers, past):
    """512 requests of 2^21 tokens fill the map; a token more is one too many, and its request and
    those after it get nothing."""
    n, each = 512, 1 << 21
    per = each // PS
    pages = n * per + 10
    new = [each] * n + [1, 5] * past
    o, table = reserve(dev, buffers, new, pages, per)
    assert int(o["device_status"].item()) == (_paged.TOO_LARGE if past else _paged.OK)
    assert o["row_off"].tolist() == [each * i for i in range(n + 1)] + [MOST] * (2 * past)
    assert o["draft_off"].tolist() == o["row_off"].tolist()
    assert o["context_len"].tolist() == [each] * n + [0] * (2 * past)
    assert o["free_count"].tolist() == [10]
    i = torch.arange(n * per, device=dev, dtype=torch.int32)
    assert torch.equal(table[:n].reshape(-1), pages - 1 - i)
    if past:
        assert bool((table[n:] == -3).all())
    for a in range(0, MOST, 1 << 26):
        t = torch.arange(a, a + (1 << 26), device=dev, dtype=torch.int32)
        assert torch.equal(o["positions"][a:a + (1 << 26)], t % each)
        assert torch.equal(o["slot_map"][a:a + (1 << 26)], (pages - 1 - t // PS) * PS + t % PS)


@pytest.mark.parametrize("new", [[MOST + 1], [(1 << 31) - 4096], [MOST - 5, 6, 1],
                                 [1 << 20] * 2100])
def test_steps_of_more_rows(dev, buffers, new):
    """Sums past 2^30, in one request and over many (more than 2^31 in all)."""
    width, pages = (max(new) + PS - 1) // PS, (1 << 21) - 2
    o, table = reserve(dev, buffers, new, pages, width)
    fit = 0
    while fit < len(new) and sum(new[:fit + 1]) <= MOST:
        fit += 1
    ends = [sum(new[:i]) for i in range(fit + 1)]
    assert int(o["device_status"].item()) == _paged.TOO_LARGE
    assert o["row_off"].tolist() == ends + [ends[-1]] * (len(new) - fit)
    assert o["context_len"].tolist() == new[:fit] + [0] * (len(new) - fit)
    held = sum(-(-n // PS) for n in new[:fit])
    assert o["free_count"].tolist() == [pages - held]
    assert bool((table[fit:] == -3).all())
    assert bool((o["slot_map"][ends[-1]:] == -1).all())
    if fit:
        last = ends[-1] - 1
        assert int(o["positions"][last].item()) == new[fit - 1] - 1
        assert int(o["slot_map"][last].item()) == (pages - held) * PS + (new[fit - 1] - 1) % PS
