"""dspark_kv_append's strides on the CPU: negative ones are refused, as the attention refuses them."""
import ctypes

import pytest

from speculative_decoding_verification_41_gb300 import binding, paged
from speculative_decoding_verification_41_gb300 import build as cuda_build


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    paged._load()
    return binding.load()


@pytest.mark.parametrize("bad", [dict(row=-1024), dict(head=-128), dict(page=-16384),
                                 dict(token=-1024), dict(chead=-128)])
def test_append_refuses_negative_strides(lib, bad):
    a = dict(row=1024, head=128, page=16384, token=1024, chead=128)
    a.update(bad)
    p = ctypes.c_void_p(256)
    assert lib.dspark_kv_append(p, p, a["row"], a["head"], p, 4, 8, 128, 1, p, p, a["page"],
                                a["token"], a["chead"], 16, 10, p, None) == 1
