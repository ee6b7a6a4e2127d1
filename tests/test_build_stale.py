"""The module behind the paged calls fits one Python and one torch: after a change of either it is
stale, whatever the files' times say, and is not loaded."""
import os

import pytest

from speculative_decoding_verification_41_gb300 import build as cuda_build
from speculative_decoding_verification_41_gb300 import paged


def test_another_torch_makes_the_module_stale(monkeypatch):
    cuda_build.build()
    assert cuda_build.binding_fits() and not cuda_build._stale()
    abi = cuda_build._binding_abi()
    monkeypatch.setattr(cuda_build, "_binding_abi", lambda: abi + ".1")
    assert not cuda_build.binding_fits() and cuda_build._stale()
    monkeypatch.setattr(paged, "_ext", None)
    with pytest.raises(RuntimeError, match="not for this Python and torch"):
        paged._native()


def test_a_module_without_its_stamp_is_stale(monkeypatch, tmp_path):
    cuda_build.build()
    monkeypatch.setattr(cuda_build, "BINDING_STAMP", str(tmp_path / "none"))
    assert not cuda_build.binding_fits() and cuda_build._stale()


def test_build_makes_it_fit_again():
    cuda_build.build()
    os.remove(cuda_build.BINDING_STAMP)
    cuda_build.build()
    assert cuda_build.binding_fits() and not cuda_build._stale()
    assert paged._native() is not None
