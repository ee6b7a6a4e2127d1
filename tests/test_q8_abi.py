"""The 8-bit cache's calls' boundary, on the CPU: the library exports what
include/dspark_q8.h declares, host checks refuse bad calls before anything is launched, the
binding refuses tensors that are not the calls', rotation tables hold the angles they
state, and the plain statements the GPU tests compare with agree with torch's own e4m3."""
import ctypes
import math
import re
import subprocess

import numpy as np
import pytest
import torch

from speculative_decoding_verification_41_gb300 import binding, paged, paged_q8
from speculative_decoding_verification_41_gb300 import build as cuda_build
from tests import _q8


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    paged._load()
    return binding.load()


def test_header_declares_the_exported_calls(lib):
    declared = set(re.findall(r"^int\s+(dspark_\w+)\s*\(", open(paged_q8.HEADER).read(), flags=re.M))
    assert declared == set(paged_q8.EXPORTED)
    out = subprocess.run(["nm", "-D", "--defined-only", binding.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    assert declared <= set(re.findall(r"\sT\s(dspark_\w+)", out))


def test_header_compiles_as_c(tmp_path):
    c = tmp_path / "probe.c"
    c.write_text('#include <stdio.h>\n#include "dspark_q8.h"\n'
                 'int main(void) { printf("%zu\\n", sizeof(dspark_rotation)); return 0; }\n')
    exe = tmp_path / "probe"
    include = paged_q8.HEADER.rsplit("/", 1)[0]
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", f"-I{include}", str(c), "-o", str(exe)],
                   check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout
    assert int(got) == ctypes.sizeof(paged_q8._Rotation)


def _p(x):
    return None if x is None else ctypes.c_void_p(x)


def _rot(turns=256, rot=64, pairs=0, gain=1.0):
    return paged_q8._Rotation(turns, rot, pairs, gain)


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(x=264), dict(out=None), dict(out=8), dict(pos=None), dict(rot=None),
    dict(rot=_rot(turns=None)), dict(rot=_rot(rot=8)), dict(rot=_rot(rot=24)),
    dict(rot=_rot(rot=144)), dict(rot=_rot(pairs=2)), dict(rot=_rot(gain=math.inf)),
    dict(rot=_rot(gain=math.nan)), dict(inv=2), dict(n=-1), dict(H=0), dict(D=96), dict(dtype=0),
    dict(row=1020), dict(head=-128), dict(orow=4), dict(out=256, orow=2048)])
def test_rotary_refuses_on_host(lib, bad):
    a = dict(x=256, row=1024, head=128, pos=256, rot=_rot(), inv=0, n=4, H=8, D=128, dtype=1,
             out=512, orow=1024, ohead=128)
    a.update(bad)
    r = a["rot"]
    assert lib.dspark_rotary(
        _p(a["x"]), a["row"], a["head"], _p(a["pos"]), None if r is None else ctypes.byref(r),
        a["inv"], a["n"], a["H"], a["D"], a["dtype"], _p(a["out"]), a["orow"], a["ohead"],
        None) == 1


CACHE = [dict(n=-1), dict(H=0), dict(D=0), dict(D=96), dict(dtype=0), dict(dtype=3), dict(k=None),
         dict(v=None), dict(k=264), dict(kc=None), dict(vc=8), dict(ks=None), dict(vs=None),
         dict(slots=None), dict(row=1028), dict(head=-8), dict(page=8), dict(token=-1024),
         dict(chead=24), dict(spage=-1), dict(sblock=-8), dict(shead=-1), dict(block=0),
         dict(block=3), dict(block=32), dict(ps=12), dict(ps=4), dict(ps=2048), dict(pages=0),
         dict(pages=1 << 28), dict(st=None)]


def _args(bad):
    a = dict(k=256, v=256, row=1024, head=128, slots=256, n=4, H=8, D=128, dtype=1, kc=256, vc=256,
             page=16384, token=1024, chead=128, ks=256, vs=256, spage=8, sblock=8, shead=1,
             block=16, ps=16, pages=10, st=256, rot=None, pos=256)
    a.update(bad)
    return a


@pytest.mark.parametrize("bad", CACHE + [dict(rot=_rot(), pos=None), dict(rot=_rot(rot=40)),
                                         dict(rot=_rot(rot=128), D=64)])
def test_append_refuses_on_host(lib, bad):
    a = _args(bad)
    r = a["rot"]
    assert lib.dspark_kv_append_q8(
        _p(a["k"]), _p(a["v"]), a["row"], a["head"], None if r is None else ctypes.byref(r),
        _p(a["pos"]), _p(a["slots"]), a["n"], a["H"], a["D"], a["dtype"], _p(a["kc"]),
        _p(a["vc"]), a["page"], a["token"], a["chead"], _p(a["ks"]), _p(a["vs"]), a["spage"],
        a["sblock"], a["shead"], a["block"], a["ps"], a["pages"], _p(a["st"]), None) == 1


@pytest.mark.parametrize("bad", CACHE)
def test_gather_refuses_on_host(lib, bad):
    a = _args(bad)
    assert lib.dspark_kv_gather_q8(
        _p(a["kc"]), _p(a["vc"]), a["page"], a["token"], a["chead"], _p(a["ks"]), _p(a["vs"]),
        a["spage"], a["sblock"], a["shead"], a["block"], a["ps"], a["pages"], _p(a["slots"]),
        a["n"], a["H"], a["D"], a["dtype"], _p(a["k"]), _p(a["v"]), a["row"], a["head"],
        _p(a["st"]), None) == 1


@pytest.mark.parametrize("bad,code", [
    (dict(B=-1), 1), (dict(n=-1), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(Hq=12), 1),
    (dict(D=80), 1), (dict(new=0), 1), (dict(scale=0.0), 1), (dict(scale=math.nan), 1),
    (dict(window=-1), 1), (dict(dtype=0), 1), (dict(ps=4), 1), (dict(ps=48), 1), (dict(pages=0), 1),
    (dict(block=0), 1), (dict(block=6), 1), (dict(block=32), 1), (dict(width=0), 1),
    (dict(stride=3), 1), (dict(q=None), 1), (dict(q=264), 1), (dict(k=None), 1), (dict(v=24), 1),
    (dict(ks=None), 1), (dict(vs=None), 1), (dict(spage=-1), 1), (dict(table=None), 1),
    (dict(ctx=None), 1), (dict(off=None), 1), (dict(out=None), 1), (dict(out=258), 1),
    (dict(st=None), 1), (dict(qrow=4100), 1), (dict(qhead=-128), 1), (dict(page=12), 1),
    (dict(token=1032), 1), (dict(width=1 << 27), 1), (dict(ws=None), 3), (dict(ws=128), 3),
    (dict(wsb=1000), 3)])
def test_attention_refuses_on_host(lib, bad, code):
    a = dict(q=256, qrow=4096, qhead=128, k=256, v=256, page=16384, token=1024, head=128, ks=256,
             vs=256, spage=8, sblock=8, shead=1, block=16, ps=16, pages=10, table=256,
             stride=1 << 27, width=8, ctx=256, off=256, B=2, n=4, Hq=32, Hkv=8, D=128, new=2,
             scale=0.1, window=0, dtype=1, out=256, lse=None, st=256, ws=256, wsb=1 << 30)
    a.update(bad)
    assert lib.dspark_paged_attention_q8(
        _p(a["q"]), a["qrow"], a["qhead"], _p(a["k"]), _p(a["v"]), a["page"], a["token"],
        a["head"], _p(a["ks"]), _p(a["vs"]), a["spage"], a["sblock"], a["shead"], a["block"],
        a["ps"], a["pages"], _p(a["table"]), a["stride"], a["width"], _p(a["ctx"]), _p(a["off"]),
        a["B"], a["n"], a["Hq"], a["Hkv"], a["D"], a["new"], a["scale"], a["window"], a["dtype"],
        _p(a["out"]), _p(a["lse"]), _p(a["st"]), _p(a["ws"]), a["wsb"], None) == code


def test_binding_refuses_cpu_tensors(lib):
    i = torch.zeros(2, dtype=torch.int32)
    c = torch.zeros(4, 16, 2, 64, dtype=torch.uint8).view(_q8.E4M3)
    s = torch.ones(4, 1, 2)
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    t = paged_q8.RotaryTable(64, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        paged_q8.dspark_rotary(x, i, t)
    with pytest.raises(ValueError, match="CUDA"):
        paged_q8.dspark_rotary(x, i, t, out=x)
    with pytest.raises(ValueError, match="CUDA"):
        paged_q8.dspark_kv_append_q8(x, x, i, c, c, s, s)
    with pytest.raises(ValueError, match="CUDA"):
        paged_q8.dspark_kv_append_q8(x, x, i, c, c, s, s, device_status=i[:1])
    with pytest.raises(ValueError, match="CUDA"):
        paged_q8.dspark_kv_gather_q8(c, c, s, s, i)
    with pytest.raises(ValueError, match="CUDA"):
        paged_q8.dspark_paged_attention_q8(x, c, c, s, s, i[:, None], i, i, scale=1.0, max_new=1)


@pytest.mark.parametrize("bad", [dict(rot_dim=8), dict(rot_dim=40), dict(rot_dim=144),
                                 dict(scaling="other"), dict(base=0.0), dict(factor=-1.0),
                                 dict(scaling="yarn"), dict(gain=math.inf),
                                 dict(scaling="yarn", original_len=10, fast=1.0, slow=2.0)])
def test_rotary_table_refuses(bad):
    with pytest.raises(ValueError):
        paged_q8.RotaryTable(**{"rot_dim": 64, "device": "cpu", **bad})


def test_rotary_table_of_angles():
    with pytest.raises(ValueError):
        paged_q8.RotaryTable.of([0.1] * 12, device="cpu")
    t = paged_q8.RotaryTable.of([0.5, -0.5, 7.0, 0.0, 2 * math.pi, 1e-12, 3.0, -9.0], device="cpu")
    assert t.rot_dim == 16
    # parts of a turn as fractions of 2^64, to the 53 bits of the angles
    for x, f in zip(t.angles, t.turns.tolist()):
        want = math.fmod(x / (2 * math.pi), 1.0)
        got = f / 2.0 ** 64
        assert abs(got - want - round(got - want)) < 2.0 ** -52 * max(1.0, abs(x))


def test_rotary_scalings():
    plain = paged_q8.RotaryTable(64, device="cpu").angles
    ntk = paged_q8.RotaryTable(64, scaling="ntk", factor=4.0, device="cpu").angles
    assert ntk[0] == plain[0] == 1.0 and math.isclose(ntk[-1], plain[-1] / 4)
    yarn = paged_q8.RotaryTable(64, scaling="yarn", factor=4.0, original_len=2048, device="cpu")
    assert yarn.angles[0] == plain[0] and math.isclose(yarn.angles[-1], plain[-1] / 4)
    assert all(p / 4 <= y <= p for p, y in zip(plain, yarn.angles))
    assert math.isclose(yarn.gain, 0.1 * math.log(4) + 1)
    linear = paged_q8.RotaryTable(64, scaling="linear", factor=4.0, device="cpu")
    assert linear.angles == [p / 4 for p in plain] and linear.gain == 1.0


def test_plain_e4m3_is_torchs():
    codes = torch.arange(256, dtype=torch.uint8).view(_q8.E4M3)
    assert np.array_equal(_q8.numbers(codes), codes.double().numpy(), equal_nan=True)
    x = torch.randn(5000, generator=torch.Generator().manual_seed(0)) * 100
    x = torch.cat([x, torch.arange(-448, 449) / 1.0, torch.arange(-64, 65) * 2.0 ** -11])
    assert np.array_equal(_q8.rounded(x.double().numpy()), x.to(_q8.E4M3).double().numpy())


@pytest.mark.parametrize("a,want", [(0.0, 2.0 ** -126), (448.0, 1.0), (448.0001, 2.0), (224.0, 0.5),
                                    (1.75, 2.0 ** -8), (3.4e38, 2.0 ** 120), (1e-45, 2.0 ** -126)])
def test_needed_scale(a, want):
    assert _q8.needed(a) == want
