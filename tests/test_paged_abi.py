"""The paged-cache calls' boundary, on the CPU: the library exports what
include/dspark_paged.h declares, its macros agree with the binding, host checks
refuse bad calls before anything is launched, the binding refuses tensors that
are not the calls', and the plain statements the GPU tests compare with keep
the pages' books."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

from speculative_decoding_verification_41_gb300 import binding, paged
from speculative_decoding_verification_41_gb300 import build as cuda_build
from tests import _paged


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    paged._load()
    return binding.load()


def test_header_declares_the_exported_calls(lib):
    txt = open(paged.HEADER).read()
    declared = set(re.findall(r"^int\s+(dspark_\w+)\s*\(", txt, flags=re.M))
    assert declared == set(paged.EXPORTED)
    out = subprocess.run(["nm", "-D", "--defined-only", binding.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    assert declared <= set(re.findall(r"\sT\s(dspark_\w+)", out))


def test_header_compiles_as_c_and_macros_match_binding(tmp_path):
    shapes = [(1, 1, 1, 64), (32, 8, 1, 128), (32, 8, 17, 128), (64, 1, 1, 64), (64, 1, 33, 128),
              (7, 7, 160, 64), (7, 7, 161, 64), (48, 16, 5, 128)]
    src = ["#include <stdio.h>", '#include "dspark_paged.h"', "int main(void) {"]
    src += [f'  printf("%zu\\n", (size_t)DSPARK_PAGED_ATTENTION_WS_BYTES({a}, {b}, {c}, {d}));'
            for a, b, c, d in shapes]
    c = tmp_path / "probe.c"
    c.write_text("\n".join(src + ["  return 0; }"]))
    exe = tmp_path / "probe"
    subprocess.run(["gcc", "-std=c11", "-Wall", "-Werror", f"-I{os.path.dirname(paged.HEADER)}",
                    str(c), "-o", str(exe)], check=True)
    got = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split()
    assert [int(x) for x in got] == [paged.paged_attention_workspace_bytes(*s) for s in shapes]


def _p(x):
    return None if x is None else ctypes.c_void_p(x)


def _reserve(lib, **kw):
    a = dict(ctx=256, new=256, extra=1, B=4, ps=16, pages=100, table=256, stride=8, width=8,
             stack=256, count=512, tokens=64, out=768, row=256, draft=None, slots=256, pos=None,
             count_out=1024, st=256)
    a.update(kw)
    return lib.dspark_pages_reserve(
        _p(a["ctx"]), _p(a["new"]), a["extra"], a["B"], a["ps"], a["pages"], _p(a["table"]),
        a["stride"], a["width"], _p(a["stack"]), _p(a["count"]), a["tokens"], _p(a["out"]),
        _p(a["row"]), _p(a["draft"]), _p(a["slots"]), _p(a["pos"]), _p(a["count_out"]),
        _p(a["st"]), None)


POOL = [dict(B=-1), dict(ps=0), dict(ps=4), dict(ps=24), dict(ps=2048), dict(pages=0),
        dict(pages=1 << 27, ps=16), dict(width=0), dict(width=9), dict(width=1 << 28, stride=1 << 28),
        dict(stride=7), dict(table=None), dict(st=None), dict(stack=None), dict(count=None),
        dict(count_out=None), dict(ctx=None), dict(out=None), dict(extra=-1)]


@pytest.mark.parametrize("bad", POOL + [dict(new=None), dict(row=None), dict(slots=None),
                                        dict(tokens=-1), dict(tokens=(1 << 30) + 1)])
def test_reserve_refuses_on_host(lib, bad):
    assert _reserve(lib, **bad) == 1


@pytest.mark.parametrize("bad", POOL + [dict(kept=None), dict(reserved=None)])
def test_release_refuses_on_host(lib, bad):
    a = dict(ctx=256, reserved=256, kept=256, extra=1, B=4, ps=16, pages=100, table=256, stride=8,
             width=8, stack=256, count=512, out=768, count_out=1024, st=256)
    a.update(bad)
    assert lib.dspark_pages_release(
        _p(a["ctx"]), _p(a["reserved"]), _p(a["kept"]), a["extra"], a["B"], a["ps"], a["pages"],
        _p(a["table"]), a["stride"], a["width"], _p(a["stack"]), _p(a["count"]), _p(a["out"]),
        _p(a["count_out"]), _p(a["st"]), None) == 1


@pytest.mark.parametrize("bad", [
    dict(n=-1), dict(H=0), dict(D=0), dict(D=96), dict(dtype=0), dict(dtype=3), dict(k=None),
    dict(v=None), dict(k=264), dict(vc=8), dict(slots=None), dict(row=1028), dict(head=12),
    dict(page=4), dict(token=20), dict(chead=1), dict(ps=12), dict(pages=0), dict(st=None)])
def test_append_refuses_on_host(lib, bad):
    a = dict(k=256, v=256, row=1024, head=128, slots=256, n=4, H=8, D=128, dtype=1, kc=256, vc=256,
             page=16384, token=1024, chead=128, ps=16, pages=10, st=256)
    a.update(bad)
    assert lib.dspark_kv_append(
        _p(a["k"]), _p(a["v"]), a["row"], a["head"], _p(a["slots"]), a["n"], a["H"], a["D"],
        a["dtype"], _p(a["kc"]), _p(a["vc"]), a["page"], a["token"], a["chead"], a["ps"],
        a["pages"], _p(a["st"]), None) == 1


@pytest.mark.parametrize("bad,code", [
    (dict(B=-1), 1), (dict(n=-1), 1), (dict(Hq=0), 1), (dict(Hkv=0), 1), (dict(Hq=12), 1),
    (dict(Hq=4), 1), (dict(D=80), 1), (dict(D=256), 1), (dict(new=0), 1), (dict(scale=0.0), 1),
    (dict(scale=-1.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(window=-1), 1), (dict(dtype=0), 1), (dict(ps=4), 1), (dict(ps=48), 1), (dict(pages=0), 1),
    (dict(width=0), 1), (dict(stride=3), 1), (dict(q=None), 1), (dict(q=264), 1), (dict(k=None), 1),
    (dict(v=24), 1), (dict(table=None), 1), (dict(ctx=None), 1), (dict(off=None), 1),
    (dict(out=None), 1), (dict(out=258), 1), (dict(st=None), 1), (dict(qrow=4100), 1),
    (dict(qhead=-128), 1), (dict(page=12), 1), (dict(width=1 << 27), 1), (dict(ws=None), 3),
    (dict(ws=128), 3), (dict(wsb=1000), 3)])
def test_attention_refuses_on_host(lib, bad, code):
    a = dict(q=256, qrow=4096, qhead=128, k=256, v=256, page=16384, token=1024, head=128, ps=16,
             pages=10, table=256, stride=1 << 27, width=8, ctx=256, off=256, B=2, n=4, Hq=32, Hkv=8,
             D=128, new=2, scale=0.1, window=0, dtype=1, out=256, lse=None, st=256, ws=256,
             wsb=1 << 30)
    a.update(bad)
    assert lib.dspark_paged_attention(
        _p(a["q"]), a["qrow"], a["qhead"], _p(a["k"]), _p(a["v"]), a["page"], a["token"],
        a["head"], a["ps"], a["pages"], _p(a["table"]), a["stride"], a["width"], _p(a["ctx"]),
        _p(a["off"]), a["B"], a["n"], a["Hq"], a["Hkv"], a["D"], a["new"], a["scale"],
        a["window"], a["dtype"], _p(a["out"]), _p(a["lse"]), _p(a["st"]), _p(a["ws"]), a["wsb"],
        None) == code


def test_binding_refuses_cpu_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    t = torch.zeros(2, 4, dtype=torch.int32)
    c = torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        paged.dspark_pages_reserve(i, i, t, i, i[:1], page_size=16, max_tokens=8)
    with pytest.raises(ValueError, match="CUDA"):
        paged.dspark_pages_release(i, i, i, t, i, i[:1], page_size=16)
    with pytest.raises(ValueError, match="CUDA"):
        paged.dspark_kv_append(c[0], c[0], i, c, c)
    with pytest.raises(ValueError, match="CUDA"):
        paged.dspark_paged_attention(c[0], c, c, t, i, i, scale=1.0, max_new=1)


@pytest.mark.parametrize("seed", range(20))
def test_plain_books_balance(seed):
    """What the plain reserve gives out and the plain release takes back is the pool: no page is
    held twice, and after all requests finish every page is free again."""
    rng = np.random.default_rng(seed)
    ps, B = int(rng.choice([8, 16, 64])), int(rng.integers(1, 9))
    width, pages = 6, 40
    table = np.full((B, width), -1, np.int32)
    stack, count = rng.permutation(pages).astype(np.int32), pages
    ctx = np.zeros(B, np.int32)
    for _ in range(6):
        new = rng.integers(0, ps + 3, B).astype(np.int32)
        o = _paged.reserve(ctx, new, 1, table, stack, count, ps, pages, 1000)
        if o["status"] == _paged.BAD_DATA:  # longer than a table row: everything ends
            break
        table, count = o["block_table"], int(o["free_count"][0])
        kept = np.minimum(rng.integers(0, ps + 3, B), new).astype(np.int32)
        q = _paged.release(ctx, o["context_len"], kept, 1, table, stack, count, ps, pages)
        stack, count, ctx = q["free_pages"], int(q["free_count"][0]), q["context_len"]
        held = [int(table[r, j]) for r in range(B) for j in range(_paged.up(int(ctx[r]), ps))]
        assert sorted(held + stack[:count].tolist()) == list(range(pages))
    q = _paged.release(ctx, ctx, np.full(B, -1, np.int32), 1, table, stack, count, ps, pages)
    assert sorted(q["free_pages"].tolist()) == list(range(pages)) and q["free_count"][0] == pages
