"""The build's check of waits that count on the compiler's loads: what it accepts, and each way a listing can be wrong."""
from __future__ import annotations

import importlib.util
import os

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _builder():
    spec = importlib.util.spec_from_file_location("_qsg_build", os.path.join(ROOT, "quantized_skinny_gemm_amd", "build.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


COPY = ["\tglobal_load_lds_dwordx4 v1, s[42:43] // 0", "\ts_cbranch_execz 11 // 0", "\tglobal_load_lds_dword v0, s[52:53] // 0"]
LOADS = ["\tglobal_load_dwordx4 v[4:7], v[0:1], off // 0", "\tglobal_load_dwordx2 v[8:9], v[2:3], off // 0"]
WAIT, MATH, JUMP = "\ts_waitcnt vmcnt(2) lgkmcnt(0) // 0", "\tv_add_f32_e32 v1, v2, v3 // 0", "\ts_cbranch_scc1 9 // 0"
BODY = [WAIT, *COPY, MATH, *LOADS, JUMP, "\tglobal_store_dword v[6:7], v1, off // 0"]
GOOD = [*LOADS, *COPY, *LOADS, JUMP, *BODY, *BODY, *BODY, JUMP, "\ts_waitcnt vmcnt(0) lgkmcnt(0) // 0", *COPY, MATH,
        "\ts_waitcnt vmcnt(0) lgkmcnt(0) // 0", *LOADS]


def _listing(lines, name="_Z5k_foov"):
    return "\n".join(["", "x.o:\tfile format elf64-amdgpu", "", "0000000000001000 <_Z5otherv>:", WAIT,
                      f"0000000000002000 <{name}>:", *lines, "0000000000003000 <_Z6other2v>:", WAIT, ""])


def test_counted_waits_accepts_whole_sets():
    assert _builder().check_counted_waits(_listing(GOOD), "k_foo", 2) == 3


@pytest.mark.parametrize("at", range(4))
@pytest.mark.parametrize("load", range(2))
def test_counted_waits_refuses_a_missing_load(at, load):
    """One load fewer behind any of the four sets of copies, the last body's included (its wait is the loop's first)."""
    lines = list(GOOD)
    starts = [i for i in range(len(lines)) if lines[i:i + 2] == LOADS][1:5]
    del lines[starts[at] + load]
    with pytest.raises(RuntimeError):
        _builder().check_counted_waits(_listing(lines), "k_foo", 2)


def test_counted_waits_refuses_other_shapes():
    check = _builder().check_counted_waits
    with pytest.raises(RuntimeError):
        check(_listing(GOOD), "k_bar", 2)                         # no such kernel
    with pytest.raises(RuntimeError):
        check(_listing([MATH]), "k_foo", 2)                       # no such wait
    jump = list(GOOD)
    jump.insert(jump.index(MATH) + 2, JUMP)                       # a way round the second load
    with pytest.raises(RuntimeError):
        check(_listing(jump), "k_foo", 2)
    late = [*BODY, *GOOD]                                         # a wait with no copies ahead of it
    with pytest.raises(RuntimeError):
        check(_listing(late), "k_foo", 2)


def test_counted_waits_of_the_built_kernels():
    b = _builder()
    for src, (kernel, count) in b.COUNTED_WAITS.items():
        obj = os.path.join(ROOT, "_build", src + ".o")
        if not os.path.exists(obj):
            pytest.skip("no objects of a build here")
        assert b.check_counted_waits(b._disassemble(obj), kernel, count) > 0
