"""The plans of the e4m3 product and of the mixture-of-experts layer, as their host sources make them (compiled here
with g++, no GPU): which kernel, tile and split a call takes."""
from __future__ import annotations

import ctypes
import functools
import os
import subprocess
import tempfile
from collections import namedtuple

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_skinny_gemm_amd", "csrc")

SOURCE = r"""
#include "plan.h"
extern "C" int probe_f8(int64_t M, int64_t N, int64_t K, int64_t given, int64_t* o) {
  qsg::F8Plan p;
  const int st = qsg::make_f8_plan(M, N, K, given != 0, &p);
  o[0] = p.kind; o[1] = p.nt; o[2] = p.bm; o[3] = p.bn; o[4] = p.split; o[5] = p.kchunk;
  return st;
}
extern "C" int probe_moe(int64_t type, int64_t T, int64_t D, int64_t F, int64_t E, int64_t k, int64_t* o) {
  qsg::MoePlan p;
  const int st = qsg::make_moe_plan((int)type, T, D, F, E, k, &p);
  o[0] = p.fold; o[1] = p.up_groups; o[2] = p.rt; o[3] = p.slices;
  return st;
}
"""

KIND = {0: "none", 1: "zero", 2: "fused", 3: "skinny", 4: "wide"}
F8 = namedtuple("F8", "kind nt bm bn split kchunk")          # bm, bn, split, kchunk: the tiled kernel's
Moe = namedtuple("Moe", "fold up_groups rt slices")


@functools.lru_cache(maxsize=None)
def _lib():
    with tempfile.TemporaryDirectory() as tmp:
        src, out = os.path.join(tmp, "probe.cpp"), os.path.join(tmp, "probe.so")
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", f"-I{CSRC}", src, os.path.join(CSRC, "f8_plan.cpp"),
                        os.path.join(CSRC, "moe_plan.cpp"), "-o", out], check=True)
        return ctypes.CDLL(out)


def _call(fn, n, *args):
    out = (ctypes.c_int64 * n)()
    st = fn(*map(ctypes.c_int64, args), out)
    assert st == 0, st
    return list(out)


def f8(m, n, k, given=False) -> F8:
    kind, *rest = _call(_lib().probe_f8, 6, m, n, k, int(given))
    return F8(KIND[kind], *rest)


def moe(mm_type, t, d, f, e, top_k) -> Moe:
    return Moe(*_call(_lib().probe_moe, 4, mm_type, t, d, f, e, top_k))
