"""The plans of the MXFP4 product and of the experts for a given routing, and the norm's launch shapes, as their host
sources make them (compiled here with g++, no GPU)."""
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
extern "C" int probe_mx4(int64_t M, int64_t N, int64_t K, int64_t given, int64_t* o) {
  qsg::Mx4Plan p;
  const int st = qsg::make_mx4_plan(M, N, K, given != 0, &p);
  const int64_t v[] = {p.kind, p.nt, p.waves, p.grid_n, p.bm, p.bn, p.split, p.kchunk, (int64_t)p.ws_bytes};
  for (int i = 0; i < 9; ++i) o[i] = v[i];
  return st;
}
extern "C" void probe_norm(int64_t T, int64_t D, int64_t* o) {
  int waves, rows;
  qsg::norm_shape(T, D, &waves, &rows);
  o[0] = waves; o[1] = rows;
}
extern "C" int probe_routed(int64_t type, int64_t T, int64_t D, int64_t F, int64_t E, int64_t k, int64_t* o) {
  qsg::MoePlan p;
  const int st = qsg::make_moe_plan((int)type, T, D, F, E, k, &p, true);
  o[0] = p.held; o[1] = p.up_groups; o[2] = p.rt; o[3] = p.slices;
  return st;
}
"""

KIND = {0: "none", 1: "zero", 2: "fused", 3: "skinny", 4: "wide"}
Routed = namedtuple("Routed", "held up_groups rt slices")
Mx4 = namedtuple("Mx4", "kind nt waves grid_n bm bn split kchunk ws_bytes")


@functools.lru_cache(maxsize=None)
def _lib():
    with tempfile.TemporaryDirectory() as tmp:
        src, out = os.path.join(tmp, "probe.cpp"), os.path.join(tmp, "probe.so")
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", f"-I{CSRC}", src, os.path.join(CSRC, "mx4_plan.cpp"),
                        os.path.join(CSRC, "moe_plan.cpp"), "-o", out], check=True)
        return ctypes.CDLL(out)


def mx4(m, n, k, given=False) -> Mx4:
    out = (ctypes.c_int64 * 9)()
    st = _lib().probe_mx4(*map(ctypes.c_int64, (m, n, k, int(given))), out)
    assert st == 0, st
    kind, *rest = list(out)
    return Mx4(KIND[kind], *rest)


def norm(t, d):
    """Waves per row, rows per workgroup."""
    out = (ctypes.c_int64 * 2)()
    _lib().probe_norm(ctypes.c_int64(t), ctypes.c_int64(d), out)
    return tuple(out)


def routed(mm_type, t, d, f, e, top_k) -> Routed:
    out = (ctypes.c_int64 * 4)()
    st = _lib().probe_routed(*map(ctypes.c_int64, (mm_type, t, d, f, e, top_k)), out)
    assert st == 0, st
    return Routed(*out)
