"""The split of x that the gate / up launch of a given routing makes in LDS for up to 4 tokens: which token's piece each thread
stores, over every width that the plan lets it hold (the index rule compiled here with g++, no GPU)."""
from __future__ import annotations

import ctypes
import os
import subprocess

import numpy as np
import pytest

from tests import mx4_plans
from tests.test_gpu_moe_held import HELD

THREADS = 512
SOURCE = r"""
#include "plan.h"
extern "C" void held_tokens(const int32_t* i, int32_t n, int32_t row, int32_t T, int32_t* t) {
  for (int k = 0; k < n; ++k) t[k] = qsg::held_token(i[k], row, T);
}
"""


def _row(d):
    """Pieces of four values of a token: its blocks of 32, padded to a multiple of four blocks."""
    return 8 * 4 * -(-d // 128)


@pytest.fixture(scope="module")
def tokens(tmp_path_factory):
    tmp = tmp_path_factory.mktemp("held")
    src, out = os.path.join(tmp, "probe.cpp"), os.path.join(tmp, "probe.so")
    with open(src, "w") as f:
        f.write(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-shared", "-fPIC", f"-I{mx4_plans.CSRC}", src, "-o", out], check=True)
    lib = ctypes.CDLL(out)

    def of(i, row, t):
        i = np.ascontiguousarray(i, np.int32)
        got = np.empty_like(i)
        lib.held_tokens(ctypes.c_void_p(i.ctypes.data), len(i), row, t, ctypes.c_void_p(got.ctypes.data))
        return got
    return of


@pytest.mark.parametrize("t", [1, 2, 3, 4])
def test_every_piece_is_stored_once_and_none_behind_its_row(tokens, t):
    widths = [d for d in range(32, 8225, 32) if mx4_plans.routed(6, t, d, 64, 64, 16).held]
    assert widths and max(widths) == 8192 // t // 128 * 128
    for d in widths:
        row, stored = _row(d), []
        # rounds of all threads, until one begins behind the last token
        for first in range(0, t * row, THREADS):
            i = np.arange(first, first + THREADS)
            whose = tokens(i, row, t)
            stored.append((i - whose * row + whose * 65536)[whose < t])
            assert np.all(whose.reshape(-1, 8) == whose.reshape(-1, 8)[:, :1]), (t, d)     # eight threads, one block
        want = (np.arange(row)[None] + np.arange(t)[:, None] * 65536).reshape(-1)
        assert np.array_equal(np.sort(np.concatenate(stored)), want), (t, d)


def test_last_rounds_that_end_inside_have_shapes_on_the_gpu():
    """For each number of tokens several rounds of which the last is partly filled, and one that ends with a token."""
    for t in (2, 3, 4):
        shapes = [_row(d) * t for n, d, f, e, k in HELD if n == t and mx4_plans.routed(6, n, d, f, e, k).held]
        assert any(n > THREADS and n % THREADS for n in shapes), t
        assert any(n > THREADS and n % THREADS == 0 for n in shapes), t
    assert all(mx4_plans.routed(kind, *s).held for s in HELD for kind in (1, 4, 5, 6))
