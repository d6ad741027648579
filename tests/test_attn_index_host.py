"""Index arithmetic of the attention kernels (csrc/attn_index.h, compiled here) at the edges of what its
arguments may hold, against the same in whole numbers."""
import ctypes
import itertools

import pytest

import host_cpp

SOURCE = """
#include "attn_index.h"
extern "C" {
int seq_ok(int tok0, int t1, int len, int T, int64_t max_len) { return moe::seq_ok(tok0, t1, len, T, max_len); }
int first_key(int pos, int window) { return moe::first_key(pos, window); }
}
"""
MIN, MAX = -2 ** 31, 2 ** 31 - 1


@pytest.fixture(scope="module")
def L(tmp_path_factory):
    L = host_cpp.library(str(tmp_path_factory.mktemp("index")), SOURCE)
    L.seq_ok.argtypes = [ctypes.c_int] * 4 + [ctypes.c_int64]
    return L


def test_offsets_that_hold_anything(L):
    """A sequence counts where its rows lie in the batch and its length in the page table, and only there."""
    edge = [MIN, MIN + 1, MIN + 5, -1, 0, 1, 5, 35, 36, 37, MAX - 1, MAX]
    for tok0, t1, len_, T in itertools.product(edge, edge, edge, [1, 36, MAX]):
        for most in (16, 36, 2 ** 31 - 16):
            want = 0 <= tok0 <= t1 <= T and 0 <= len_ <= most
            assert L.seq_ok(tok0, t1, len_, T, most) == want, (tok0, t1, len_, T, most)


def test_first_key(L):
    for pos in [MIN, MIN + 1, -100, -1, 0, 1, 99, 100, 101, 5000, MAX - 17, MAX]:
        for window in [0, 1, 2, 99, 100, 101, 5000, MAX - 1, MAX]:
            assert L.first_key(pos, window) == (max(0, pos - window + 1) if window else 0), (pos, window)
