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
int tile_inside(int key, int count, int from, int to) { return moe::tile_inside(key, count, from, to); }
int tile_meets(int key, int count, int from, int to) { return moe::tile_meets(key, count, from, to); }
int tiles_until(int to, int log2) { return moe::tiles_until(to, log2); }
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


def test_tiles_up_to_the_last_key(L):
    """A tile's keys against a range of keys, to the longest length that a page table allows."""
    last = 2 ** 31 - 128
    for count in (16, 32, 128):
        keys = [0, count, 10 * count, last - count, last, 2 ** 31 - count]
        ends = [0, 1, count - 1, count, count + 1, last - 1, last, last + 1, MAX - 100, MAX - 15, MAX]
        for key, lo, hi in itertools.product(keys, ends, ends):
            assert L.tile_inside(key, count, lo, hi) == (lo <= key and key + count <= hi), (key, count, lo, hi)
            assert L.tile_meets(key, count, lo, hi) == (key < hi and key + count > lo), (key, count, lo, hi)
    for log2 in (4, 6, 7, 8):
        for to in [0, 1, 15, 16, 17, 128, 129, 300, last - 1, last, last + 1, MAX - 15, MAX]:
            assert L.tiles_until(to, log2) == -(-to // 2 ** log2)
