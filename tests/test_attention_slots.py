"""The rows that a work-group of the attention kernels takes, for any offsets (csrc/attention_slots.h on
the host, where a lane is a loop index): every access stays inside the tensors, and offsets as they should be
give every row to exactly one lane."""

import ctypes
import os
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "equivariant_gnn_message_amd", "csrc")

SOURCE = r"""
#include "attention_slots.h"
using namespace e3c::attn;

// Lanes whose (query, head of the group) lies outside n x group; taken[row] counts the lanes of the others.
extern "C" long walk(const int* ptr, int graphs, long n, int group, int tile, int* taken) {
  const GroupDiv by = group_div(group);
  const long slots = n * group / tile + graphs;
  long outside = 0;
  for (int slot = 0; slot < slots; ++slot) {
    const auto first = [&](int g) { return slot_at(clamp_offset(ptr[g], n), g, group, tile); };
    const int g = search_graph(graphs, [&](int lo, int step, int count) {
      int hits = 0;
      for (int lane = 0; lane < 64; ++lane)
        if (lane * step < count) hits += first(lo + lane * step) <= slot;
      return hits;
    });
    const int q0 = clamp_offset(ptr[g], n), nrows = (clamp_offset(ptr[g + 1], n) - q0) * group;
    const int r0 = tile_start(slot, first(g), tile, nrows);
    if (r0 < 0) continue;
    for (int r = r0; r < r0 + tile && r < nrows; ++r) {
      const long q = (long)q0 + div_group(r, group, by.magic, by.shift), head = r - (q - q0) * group;
      if (q < 0 || q >= n || head < 0 || head >= group) ++outside;
      else ++taken[q * group + head];
    }
  }
  return outside;
}
extern "C" int divide(int r, int group) {
  const GroupDiv by = group_div(group);
  return div_group(r, group, by.magic, by.shift);
}
extern "C" int step_queries(int group, int step) { return step >> group_div(group).log2 << group_div(group).log2; }
extern "C" int log2_of(int group) { return group_div(group).log2; }
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    where = tmp_path_factory.mktemp("slots")
    src, lib = where / "slots.cpp", where / "slots.so"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-O1", "-shared", "-fPIC", "-I", CSRC, "-o", str(lib), str(src)], check=True)
    lib = ctypes.CDLL(str(lib))
    lib.walk.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_long, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]
    lib.walk.restype = ctypes.c_long
    return lib


def walk(host, ptr, n, group, tile):
    ptr = np.ascontiguousarray(ptr, dtype=np.int32)
    taken = np.zeros(max(n * group, 1), dtype=np.int32)
    outside = host.walk(ptr.ctypes.data, len(ptr) - 1, n, group, tile, taken.ctypes.data)
    return outside, taken[:n * group]


@pytest.mark.parametrize("tile", [32, 128])
@pytest.mark.parametrize("group", [1, 2, 3, 4, 8])
def test_every_row_once(host, group, tile):
    rng = np.random.default_rng(group)
    for graphs in (1, 3, 64, 65, 300, 5000):
        lens = rng.integers(0, 40, graphs) * (rng.random(graphs) < 0.7)
        if graphs < 100:
            lens[rng.integers(graphs)] = 1000
        ptr = np.concatenate([[0], np.cumsum(lens)])
        outside, taken = walk(host, ptr, int(ptr[-1]), group, tile)
        assert outside == 0 and np.all(taken == 1)


@pytest.mark.parametrize("tile", [32, 128])
@pytest.mark.parametrize("group", [1, 2, 3, 4, 8])
def test_any_offsets_stay_inside(host, group, tile):
    """Offsets of part of a batch, in no order, negative, past the end."""
    rng = np.random.default_rng(10 + group)
    tables = [([100, 200], 300), ([200, 100], 300), ([300, 0, 300], 300), ([0, 5, 3, 300], 300), ([-5, 1 << 30], 77),
              ([150] * 9, 300)]
    for _ in range(200):
        n = int(rng.integers(1, 700))
        tables.append((rng.integers(-50, n + 50, int(rng.integers(2, 200))), n))
    for ptr, n in tables:
        outside, taken = walk(host, ptr, n, group, tile)
        assert outside == 0, (list(ptr)[:10], n)
    # offsets of part of a batch: its rows are taken once, the others not at all
    outside, taken = walk(host, [100, 130, 200], 300, group, tile)
    want = np.repeat((np.arange(300) >= 100) & (np.arange(300) < 200), group)
    assert outside == 0 and np.array_equal(taken, want.astype(np.int32))


@pytest.mark.parametrize("group", [1, 2, 3, 5, 7, 8, 12, 100, 4097])
def test_division(host, group):
    for r in [0, 1, group - 1, group, 2 * group - 1, 12345678, (1 << 31) - 1 - (1 << 20), (1 << 31) - 1]:
        assert host.divide(r, group) == r // group


@pytest.mark.parametrize("group", [1, 2, 3, 4, 6, 8, 12, 32, 100, 4096])
@pytest.mark.parametrize("step", [4, 8, 16, 64])
def test_rows_a_step_apart(host, group, step):
    """A kernel shifts by log2 before it knows whether the heads of a group divide a step of rows."""
    assert 0 <= host.log2_of(group) <= 31
    assert (host.step_queries(group, step) == step) == (step % group == 0)
