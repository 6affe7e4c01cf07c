"""Host walk over the shares of the paged attention's work and the joins of its parts
(csrc/gdn_attn_shares.h, the kernel's own arithmetic): every part is joined once, and no two
tasks count in one word, for all that run at the same time."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_deltanet_layer_gb300", "csrc")
PROGRAM = r"""
#include "gdn_attn_shares.h"
using namespace gdn;
// Joins of the tasks that several CTAs share, a row for each level and group: {task, level, group, word, count, begin, step,
// parts, first CTA}. Returns the number of rows.
extern "C" int walk(const long long* tasks, int n, int ctas, int grid, int* out) {
  long long units = 0, u = 0;
  for (int i = 0; i < n; ++i) units += tasks[i];
  const Shares s(units, ctas);
  int rows = 0;
  for (int i = 0; i < n; u += tasks[i++]) {
    const int c0 = s.owner(u), c1 = s.owner(u + tasks[i] - 1);
    if (s.first(c0) > u || s.first(c0 + 1) <= u || s.first(c1 + 1) < u + tasks[i]) return -1;
    if (c0 == c1) continue;
    const Join j(c0, c1);
    for (int level = j.first_level(); level < 2; ++level)
      for (int g = 0; g < (level == 0 ? j.groups : 1); ++g) {
        const int row[9] = {i, level, g, j.word(level, g, grid), j.count(level, g), j.begin(level, g), j.step(level), j.parts, c0};
        for (int x : row) *out++ = x;
        ++rows;
      }
    for (int c = c0; c <= c1; ++c)
      if (j.group(c) < 0 || j.group(c) >= j.groups) return -1;
  }
  return rows;
}
"""


@pytest.fixture(scope="module")
def walk(tmp_path_factory):
    d = tmp_path_factory.mktemp("shares")
    (d / "walk.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(d / "walk.cpp"), "-o", str(d / "walk.so")],
                   check=True)
    f = ctypes.CDLL(str(d / "walk.so")).walk
    f.argtypes = [ctypes.c_void_p, ctypes.c_int, ctypes.c_int, ctypes.c_int, ctypes.c_void_p]

    def rows(tasks, grid):
        tasks = np.ascontiguousarray(tasks, dtype=np.int64)
        ctas = int(min(grid, (tasks.sum() + 1) // 2))
        out = np.zeros((4 * grid + 4 * len(tasks), 9), np.int32)
        n = f(tasks.ctypes.data, len(tasks), ctas, grid, out.ctypes.data)
        assert n >= 0, "a task's CTAs are not those that have its units"
        return out[:n]
    return rows


def verify(rows, grid):
    words = rows[:, 3]
    assert ((words >= 0) & (words < 2 * grid)).all()
    assert len(np.unique(words)) == len(words), "two joins count in one word"
    for t in np.unique(rows[:, 0]):
        mine = rows[rows[:, 0] == t]
        parts = mine[0, 7]
        groups = mine[mine[:, 1] == 0]
        ends = groups if len(groups) else mine
        covered = np.concatenate([b + s * np.arange(n) for _, _, _, _, n, b, s, _, _ in ends])
        assert np.array_equal(np.sort(covered), np.arange(parts))
        top = mine[mine[:, 1] == 1]
        assert len(top) == 1
        if len(groups):  # the groups' first parts, in order
            assert np.array_equal(top[0, 5] + top[0, 6] * np.arange(top[0, 4]), groups[:, 5])
        assert (ends[:, 4] <= 16).all() and top[0, 4] <= 16


def tiles(keys, key_tile=128):
    return -(-np.asarray(keys) // key_tile)


@pytest.mark.parametrize("requests,keys,heads,key_tile", [
    (8, 32769, 1, 128), (8, 17953, 1, 128), (5, 18950, 1, 128), (5, 65537, 1, 128), (1, 33401, 8, 128), (2, 131073, 4, 64)])
def test_long_neighbours(walk, requests, keys, heads, key_tile):
    """Tasks of more parts than are joined at once, one beginning in the CTA that ends the one before."""
    rows = walk(np.repeat(tiles([keys] * requests, key_tile), heads), 152)
    assert (rows[:, 7] > 16).sum() > 1
    verify(rows, 152)


@pytest.mark.parametrize("grid", [152, 148, 132, 20])
def test_equal_tasks(walk, grid):
    for n in range(1, 12):
        for units in list(range(1, 700)) + list(range(701, 9000, 37)):
            verify(walk([units] * n, grid), grid)


def test_ragged_tasks(walk):
    rng = np.random.default_rng(1)
    for _ in range(3000):
        n = int(rng.integers(1, 9))
        heads = int(rng.choice([1, 2, 4, 8]))
        verify(walk(np.repeat(tiles(np.exp(rng.uniform(0, 12.5, n)).astype(np.int64) + 1), heads), 152), 152)
