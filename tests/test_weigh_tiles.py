"""Which row tiles a pass of the window's weights goes through (csrc/weigh_tiles.cuh, compiled
for the host), and that its two sides cannot fall out of step: the warps that write q
complete one phase of a barrier for each row tile, the issuing warp tells them apart by
parity alone, and all that keeps the first from completing two of them in between is the
wait for the row tile's products, of which a row tile without keys has none."""
import ctypes
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
SOURCE = """
#include "weigh_tiles.cuh"
using namespace attn::weigh_tiles;
extern "C" {
void segment_(int keys, int splits, int s, int* k) { segment(keys, splits, s, k, k + 1); }
int tiles_(int ctx, int rows, int k0, int k1, int rt) { return tiles(ctx, rows, k0, k1, rt); }
int first_seeing_(int ctx, int k0, int k1, int rt0, int rt1) { return first_seeing(ctx, k0, k1, rt0, rt1); }
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    at = tmp_path_factory.mktemp("tiles")
    (at / "t.cpp").write_text(SOURCE)
    subprocess.run([cxx, "-std=c++17", "-shared", "-fPIC", "-I", os.path.join(ROOT, "chunked_prefill_gqa_gb300", "csrc"),
                    "-o", str(at / "t.so"), str(at / "t.cpp")], check=True)
    return ctypes.CDLL(str(at / "t.so"))


def segment(lib, keys, splits, s):
    k = (ctypes.c_int * 2)()
    lib.segment_(keys, splits, s, k)
    return k[0], k[1]


def stuck(tiles, start):
    """States of the two sides, going through row tiles `start` and on, from which neither
    can go on: (row tile of the writers, whether its q is written, row tile of the issuer)."""
    n, seen, todo, found = len(tiles) - start, set(), [(0, 0, 0)], []
    while todo:
        state = todo.pop()
        if state in seen:
            continue
        seen.add(state)
        i, written, j = state
        after = []
        if i < n and not written:
            after.append((i, 1, j))  # completes phase i
        if i < n and written and (tiles[start + i] == 0 or j > i):
            after.append((i + 1, 0, j))  # has seen its products, or waits for none
        if j < n and (i + written) % 2 != j % 2:  # the phase it waits for is the one that has just completed
            after.append((i, written, j + 1))
        if not after and (i, j) != (n, n):
            found.append(state)
        todo += after
    return found


def test_the_model_finds_row_tiles_without_keys():
    assert stuck([0, 0, 1], 0) and stuck([0, 1], 0) and not stuck([1, 1, 2, 2], 0) and not stuck([0, 0, 1], 2)


CASES = [(90, 64, 2), (60, 64, 2), (0, 300, 3), (0, 2000, 4), (500, 64, 5), (0, 64, 2), (0, 5000, 19), (700, 2500, 25), (127, 33, 2)]
RANDOM = random.Random(0)
CASES += [(RANDOM.randrange(600), RANDOM.randrange(1, 900), RANDOM.randrange(1, 9)) for _ in range(300)]


def test_passes_begin_at_a_row_tile_with_keys_and_stay_in_step(lib):
    unseen = 0
    for ctx, rows, splits in CASES:
        at, count = 0, (rows + 31) // 32
        for s in range(splits):
            k0, k1 = segment(lib, ctx + rows, splits, s)
            assert k0 == at and k1 >= k0 and (k0 % 128 == 0 or k0 == k1)
            at = k1
            tiles = [lib.tiles_(ctx, rows, k0, k1, rt) for rt in range(count)]
            for rt, n in enumerate(tiles):  # of the keys that the tile's last row sees
                end = min(k1, ctx + min(rows, 32 * (rt + 1)))
                assert n == -(-max(0, end - k0) // 128)
                # a pass of this row tile alone
                assert lib.first_seeing_(ctx, k0, k1, rt, rt + 1) == (rt if n else rt + 1)
            first = lib.first_seeing_(ctx, k0, k1, 0, count)
            assert all(n == 0 for n in tiles[:first]) and all(n > 0 for n in tiles[first:])
            assert not stuck(tiles, first), (ctx, rows, s)
            unseen += first
        assert at == ctx + rows
    assert unseen > 100  # such windows were among them


def test_the_longest_sequences(lib):
    for keys, splits in ((1 << 24, 64), ((1 << 24) - 1, 63), (1, 64)):
        ends = [segment(lib, keys, splits, s) for s in range(splits)]
        assert ends[0][0] == 0 and ends[-1][1] == keys and all(a[1] == b[0] for a, b in zip(ends, ends[1:]))
