"""The workgroups of an attention call and what they find, from its sizes (compiled for the host)."""

import ctypes
import os
import random
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

PROBE = r"""
#include "attn_grid.h"
extern "C" void grid(int64_t blocks, int64_t* xy) {
  const tb::GridXY g = tb::grid_of(blocks);
  xy[0] = g.x;
  xy[1] = g.y;
}
extern "C" int64_t tokens(int64_t max_q, int64_t total_q) { return tb::most_tokens(max_q, total_q); }
extern "C" int64_t tiles(int64_t total_q, int64_t B, int64_t group, int64_t few, int64_t tile) {
  return tb::most_row_tiles(total_q, B, group, few, tile);
}
extern "C" int head(int64_t at, int tiles) { return tb::head_of(at, tiles); }
"""


@pytest.fixture(scope="module")
def probe(tmp_path_factory):
    if shutil.which("g++") is None:
        pytest.skip("no host compiler")
    d = tmp_path_factory.mktemp("grid")
    src, so = d / "probe.cpp", d / "probe.so"
    src.write_text(PROBE)
    csrc = os.path.join(ROOT, "ternary_weights_hadamard_amd", "csrc")
    subprocess.run(["g++", "-O1", "-shared", "-fPIC", f"-I{csrc}", str(src), "-o", str(so)], check=True)
    lib = ctypes.CDLL(str(so))
    i64 = ctypes.c_int64
    lib.grid.argtypes = [i64, ctypes.POINTER(i64)]
    lib.tokens.argtypes, lib.tokens.restype = [i64] * 2, i64
    lib.tiles.argtypes, lib.tiles.restype = [i64] * 5, i64
    lib.head.argtypes = [i64, ctypes.c_int]
    return lib


def _xy(lib, blocks):
    xy = (ctypes.c_int64 * 2)()
    lib.grid(blocks, xy)
    return xy[0], xy[1]


def test_grid_holds_every_accepted_size(probe):
    # 2^27 tokens of 2^16 heads are 2^36 row tiles; 65535 sequences of 65535 heads have an item more each, of either kind
    for blocks in (1, 512, 1024, (1 << 23) - 1, 1 << 23, (1 << 23) + 1, 1 << 24, 1 << 32, 8192 * 8 << 16,
                   65535 * 65535, (1 << 36) + 2 * 65535 * 65535):
        x, y = _xy(probe, blocks)
        assert 1 <= x and x * 256 < 1 << 32 and 1 <= y <= 65535
        assert blocks <= x * y < blocks + x


def test_row_tiles_bound_the_ones_there_are(probe):
    rng = random.Random(1)
    for _ in range(2000):
        group, few, tile = rng.choice([1, 2, 3, 5, 8, 16, 17, 40]), rng.choice([0, 16]), 128
        n = [rng.choice([0, 1, rng.randint(0, 20), rng.randint(0, 900)]) for _ in range(rng.randint(1, 40))]
        max_q = rng.choice([max(n), max(n) + 7, 1 << 27, max(max(n) // 2, 1)])
        total = sum(n) + rng.choice([0, 0, 5, 400])
        rows = [min(x, probe.tokens(max_q, total)) * group for x in n]
        there = sum(-(-r // tile) for r in rows if r > few)
        bound = probe.tiles(total, len(n), group, few, tile)
        assert there <= bound <= total * group // tile + len(n)


def test_lengths_and_not_max_q_make_the_grid(probe):
    # 8191 single tokens and a prompt of 200: 64 query heads on 8
    assert probe.tokens(1 << 20, 8391) == 8391
    assert probe.tiles(8391, 8192, 8, 16, 128) == 8391 * 8 // 128 + 8391 // 3
    # 255 single tokens of 5 rows each cannot all have more than 16: at most a fourth of them
    assert probe.tiles(2303, 256, 5, 16, 128) == 2303 * 5 // 128 + 256
    assert probe.tiles(300, 256, 5, 16, 128) == 300 * 5 // 128 + 75


def test_head_of_a_place_past_32_bits(probe):
    for heads, tiles in ((8, 1000), (128, 1 << 25), (129, 1 << 25), (65535, (1 << 25) - 3), (65535, 1), (300, 1 << 24)):
        for h in (0, 1, heads // 2, heads - 1):
            for at in (h * tiles, h * tiles + tiles // 2, (h + 1) * tiles - 1):
                assert probe.head(at, tiles) == h
