"""The tile search of the expert-grouped products on the CPU: the header's
arithmetic, with the wave's scan written out, over offsets of every kind.  Each
block gets a tile inside an expert's rows or none; offsets that do not decrease
give every row and column exactly once."""
import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "conv_implicit_gemm_amd", "csrc")

SHIM = r"""
#include "expert_tiles.hpp"
using namespace ox;

static int clampi(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

struct Round { int lo[64], hi[64], n[64], s[64]; };
// 64 experts' rows, tiles and their inclusive 32-bit scan, as the wave holds them
static void scan(const int* off, int E, int T, int BM, int base, Round& r) {
  unsigned sum = 0;
  for (int l = 0; l < 64; ++l) {
    r.lo[l] = r.hi[l] = 0;
    if (base + l < E) {
      r.lo[l] = clampi(off[base + l], 0, T);
      r.hi[l] = clampi(off[base + l + 1], r.lo[l], T);
    }
    r.n[l] = ceil_div(r.hi[l] - r.lo[l], BM);
    r.s[l] = (int)(sum += (unsigned)r.n[l]);
  }
}

extern "C" long long tile_count(const int* off, int E, int T, int BM) {
  Round r;
  long long total = 0;
  for (int base = 0; base < E; base += 64) {
    scan(off, E, T, BM, base, r);
    total += r.s[63];
  }
  return total;
}

extern "C" int up(int n, int d) { return ceil_div(n, d); }

extern "C" long long bound(int T, int E, int BM) { return expert_tile_bound(T, E, BM); }

// out: expert, row0, rows, column tile; returns whether block b has a tile
extern "C" int find(const int* off, int E, int T, int BM, int NT, long long total, int b, int* out) {
  if (!block_has_tile(b, total, NT, expert_tile_bound(T, E, BM))) return 0;
  const int all = (int)total * NT, q = all / 8, rest = all % 8, x = b % 8;      // an XCD's contiguous range
  const int u = (x < rest ? x * (q + 1) : rest * (q + 1) + (x - rest) * q) + b / 8;
  int t, nt;
  tile_order(u, (int)total, NT, t, nt);
  long long before = 0;
  for (int base = 0; base < E; base += 64) {
    Round r;
    scan(off, E, T, BM, base, r);
    for (int l = 0; l < 64; ++l)
      if (before + r.s[l] > t) {
        ExpertTile k;
        if (!expert_tile_rows(r.lo[l], r.hi[l], t - before - (r.s[l] - r.n[l]), BM, k)) return 0;
        out[0] = base + l;
        out[1] = k.row0;
        out[2] = k.rows;
        out[3] = nt;
        return 1;
      }
    before += r.s[63];
  }
  return 0;
}
"""


@pytest.fixture(scope="module")
def tiles(tmp_path_factory):
    gxx = shutil.which("g++")
    if not gxx:
        pytest.skip("needs g++")
    d = tmp_path_factory.mktemp("tiles")
    (d / "shim.cpp").write_text(SHIM)
    lib = str(d / "shim.so")
    subprocess.run([gxx, "-std=c++17", "-O2", "-Wall", "-Werror", "-fsanitize=undefined", "-fno-sanitize-recover",
                    "-shared", "-fPIC", "-I" + CSRC, str(d / "shim.cpp"), "-o", lib], check=True)
    f = ctypes.CDLL(lib)
    f.bound.restype = f.tile_count.restype = ctypes.c_longlong
    return f


def search(f, off, T, BM, NT, blocks):
    E = len(off) - 1
    p = np.ascontiguousarray(off, np.int32).ctypes.data_as(ctypes.c_void_p)
    total = f.tile_count(p, E, T, BM)
    out = (ctypes.c_int * 4)()
    for b in blocks:
        if f.find(p, E, T, BM, NT, ctypes.c_longlong(total), int(b), out):
            yield tuple(out)


def inside(off, T, BM, NT, tile):
    e, row0, rows, nt = tile
    assert 0 <= e < len(off) - 1 and 0 <= nt < NT and 0 < rows <= BM and 0 <= row0 and row0 + rows <= T, tile


@pytest.mark.parametrize("BM", [32, 64, 256])
@pytest.mark.parametrize("seed", range(6))
def test_rows_and_columns_are_covered_once(tiles, BM, seed):
    rng = np.random.default_rng(seed)
    E, T, NT = int(rng.integers(1, 200)), int(rng.integers(1, 3000)), int(rng.integers(1, 6))
    off = np.sort(rng.integers(0, T + 1, E + 1))
    blocks = tiles.bound(T, E, BM) * NT
    seen = np.zeros((T, NT), int)
    owner = np.full(T, -1)
    for e, row0, rows, nt in search(tiles, off, T, BM, NT, range(blocks)):
        seen[row0:row0 + rows, nt] += 1
        owner[row0:row0 + rows] = e
    rows = np.arange(T)
    mine = (rows >= off[0]) & (rows < off[-1])
    assert (seen == mine[:, None]).all()
    assert (owner[mine] == np.searchsorted(off, rows[mine], side="right") - 1).all()


def test_offsets_whose_tiles_leave_32_bits_give_no_tile_outside(tiles):
    # 32768 experts whose offsets swing over 131072 rows: 2^26 row tiles of 32
    # rows, times 32 column tiles, are 2^31
    E, T, BM, NT = 32768, 131072, 32, 32
    off = np.where(np.arange(E + 1) % 2, T, 0)
    blocks = tiles.bound(T, E, BM) * NT
    assert blocks < 2 ** 31
    for tile in search(tiles, off, T, BM, NT, np.linspace(0, blocks - 1, 500).astype(int)):
        inside(off, T, BM, NT, tile)


@pytest.mark.parametrize("E,T,BM,NT", [(128, 2 ** 31 - 1, 32, 1), (64, 2 ** 31 - 1, 64, 1), (4096, 2 ** 20, 32, 32),
                                       (70, 40, 32, 5), (1000, 513, 256, 3)])
@pytest.mark.parametrize("seed", range(4))
def test_wild_offsets_give_no_tile_outside(tiles, E, T, BM, NT, seed):
    rng = np.random.default_rng([seed, E])
    off = rng.integers(-2 ** 31, 2 ** 31, E + 1) if seed % 2 else rng.integers(0, T + 1, E + 1)
    blocks = min(tiles.bound(T, E, BM) * NT, 2 ** 31 - 1)
    for tile in search(tiles, off, T, BM, NT, np.linspace(0, blocks - 1, 300).astype(int)):
        inside(off, T, BM, NT, tile)


@pytest.mark.parametrize("d", [16, 32, 64, 127, 128, 256, 512])
def test_blocks_of_sizes_next_to_the_limit(tiles, d):
    # K, N and T go up to 2^31 - 1 elements; one block too few or a negative
    # count leaves sums out
    for n in [0, 1, d - 1, d, d + 1] + [2 ** 31 - i for i in range(1, 2 * d)]:
        assert tiles.up(n, d) == -(-n // d), (n, d)
