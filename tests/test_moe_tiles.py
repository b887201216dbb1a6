"""The experts' products' own index arithmetic (csrc/moe_tiles.h), compiled for
the host: every output element is handed out once whatever the groups, the
snake reaches every tile, and the transposed LDS reads of both MN-major
layouts find what the loads put there, half-waves without bank conflicts."""
from __future__ import annotations

import ctypes
import subprocess
from pathlib import Path

import numpy as np
import pytest

from tests import test_lds_poison_build as poison

SOURCE = """#include "moe_tiles.h"
#include <algorithm>
namespace {
template <int TM>
int tiles(const int32_t *rows, int start, int E, int tiles_n, int tno, int32_t *out)
{
    static dbs::Table<TM> tab;
    tab.first[0] = start;
    tab.whole[0] = 0;
    for (auto &r : tab.rest) r[0] = 0;
    for (int e = 0; e < E; ++e) {
        tab.first[e + 1] = tab.first[e] + rows[e];
        tab.whole[e + 1] = tab.whole[e] + dbs::Table<TM>::whole_of(rows[e]);
        for (int b = 1; b < TM / 64; ++b)
            tab.rest[b - 1][e + 1] = (uint16_t)(tab.rest[b - 1][e] + dbs::Table<TM>::rest_of(rows[e], b));
    }
    const int n = dbs::count_tiles(tab, E, tiles_n);
    auto group_of = [&](const auto *at, int id) { return int(std::upper_bound(at, at + E, id) - at) - 1; };
    for (int id = 0; out && id <= n; ++id) {              // (one past the last)
        const dbs::RowTile t = dbs::find_tile(tab, E, n, tiles_n, tno, id, group_of);
        const int32_t v[5] = {t.m0, t.mend, t.n0, t.g, t.blocks};
        std::copy(v, v + 5, out + 5 * id);
    }
    return n;
}
}
extern "C" int tiles_of(int tm, const int32_t *rows, int start, int E, int tiles_n, int tno, int32_t *out)
{
    return tm == 64 ? tiles<64>(rows, start, E, tiles_n, tno, out)
                    : tm == 128 ? tiles<128>(rows, start, E, tiles_n, tno, out) : tiles<256>(rows, start, E, tiles_n, tno, out);
}
extern "C" int snake_of(int round, int nwg, int self) { return dbs::snake(round, nwg, self); }
extern "C" int kgroup_of(int g) { return dbs::kgroup(g); }
extern "C" int mn_swz_of(int r) { return dbs::mn_swz(r); }
extern "C" int narrow_swz_of(int r) { return dbs::narrow_swz(r); }
"""


@pytest.fixture(scope="module")
def host(tmp_path_factory):
    if not Path(poison.HIPCC).exists():
        pytest.skip("hipcc not available")
    d = tmp_path_factory.mktemp("moe_tiles")
    (d / "tiles.hip").write_text(SOURCE)
    subprocess.run([poison.HIPCC, "--offload-arch=gfx950", "-O1", "-std=c++17", "-shared", "-fPIC",
                    f"-I{poison.CSRC}", str(d / "tiles.hip"), "-o", str(d / "tiles.so")], check=True, capture_output=True)
    return ctypes.CDLL(str(d / "tiles.so"))


def _tiles(host, tm, rows, start, tiles_n, tno):
    c = (ctypes.c_int32 * len(rows))(*rows)
    n = host.tiles_of(tm, c, start, len(rows), tiles_n, tno, None)
    out = np.zeros((n + 1, 5), dtype=np.int32)
    host.tiles_of(tm, c, start, len(rows), tiles_n, tno, out.ctypes.data_as(ctypes.c_void_p))
    return out


GROUPS = [[1024] * 8, [0, 5, 0, 0, 300, 256, 255, 193, 192, 64, 65, 0], [3000, 1, 0, 2049], [0, 0, 0], [128], [1],
          [255, 257, 511, 513], [0] * 500 + [7] + [0] * 523, [64, 128, 192, 256, 320, 384, 448]]


def _random(seed):
    rng = np.random.default_rng(seed)
    return [int(v) for v in rng.exponential(200.0, rng.integers(1, 1025)) * rng.integers(0, 2, 1)[0]
            + rng.integers(0, 3, 1)[0]]


@pytest.mark.parametrize("tm", [64, 128, 256])
@pytest.mark.parametrize("rows,start,tiles_n", [(g, 17 * (i % 2), 1 + i % 4) for i, g in enumerate(GROUPS)]
                         + [(_random(s), s, 1 + s % 3) for s in range(6)])
def test_every_row_and_column_is_handed_out_once(host, tm, rows, start, tiles_n):
    tno = 128
    t = _tiles(host, tm, rows, start, tiles_n, tno)
    assert list(t[-1]) == [0, 0, 0, 0, 0]                   # past the last: nothing
    t = t[:-1]
    assert np.all(np.diff(t[:, 4]) <= 0)                    # by descending cost
    first = start + np.concatenate([[0], np.cumsum(rows)])
    seen = np.zeros((start + sum(rows), tiles_n), dtype=int)
    for m0, mend, n0, g, blocks in t:
        assert 1 <= blocks <= tm // 64 and first[g] <= m0 < mend == first[g + 1]
        assert (m0 - first[g]) % tm == 0 and n0 % tno == 0
        here = min(mend, m0 + 64 * blocks)
        assert here == min(mend, m0 + tm)                   # the blocks hold all of the tile's rows
        seen[m0:here, n0 // tno] += 1
    assert np.all(seen[start:] == 1) and np.all(seen[:start] == 0)


@pytest.mark.parametrize("ntiles,nwg", [(1, 1), (7, 8), (256, 256), (1000, 256), (1023, 64), (513, 256)])
def test_the_snake_ends_where_nothing_is_left(host, ntiles, nwg):
    seen = []
    for self_ in range(nwg):
        r = 0
        while (t := host.snake_of(r, nwg, self_)) < ntiles:
            seen.append(t)
            r += 1
        # a workgroup stops at its first tile past the last: all later ones are past it too
        assert all(host.snake_of(q, nwg, self_) >= ntiles for q in range(r, r + 4))
    assert sorted(seen) == list(range(ntiles))


# name, swizzle, bytes of a K-row, K-rows of a wave-load
LAYOUTS = [("mn_swz_of", 256, 4), ("narrow_swz_of", 128, 8)]


@pytest.mark.parametrize("swz,row_bytes,rows", LAYOUTS)
@pytest.mark.parametrize("kk", [0, 1])
@pytest.mark.parametrize("sub", [0, 1])
def test_transposed_reads(host, swz, row_bytes, rows, kk, sub):
    """Lane 16 g + j addresses K-row 32 kk + 8 kgroup(g) + 4 sub + j / 4 at
    columns 16 block + 4 (j % 4) .. of a part that wave-loads filled: lane i of
    one puts logical chunk (i % chunks) ^ swz(K-row) at physical chunk i % chunks."""
    s = getattr(host, swz)
    chunks = row_bytes // 16
    for block in range(row_bytes // 32):
        addr = []
        for lane in range(64):
            j, g = lane & 15, lane >> 4
            r = 8 * host.kgroup_of(g) + (j >> 2)
            # the kernel's form: the swizzle of row r, and the steps of kk and sub added behind it
            a = r * row_bytes + ((32 * block + 8 * (j & 3)) ^ (s(r) << 4)) + (32 * kk + 4 * sub) * row_bytes
            row, byte = 32 * kk + 4 * sub + r, 32 * block + 8 * (j & 3)
            load, i = row // rows, [i for i in range(64) if i // chunks == row % rows
                                    and ((i % chunks) ^ s(row)) == byte // 16]
            assert len(i) == 1 and a == load * 1024 + 16 * i[0] + byte % 16
            addr.append(a)
        for half in (0, 32):
            banks = [(addr[l] + 4 * d) // 4 % 64 for l in range(half, half + 32) for d in range(2)]
            assert len(set(banks)) == 64


def test_kgroup_is_a_permutation(host):
    assert sorted(host.kgroup_of(g) for g in range(4)) == [0, 1, 2, 3]
