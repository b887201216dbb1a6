"""CPU checks of the mixture-of-experts operators: refusals of the C ABI and
of the binding before any device work, the plain forms the GPU tests use
against brute force and differences, and a model of the order in which the
expert products hand out their output tiles."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import dense_block_scaled_amd as dbs
from tests import _moe
from tests import test_gpu_moe as shapes

P = ctypes.c_void_p(1 << 20)          # 16-byte aligned, never dereferenced
P2 = ctypes.c_void_p((1 << 20) + 2)   # 2-byte aligned
P1 = ctypes.c_void_p((1 << 20) + 1)
N0 = ctypes.c_void_p(0)

EINVAL, EUNSUP = dbs.DBS_EINVAL, dbs.DBS_EUNSUPPORTED


def _refused(name, args, want):
    L = dbs.lib()
    assert getattr(L, name)(*args, N0) == want
    assert L.dbs_last_error().decode() != ""


# type, logits, T, E, k, renorm, experts, weights, offsets, rows, slots, ws, bytes
@pytest.mark.parametrize("args,want", [
    ((0, N0, 4, 8, 2, 1, P, P, P, P, P, N0, 0), EINVAL),
    ((2, P, 4, 8, 2, 1, P, P, P, P, P, N0, 0), EINVAL),            # type
    ((0, P, 0, 8, 2, 1, P, P, P, P, P, N0, 0), EINVAL),            # no tokens
    ((0, P, 4, 0, 2, 1, P, P, P, P, P, N0, 0), EINVAL),
    ((0, P, 4, 8, 0, 1, P, P, P, P, P, N0, 0), EINVAL),
    ((0, P, 4, 8, 9, 1, P, P, P, P, P, N0, 0), EINVAL),            # k above E
    ((0, P, 4, 1025, 2, 1, P, P, P, P, P, N0, 0), EINVAL),         # too many experts
    ((0, P, 4, 64, 17, 1, P, P, P, P, P, N0, 0), EUNSUP),          # k above 16
    ((0, P, 1 << 25, 64, 2, 1, P, P, P, P, P, P, 1 << 40), EINVAL),  # T k
    ((0, P, 4, 8, 2, 2, P, P, P, P, P, N0, 0), EINVAL),            # renormalize
    ((0, P, 4, 8, 2, 1, P, N0, P, P, P, N0, 0), EINVAL),           # null output
    ((0, P2, 4, 8, 2, 1, P, P, P, P, P, N0, 0), EINVAL),           # fp32 on 2 bytes
    ((0, P, 65, 8, 2, 1, P, P, P, P, P, N0, 0), EINVAL),           # workspace missing
    ((0, P, 65, 8, 2, 1, P, P, P, P, P, P, 4), EINVAL),            # too small
    ((0, P, 65, 8, 2, 1, P, P, P, P, P, P2, 1 << 20), EINVAL),     # misaligned
])
def test_route_refusals(args, want):
    _refused("moe_route", args, want)


def test_route_workspace_sizes():
    ws = dbs.lib().moe_route_workspace
    assert ws(64, 128, 8) == 0 and ws(0, 8, 2) == 0 and ws(100, 8, 9) == 0 and ws(100, 2000, 2) == 0
    assert ws(65, 8, 2) == (2 + 1) * 8 * 4


@pytest.mark.parametrize("args,want", [
    ((0, P, 4, 8, 2, 1, N0, P, P), EINVAL),
    ((0, P, 4, 8, 2, 1, P, P, N0), EINVAL),
    ((0, P, 4, 8, 9, 1, P, P, P), EINVAL),
    ((0, P, 4, 8, 2, 3, P, P, P), EINVAL),
    ((5, P, 4, 8, 2, 1, P, P, P), EINVAL),
])
def test_route_bwd_refusals(args, want):
    _refused("moe_route_bwd", args, want)


# X, W, D, offsets, rows, T, M, E, N, K, lw
@pytest.mark.parametrize("args,want", [
    ((N0, P, P, P, P, 4, 8, 2, 16, 16, 0), EINVAL),
    ((P, P, P, N0, P, 4, 8, 2, 16, 16, 0), EINVAL),
    ((P, P, P, P, P, 0, 8, 2, 16, 16, 0), EINVAL),
    ((P, P, P, P, P, 4, 0, 2, 16, 16, 0), EINVAL),
    ((P, P, P, P, P, 4, 8, 0, 16, 16, 0), EINVAL),
    ((P, P, P, P, P, 4, 8, 1025, 16, 16, 0), EINVAL),
    ((P, P, P, P, P, 4, 8, 2, 16, 12, 0), EINVAL),                 # K % 8
    ((P, P, P, P, P, 4, 8, 2, 1 << 22, 16, 0), EINVAL),
    ((P, P, P, P, N0, 4, 8, 2, 16, 16, 0), EINVAL),                # sorted, T != M
    ((P2, P, P, P, P, 4, 8, 2, 16, 16, 0), EINVAL),
    ((P, P2, P, P, P, 4, 8, 2, 16, 16, 0), EINVAL),
    ((P, P, P1, P, P, 4, 8, 2, 16, 16, 0), EINVAL),
    ((P, P, P, P2, P, 4, 8, 2, 16, 16, 0), EINVAL),
    ((P, P, P, P, P2, 4, 8, 2, 16, 16, 0), EINVAL),
    ((P, P, P, P, P, 4, 8, 2, 16, 16, 3), EINVAL),                 # layout
    ((P, P, P, P, P, 4, 8, 2, 12, 16, 1), EUNSUP),                 # MN-major, N % 8
    ((P, P, P, P, P, 4, 8, 2, 1 << 15, 1 << 15, 0), EUNSUP),       # a 2 GiB matrix
    ((P, P, P, P, P, 1 << 20, 8, 2, 16, 1 << 11, 0), EUNSUP),      # a 4 GiB gathered X
    ((P, P, P, P, P, (1 << 25) + 1, 8, 2, 16, 8, 0), EINVAL),
])
def test_product_refusals(args, want):
    _refused("gemm_moe_bf16", args, want)
    if args[-1] == 0 and want == EINVAL:
        _refused("gemm_moe_swiglu_bf16", args[:-1], want)


@pytest.mark.parametrize("name,args", [
    ("gemm_moe_bf16", (P, P, P, P, N0, 1 << 25, 1 << 25, 1, 1 << 18, 8, 0)),            # 2^19 x 2^13 tiles of 64 x 32
    ("gemm_moe_bf16", (P, P, P, P, P, 8, 1 << 25, 1024, 1 << 21, 8, 1)),                # 2^19 x 2^16
    ("gemm_moe_swiglu_bf16", (P, P, P, P, N0, 1 << 25, 1 << 25, 1, 1 << 17, 8)),        # 2^19 x 2^12
])
def test_products_refuse_more_tiles_than_32_bits_count(name, args):
    """Refused for the count itself, before any device is asked for."""
    _refused(name, args, EUNSUP)
    assert "tiles" in dbs.lib().dbs_last_error().decode()


def test_swiglu_product_width():
    _refused("gemm_moe_swiglu_bf16", (P, P, P, P, P, 4, 8, 2, (1 << 20) + 1, 16), EINVAL)


# type, dY, X, dW, offsets, rows, T, M, E, N, K, accumulate
@pytest.mark.parametrize("args,want", [
    ((0, N0, P, P, P, P, 4, 8, 2, 16, 16, 0), EINVAL),
    ((0, P, P, P, P, P, 4, 8, 2, 12, 16, 0), EINVAL),              # N % 8
    ((0, P, P, P, P, P, 4, 8, 2, 16, 20, 0), EINVAL),              # K % 8
    ((2, P, P, P, P, P, 4, 8, 2, 16, 16, 0), EINVAL),
    ((0, P, P, P, P, P, 4, 8, 2, 16, 16, 2), EINVAL),
    ((1, P, P, P, P, P, 4, 8, 2, 16, 16, 1), EUNSUP),              # accumulation in bf16
    ((0, P, P, P2, P, P, 4, 8, 2, 16, 16, 0), EINVAL),
    ((0, P, P, P, P, N0, 4, 8, 2, 16, 16, 0), EINVAL),
])
def test_dw_refusals(args, want):
    _refused("gemm_moe_dw_bf16", args, want)


@pytest.mark.parametrize("name,args", [
    ("swiglu_bf16", (N0, P, 4, 8)), ("swiglu_bf16", (P, P, 0, 8)), ("swiglu_bf16", (P, P, 4, 0)),
    ("swiglu_bf16", (P1, P, 4, 8)), ("swiglu_bf16", (P, P, (1 << 25) + 1, 8)),
    ("swiglu_bwd_bf16", (P, P, N0, 4, 8)), ("swiglu_bwd_bf16", (P, P1, P, 4, 8)), ("swiglu_bwd_bf16", (P, P, P, -1, 8)),
    ("moe_combine_bf16", (N0, P, P, P, 4, 8, 2, 16)), ("moe_combine_bf16", (P, P, P, P, 0, 8, 2, 16)),
    ("moe_combine_bf16", (P, P, P, P, 4, 0, 2, 16)), ("moe_combine_bf16", (P, P2, P, P, 4, 8, 2, 16)),
    ("moe_combine_bwd_bf16", (P, P, P, N0, P, 2, P, P, 4, 2, 16)),
    ("moe_combine_bwd_bf16", (P, P, P, P, P, 0, P, P, 4, 2, 16)),
    ("moe_combine_bwd_bf16", (P, P, P, P, P, 2, P, P, 4, 0, 16)),
])
def test_pointwise_refusals(name, args):
    _refused(name, args, EINVAL)


def test_combine_takes_at_most_16_rows_per_token():
    _refused("moe_combine_bf16", (P, P, P, P, 4, 8, 17, 16), EUNSUP)


def test_binding_refuses_what_is_not_on_the_gpu():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    i = torch.zeros(5, dtype=torch.int32)
    w = torch.zeros(4, 16, 8, dtype=torch.bfloat16)
    for call in (lambda: dbs.moe_route(x, 2), lambda: dbs.gemm_moe_bf16(x, w, i),
                 lambda: dbs.gemm_moe_swiglu_bf16(x, w, i), lambda: dbs.gemm_moe_dw_bf16(x, x, i), lambda: dbs.swiglu(x),
                 lambda: dbs.swiglu_backward(x[:, :4], x), lambda: dbs.moe_combine(x, i[:4].view(2, 2)),
                 lambda: dbs.moe_route_backward(x, i[:4].view(4, 1), torch.zeros(4, 1)),
                 lambda: dbs.moe_combine_backward(x, x, i[:4].view(4, 1), torch.zeros(4, 1), i)):
        with pytest.raises(ValueError, match="GPU tensor"):
            call()
    with pytest.raises(TypeError):
        dbs.swiglu(None)
    with pytest.raises(ValueError, match="dimensions"):
        dbs.moe_route(x[0], 2)
    with pytest.raises(ValueError, match="even"):
        dbs.swiglu(torch.zeros(4, 7, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="even"):
        dbs.gemm_moe_swiglu_bf16(x, torch.zeros(4, 15, 8, dtype=torch.bfloat16), i)
    with pytest.raises(TypeError):
        dbs.gemm_moe_dw_bf16(x, x, i, out_dtype=torch.float16)


@pytest.mark.parametrize("T", [(1 << 60) + 16, 1 << 60, (1 << 63) - 1, (1 << 25) + 1])
def test_routing_refuses_more_pairs_than_64_bits_count(T):
    """T k passes 2^64 here: it must not come back as a small number."""
    big = 1 << 62
    _refused("moe_route", (0, P, T, 64, 16, 1, P, P, P, P, P, P, big), EINVAL)
    _refused("moe_route_bwd", (0, P, T, 64, 16, 1, P, P, P), EINVAL)
    assert dbs.lib().moe_route_workspace(T, 64, 16) == 0


@pytest.mark.parametrize("place,bad", [(6, P2), (7, P2), (8, P1), (9, P2), (10, P2)])
def test_route_refuses_misaligned_outputs(place, bad):
    args = [1, P, 4, 8, 2, 1, P, P, P, P, P, N0, 0]
    args[place] = bad
    _refused("moe_route", tuple(args), EINVAL)


@pytest.mark.parametrize("kind,place,bad", [(0, 6, P2), (0, 7, P2), (0, 8, P2), (1, 8, P1)])
def test_route_bwd_refuses_misaligned_arrays(kind, place, bad):
    args = [kind, P, 4, 8, 2, 1, P, P, P]
    args[place] = bad
    _refused("moe_route_bwd", tuple(args), EINVAL)


@pytest.mark.parametrize("k", [2.5, "2", None])
def test_route_takes_whole_numbers_of_experts(k):
    """Not cut to a whole number without a word."""
    with pytest.raises(TypeError):
        dbs.moe_route(torch.zeros(4, 8), k)


# ------------------------------------------------- the plain forms themselves

def test_plain_routing_and_gradient():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 7))
    for renorm in (True, False):
        e, w = _moe.route(x, 3, renorm)
        for t in range(5):
            assert list(e[t]) == list(np.argsort(-x[t], kind="stable")[:3])
        if renorm:
            assert np.allclose(w.sum(1), 1)
        d = rng.standard_normal((5, 3))
        g, h = _moe.route_grad(x, e, d, renorm), 1e-6
        for t in range(5):
            for j in range(7):
                hi, lo = x.copy(), x.copy()
                hi[t, j] += h
                lo[t, j] -= h
                diff = ((_moe.route(hi, 3, renorm)[1] - _moe.route(lo, 3, renorm)[1]) * d).sum() / (2 * h)
                assert abs(diff - g[t, j]) < 1e-7
    off, rows, slots = _moe.routing(np.array([[1, 0], [-1, 1], [0, 2]]), 3)
    assert list(off) == [0, 2, 4, 5] and list(rows) == [0, 2, 0, 1, 2, -1]
    assert slots.tolist() == [[2, 0], [-1, 3], [1, 4]]


# ------------------------------------- which kernel a size goes to: the library's rules

def _tile_rows(T, M, E, N, mn, gate):
    return dbs.lib().dbs_moe_tile_rows(*map(ctypes.c_int64, (M or T, E, N)), int(mn), int(gate), 256)


def test_the_gpu_tests_shapes_reach_every_tile_height():
    """The library's own rule on 256 CUs: LARGE is for 256-row tiles, MID for
    128-row ones, and every form reaches each height three times."""
    g = shapes
    for which, want in ((g.LARGE, 256), (g.MID, 128)):
        for T, M, E, N, K, groups in which:
            assert _tile_rows(T, M, E, N, False, False) == want, (T, M, E, N, K, groups)
    for mn, gate in ((False, False), (False, True), (True, False)):
        reached = [_tile_rows(T, M, E, 2 * N if gate else N, mn, gate)
                   for T, M, E, N, K, _ in g.SHAPES + g.MID + g.LARGE + (g.HALF if gate else []) if not mn or N % 8 == 0]
        assert all(reached.count(h) >= 3 for h in (64, 128, 256)), (mn, gate, reached)


def test_the_gpu_tests_shapes_reach_both_tiles_of_dw():
    g = shapes
    for which, want in ((g.NARROW, 1), (g.WIDE, 0)):
        for T, M, E, N, K, groups in which:
            off = g._groups(groups, E, M or T, N + K + 3)
            stages = (ctypes.c_int32 * E)(*[-(-int(n) // 64) for n in np.diff(off)])
            assert dbs.lib().dbs_moe_dw_small(stages, E, N, K, 0, 0, 256) == want, (T, M, E, N, K, groups)


# ----------------------------------------- order of the products' output tiles

TM, BAND = 256, 4


def _tiles(rows, tiles_n):
    """(group, first row, blocks, column) of every tile id, as the kernel's
    table and search define them."""
    blocks = [(r % TM + 63) // 64 for r in rows]
    whole = np.concatenate([[0], np.cumsum([r // TM + (b == 4) for r, b in zip(rows, blocks)])])
    rest = {b: np.concatenate([[0], np.cumsum([x == b for x in blocks])]) for b in (1, 2, 3)}
    n = (whole[-1] + sum(rest[b][-1] for b in rest)) * tiles_n
    out = []
    for tid in range(n):
        i = tid
        if i < whole[-1] * tiles_n:
            g = int(np.searchsorted(whole[:-1], i // tiles_n, side="right")) - 1
            m = whole[g + 1] - whole[g]
            local = i - whole[g] * tiles_n
            band = local // (BAND * tiles_n)
            height = min(m - band * BAND, BAND)
            at = local - band * BAND * tiles_n
            out.append((g, (band * BAND + at % height) * TM, 4, at // height))
        else:
            i -= whole[-1] * tiles_n
            for b in (3, 2, 1):
                if i < rest[b][-1] * tiles_n:
                    g = int(np.searchsorted(rest[b][:-1], i // tiles_n, side="right")) - 1
                    out.append((g, rows[g] // TM * TM, b, i % tiles_n))
                    break
                i -= rest[b][-1] * tiles_n
    return out


@pytest.mark.parametrize("rows,tiles_n", [([1024] * 8, 3), ([0, 5, 0, 0, 300, 256, 255, 193, 192, 64, 65, 0], 2),
                                          ([3000, 1, 0, 2049], 5), ([0, 0, 0], 4), ([128], 1), ([255, 257, 511, 513], 7)])
def test_every_output_row_and_column_is_handed_out_once(rows, tiles_n):
    seen = {}
    for g, m0, blocks, col in _tiles(rows, tiles_n):
        for r in range(m0, min(m0 + 64 * blocks, rows[g])):
            key = (g, r, col)
            assert key not in seen
            seen[key] = True
    assert len(seen) == sum(rows) * tiles_n


@pytest.mark.parametrize("ntiles,nwg", [(1, 1), (7, 8), (256, 256), (1000, 256), (1023, 64), (513, 256)])
def test_the_snake_reaches_every_tile_once(ntiles, nwg):
    seen = []
    for self_ in range(min(ntiles, nwg)):
        r = 0
        while True:
            t = r * nwg + (nwg - 1 - self_ if r & 1 else self_)
            if t >= ntiles:
                break
            seen.append(t)
            r += 1
    # a workgroup ends at its first tile past the last: nothing may lie behind it
    assert sorted(seen) == list(range(ntiles))


# --------------------------------------------- LDS layout of the 256-row core

def _swz(r):
    return (r ^ (r >> 3)) & 7


def _mn_swz(r):
    return 4 * (r & 3) ^ 2 * (((r >> 3) ^ (r >> 4)) & 1)


def _kgroup(g):
    return (g >> 1) | (g & 1) << 1


@pytest.mark.parametrize("i,u,kk,block0", [(i, u, kk, b) for i in (0, 1) for u in (0, 1) for kk in (0, 1) for b in (0, 1)])
def test_k_major_part_reads(i, u, kk, block0):
    """Lane l reads row 32 block0 + 64 i + 16 u + l % 16, K 32 kk + 8 kgroup(l / 16)
    .., where the loads put it, and lanes l, l + 32 (eight of each) share no bank."""
    addr = []
    for lane in range(64):
        j, g = lane & 15, lane >> 4
        r = 32 * block0 + j
        base = r * 128 + ((_kgroup(g) ^ _swz(r)) << 4)
        a = (base ^ ((kk << 6) ^ (u << 5))) + (64 * i + 16 * u) * 128
        row, chunk = 32 * block0 + 64 * i + 16 * u + j, 4 * kk + _kgroup(g)
        # wave-load L = row / 8, lane (row % 8) * 8 + physical chunk
        assert a == row * 128 + ((chunk ^ _swz(row)) << 4)
        addr.append(a)
    for first in range(0, 32, 8):
        banks = [(addr[l] + 4 * d) // 4 % 64 for l in list(range(first, first + 8)) + list(range(first + 32, first + 40))
                 for d in range(4)]
        assert len(set(banks)) == 64


@pytest.mark.parametrize("i,u,kk,sub,block0", [(i, u, kk, s, b) for i in (0, 1) for u in (0, 1) for kk in (0, 1)
                                               for s in (0, 1) for b in (0, 1, 3) if not (i and b == 3)])
def test_mn_major_part_reads(i, u, kk, sub, block0):
    """Lane 16 g + j of a transposed read addresses K-row 32 kk + 8 kgroup(g) + 4 sub
    + j / 4 at columns 32 block0 + 64 i + 16 u + 4 (j % 4) ..; half-waves share no bank."""
    addr = []
    for lane in range(64):
        j, g = lane & 15, lane >> 4
        r = 8 * _kgroup(g) + (j >> 2)
        base = r * 256 + ((64 * block0 + 8 * (j & 3)) ^ (_mn_swz(r) << 4))
        a = (base ^ (128 * i + 32 * u)) + kk * 32 * 256 + 4 * sub * 256
        row, byte = 32 * kk + r + 4 * sub, 2 * (32 * block0 + 64 * i + 16 * u + 4 * (j & 3))
        # wave-load L = row / 4 of wave row / 8: lane (row % 4) * 16 + physical chunk
        w, rr = row // 8, row % 4
        phys = (byte // 16) ^ _mn_swz(8 * w + rr)
        assert a == row * 256 + 16 * phys + byte % 16
        addr.append(a)
    for half in (0, 32):
        banks = [(addr[l] + 4 * d) // 4 % 64 for l in range(half, half + 32) for d in range(2)]
        assert len(set(banks)) == 64
